// RMS norm with the residual's addition and FP8 output, and the FP8 quantiser.
//
// The layer's input is the normed residual stream, and its output joins that
// stream before the next norm; the routed experts read bf16, the FP8 shared
// expert reads E4M3 with a scale per 128 (the block rule is in fp8.cuh).
#include "common.cuh"
#include "fp8.cuh"
#include "fp8.h"
#include "ptx.cuh"

namespace moe {
namespace {

// A unit is four neighbouring blocks of a row (512 elements), one warp, 16 fp32
// values per lane. VEC: eight lanes per block, a lane holding elements 8 j .. 8 j
// + 7 and 64 + 8 j .. of its block (16-byte accesses; the scale arithmetic, two
// quotients, runs once for all four blocks: with a warp per block the kernels
// were bound by instructions, 13.6 against 9 us for 4096 x 4096 bf16). Otherwise
// the warp takes the blocks one after the other, value 4 b + i being element
// lane + 32 i of block b (coalesced scalar accesses at any alignment).
constexpr int kUnit = 4 * kFp8Block;

template <bool VEC>
__device__ __forceinline__ int elem_of(int lane, int i) {
    return VEC ? (lane >> 3) * kFp8Block + (i >> 3) * 64 + 8 * (lane & 7) + (i & 7)
               : (i >> 2) * kFp8Block + lane + 32 * (i & 3);
}

// *p, or 0 when !in. A 2-byte load fills a 32-bit register: left to the compiler it
// fills half of one, and every load then waits for the one before (3001 x 5003 bf16
// by tiles 60 us instead of 14.8, by rows 21.7 instead of 15.2).
__device__ __forceinline__ float load_one(const float *p, bool in) { return in ? *p : 0.f; }
__device__ __forceinline__ float load_one(const uint16_t *p, bool in) {
    uint32_t u;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t@p ld.global.u16 %0, [%1];\n\t}"
                 : "=r"(u)
                 : "l"(p), "r"((uint32_t)in)
                 : "memory");
    return __uint_as_float(u << 16);
}

// The unit at p, of which n elements exist (the others are 0; VEC: n is a multiple of 8).
template <typename TYPE, bool VEC>
__device__ __forceinline__ void load_unit(const TYPE *p, int lane, int n, float (&v)[16]) {
    if constexpr (VEC) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int e = elem_of<true>(lane, 8 * h);
            float *o = &v[8 * h];
            if (e < n) {
                if constexpr (sizeof(TYPE) == 4) {
                    const float4 f = reinterpret_cast<const float4 *>(p + e)[0], g = reinterpret_cast<const float4 *>(p + e)[1];
                    o[0] = f.x; o[1] = f.y; o[2] = f.z; o[3] = f.w;
                    o[4] = g.x; o[5] = g.y; o[6] = g.z; o[7] = g.w;
                } else {
                    const uint4 u = *reinterpret_cast<const uint4 *>(p + e);
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        o[2 * i] = __uint_as_float(w[i] << 16);
                        o[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = 0.f;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int e = elem_of<false>(lane, i);
            v[i] = load_one(p + e, e < n);
        }
    }
}

template <typename TYPE, bool VEC>
__device__ __forceinline__ void store_unit(TYPE *p, int lane, int n, const float (&v)[16]) {
    if constexpr (VEC) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int e = elem_of<true>(lane, 8 * h);
            const float *o = &v[8 * h];
            if (e < n) {
                if constexpr (sizeof(TYPE) == 4) {
                    reinterpret_cast<float4 *>(p + e)[0] = make_float4(o[0], o[1], o[2], o[3]);
                    reinterpret_cast<float4 *>(p + e)[1] = make_float4(o[4], o[5], o[6], o[7]);
                } else {
                    *reinterpret_cast<uint4 *>(p + e) =
                        make_uint4(f32x2_to_bf16x2_rn(o[0], o[1]), f32x2_to_bf16x2_rn(o[2], o[3]),
                                   f32x2_to_bf16x2_rn(o[4], o[5]), f32x2_to_bf16x2_rn(o[6], o[7]));
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int e = elem_of<false>(lane, i);
            if (e < n) {
                if constexpr (sizeof(TYPE) == 4) p[e] = v[i];
                else p[e] = (uint16_t)f32x2_to_bf16x2_rn(v[i], 0.f);
            }
        }
    }
}

// The unit's E4M3 codes at p and its blocks' scales at sc[0 .. 3] (those that exist). v is scaled on the way.
template <bool VEC>
__device__ __forceinline__ void quant_unit(float (&v)[16], int lane, int n, bool pow2, uint8_t *p, float *sc) {
    if constexpr (VEC) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) m = max(m, abs_bits(v[i]));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const BlockScale b = block_scale(m, pow2);
        scale_values(v, b);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int e = elem_of<true>(lane, 8 * h);
            const float *o = &v[8 * h];
            if (e < n)
                *reinterpret_cast<uint2 *>(p + e) =
                    make_uint2(f32x4_to_e4m3x4(o[0], o[1], o[2], o[3]), f32x4_to_e4m3x4(o[4], o[5], o[6], o[7]));
        }
        if ((lane & 7) == 0 && (lane >> 3) * kFp8Block < n) sc[lane >> 3] = b.scale;
    } else {
        // the four blocks' scales at once, lane k that of block k
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float *o = &v[4 * k];
            const uint32_t a = max(max(abs_bits(o[0]), abs_bits(o[1])), max(abs_bits(o[2]), abs_bits(o[3])));
            const uint32_t r = __reduce_max_sync(0xffffffffu, a);
            if ((lane & 3) == k) m = r;
        }
        const BlockScale mine = block_scale(m, pow2);
        if (lane < 4 && lane * kFp8Block < n) sc[lane] = mine.scale;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float o[4] = {v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]};
            BlockScale b;
            b.hi = __shfl_sync(0xffffffffu, mine.hi, k);
            b.lo = __shfl_sync(0xffffffffu, mine.lo, k);
            b.pre = __shfl_sync(0xffffffffu, mine.pre, k);
            scale_values(o, b);
            const uint32_t q = f32x4_to_e4m3x4(o[0], o[1], o[2], o[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = elem_of<false>(lane, 4 * k + i);
                if (e < n) p[e] = (uint8_t)(q >> (8 * i));
            }
        }
    }
}

struct NormArgs {
    const void *x, *res, *w;
    void *sum;
    uint16_t *y;
    uint8_t *codes;
    float *scales;
    int64_t ldx, ldr, ldy, ldq;
    int d, nb;        // elements and 128-blocks of a row
    int w_bf16, pow2;
    float eps;
};

struct NoRes {};

// One CTA per row, NU units per warp (unit u goes to warp u mod warps): the row
// stays in registers between the sum of squares and the scaling, so every input
// is read once and every output written once.
//   s = x + r,  n = (s / sqrt(mean s^2 + eps)) * w:  sums and products fp32,
// one rounding per output (the bf16 and the FP8 output both start from fp32 n).
template <typename X, typename R, bool VEC, int NU>
__global__ void __launch_bounds__(512) rms_norm_kernel(const __grid_constant__ NormArgs a) {
    constexpr bool HAS_RES = !std::is_same<R, NoRes>::value;
    __shared__ float part[16];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int64_t row = blockIdx.x;
    grid_dep_wait();
    grid_dep_launch();
    float v[NU][16];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
        const int at = (warp + i * warps) * kUnit, n = a.d - at;
        load_unit<X, VEC>(static_cast<const X *>(a.x) + row * a.ldx + at, lane, n, v[i]);
        if constexpr (HAS_RES) {
            float r[16];
            load_unit<R, VEC>(static_cast<const R *>(a.res) + row * a.ldr + at, lane, n, r);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[i][j] += r[j];
        }
    }
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) ss = fmaf(v[i][j], v[i][j], ss);
    ss = warp_sum(ss);
    if (lane == 0) part[warp] = ss;
    __syncthreads();
    ss = warp_sum(lane < warps ? part[lane] : 0.f);
    const float inv = 1.0f / sqrtf(ss / (float)a.d + a.eps);
#pragma unroll
    for (int i = 0; i < NU; ++i) {
        const int at = (warp + i * warps) * kUnit, n = a.d - at;
        if (n <= 0) break;
        if constexpr (HAS_RES) {
            if (a.sum) store_unit<R, VEC>(static_cast<R *>(a.sum) + row * a.ldr + at, lane, n, v[i]);
        }
        if (a.w) {
            float w[16];
            if (a.w_bf16) load_unit<uint16_t, VEC>(static_cast<const uint16_t *>(a.w) + at, lane, n, w);
            else load_unit<float, VEC>(static_cast<const float *>(a.w) + at, lane, n, w);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[i][j] = v[i][j] * inv * w[j];
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[i][j] *= inv;
        }
        if (a.y) store_unit<uint16_t, VEC>(a.y + row * a.ldy + at, lane, n, v[i]);
        if (a.codes)
            quant_unit<VEC>(v[i], lane, n, a.pow2, a.codes + row * a.ldq + at, a.scales + row * a.nb + at / kFp8Block);
    }
}

template <typename X, typename R, bool VEC>
cudaError_t norm_launch(const NormArgs &a, int T, cudaStream_t s) {
    // one unit per warp up to 16 warps (8192 elements), then two and four
    const int units = ceil_div(a.d, kUnit), nu = units <= 16 ? 1 : units <= 32 ? 2 : 4;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(T);
    cfg.blockDim = dim3(32 * ceil_div(units, nu));
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    count_launches(1);
    switch (nu) {
        case 1: return cudaLaunchKernelEx(&cfg, rms_norm_kernel<X, R, VEC, 1>, a);
        case 2: return cudaLaunchKernelEx(&cfg, rms_norm_kernel<X, R, VEC, 2>, a);
        default: return cudaLaunchKernelEx(&cfg, rms_norm_kernel<X, R, VEC, 4>, a);
    }
}

template <typename X, bool VEC>
cudaError_t norm_res(const NormArgs &a, int T, int res_type, cudaStream_t s) {
    if (!a.res) return norm_launch<X, NoRes, VEC>(a, T, s);
    return res_type == MOE_T_BF16 ? norm_launch<X, uint16_t, VEC>(a, T, s) : norm_launch<X, float, VEC>(a, T, s);
}

// ---------------------------------------------------------------- quantiser

struct QuantArgs {
    const void *v;
    uint8_t *codes;
    float *scales;
    int64_t lds, ldq, rows;
    int cols, nb, pow2;
};

// Units per warp, all loads in flight at once (4096 x 4096 bf16: 9.1 us; when each unit had its scales to itself,
// 9.8, and before that 9.5, 10.1 with one unit and 9.8 with four).
constexpr int kRowUnits = 2;

// A lane's 16 values of a unit as the bits they have in memory: fp32 words, or two
// bf16 per word, whose largest magnitude takes half of the instructions (4096 x 4096
// bf16: 9.1 us, 87% of the measured HBM rate; with values widened on loading a tenth
// more).
template <typename X>
struct RawUnit {
    static constexpr int kPer = 4 / (int)sizeof(X), kWords = 16 / kPer;
    uint32_t w[kWords];

    __device__ __forceinline__ void load(const X *p, int lane, int n) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int e = elem_of<true>(lane, 8 * h);
#pragma unroll
            for (int i = 0; i < kWords / 8; ++i) {
                uint4 u = make_uint4(0, 0, 0, 0);
                if (e < n) u = reinterpret_cast<const uint4 *>(p + e)[i];
                uint32_t *o = &w[h * kWords / 2 + 4 * i];
                o[0] = u.x; o[1] = u.y; o[2] = u.z; o[3] = u.w;
            }
        }
    }
    __device__ __forceinline__ uint32_t largest() const {  // bits of the largest magnitude, as fp32
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            m = kPer == 1 ? max(m, w[i] & 0x7FFFFFFFu) : __vmaxu2(m, w[i] & 0x7FFF7FFFu);
        return kPer == 1 ? m : max(m << 16, m & 0xFFFF0000u);
    }
    __device__ __forceinline__ float value(int i) const {
        if constexpr (kPer == 1) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
    }
    __device__ __forceinline__ uint32_t block_largest() const {  // of the lane's block
        uint32_t m = largest();
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        return m;
    }
    __device__ __forceinline__ void encode(int lane, int n, const BlockScale &b, uint8_t *p) const {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int e = elem_of<true>(lane, 8 * h);
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = value(8 * h + i);
            scale_values(o, b);
            if (e < n)
                *reinterpret_cast<uint2 *>(p + e) =
                    make_uint2(f32x4_to_e4m3x4(o[0], o[1], o[2], o[3]), f32x4_to_e4m3x4(o[4], o[5], o[6], o[7]));
        }
    }
};
template <typename X>
struct WideUnit {  // the same for rows at any alignment, widened
    float v[16];
    __device__ __forceinline__ void load(const X *p, int lane, int n) { load_unit<X, false>(p, lane, n, v); }
    __device__ __forceinline__ void quantise(int lane, int n, bool pow2, uint8_t *p, float *sc) {
        quant_unit<false>(v, lane, n, pow2, p, sc);
    }
};

// Scales by rows: a warp per kRowUnits neighbouring units of a row.
template <typename X, bool VEC>
__global__ void __launch_bounds__(256) fp8_quant_rows_kernel(const __grid_constant__ QuantArgs a) {
    constexpr int kSpan = kRowUnits * kUnit;
    const int lane = threadIdx.x & 31;
    const uint32_t w = blockIdx.x * 8u + (threadIdx.x >> 5), per_row = (uint32_t)(a.cols + kSpan - 1) / kSpan;
    const uint32_t row = w / per_row;
    const int at = (int)(w - row * per_row) * kSpan;
    grid_dep_wait();
    grid_dep_launch();
    if (row >= (uint32_t)a.rows) return;
    const X *src = static_cast<const X *>(a.v) + (int64_t)row * a.lds + at;
    typename std::conditional<VEC, RawUnit<X>, WideUnit<X>>::type v[kRowUnits];
#pragma unroll
    for (int u = 0; u < kRowUnits; ++u) v[u].load(src + u * kUnit, lane, a.cols - at - u * kUnit);
    uint8_t *dst = a.codes + (int64_t)row * a.ldq + at;
    float *sc = a.scales + (int64_t)row * a.nb + at / kFp8Block;
    if constexpr (VEC) {
        // of the eight lanes of a block, even ones work out its scale in the first unit, odd ones in the second
        static_assert(kRowUnits == 2, "two units");
        const uint32_t m0 = v[0].block_largest(), m1 = v[1].block_largest();
        const BlockScale mine = block_scale(lane & 1 ? m1 : m0, a.pow2);
        const int block = (lane & 1) * 4 + (lane >> 3);
        if ((lane & 6) == 0 && at + block * kFp8Block < a.cols) sc[block] = mine.scale;
#pragma unroll
        for (int u = 0; u < kRowUnits; ++u) {
            BlockScale b;
            b.hi = __shfl_sync(0xffffffffu, mine.hi, (lane & 30) | u);
            b.lo = __shfl_sync(0xffffffffu, mine.lo, (lane & 30) | u);
            b.pre = __shfl_sync(0xffffffffu, mine.pre, (lane & 30) | u);
            v[u].encode(lane, a.cols - at - u * kUnit, b, dst + u * kUnit);
        }
    } else {
#pragma unroll
        for (int u = 0; u < kRowUnits; ++u) {
            const int n = a.cols - at - u * kUnit;
            if (n <= 0) break;
            v[u].quantise(lane, n, a.pow2, dst + u * kUnit, sc + u * kUnit / kFp8Block);
        }
    }
}

// A 128 x 128 block in a CTA's registers, every value once, as the bits it has in
// memory: fp32 words, or two bf16 per word (half of the registers, four CTAs per
// SM: 3001 x 5000 bf16 8.5 us, 16.7 as fp32 in three; with five, which leaves 48
// registers, 10.9). VEC: 16-byte accesses, 16 or 32 threads per row; otherwise
// a warp per row, lane l holding l, l + 32, l + 64, l + 96.
template <typename X, bool VEC>
struct Tile {
    static constexpr int kPer = 4 / (int)sizeof(X), kWords = 64 / kPer;  // values per word, words per thread
    static constexpr int kEl = VEC ? 4 * kPer : 4;                      // values of a piece, all in one row
    static constexpr int kPieces = 64 / kEl, kPieceWords = kWords / kPieces;
    static constexpr int kRowThreads = kFp8Block / kEl, kRows = 256 / kRowThreads;  // rows per pass of the CTA

    static __device__ __forceinline__ void load(const X *p, int t, int n, uint32_t *w) {  // p: the row's start
        if constexpr (VEC) {
            uint4 u = make_uint4(0, 0, 0, 0);
            if (kEl * t < n) u = *reinterpret_cast<const uint4 *>(p + kEl * t);
            w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
        } else if constexpr (kPer == 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(load_one(p + t + 32 * i, t + 32 * i < n));
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                w[i] = __float_as_uint(load_one(p + t + 64 * i, t + 64 * i < n)) >> 16 |
                       __float_as_uint(load_one(p + t + 64 * i + 32, t + 64 * i + 32 < n));
        }
    }
    static __device__ __forceinline__ float value(const uint32_t *w, int i) {  // i-th of the piece
        if constexpr (kPer == 1) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
    }
    static __device__ __forceinline__ void store(const uint32_t *w, int t, int n, const BlockScale &s, uint8_t *p) {
        float o[kEl];
#pragma unroll
        for (int i = 0; i < kEl; ++i) o[i] = value(w, i);
        scale_values(o, s);
        uint32_t q[kEl / 4];
#pragma unroll
        for (int i = 0; i < kEl / 4; ++i) q[i] = f32x4_to_e4m3x4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        if constexpr (!VEC) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (t + 32 * j < n) p[t + 32 * j] = (uint8_t)(q[0] >> (8 * j));
        } else if (kEl * t < n) {
            if constexpr (kEl == 4) *reinterpret_cast<uint32_t *>(p + kEl * t) = q[0];
            else *reinterpret_cast<uint2 *>(p + kEl * t) = make_uint2(q[0], q[1]);
        }
    }
};

// Scales by 128 x 128 blocks: one CTA of 8 warps per block. 2048 x 4096 fp32 (512
// blocks on 444 CTAs that are there at once): 8.5 us, 76% of the measured HBM
// rate; 4096 x 4096: 13.9 us, 93%.
template <typename X, bool VEC>
__global__ void __launch_bounds__(256, sizeof(X) == 2 && VEC ? 4 : 3) fp8_quant_tile_kernel(const __grid_constant__ QuantArgs a) {
    using B = Tile<X, VEC>;
    __shared__ uint32_t part[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = threadIdx.x % B::kRowThreads;
    const int64_t r0 = (int64_t)(blockIdx.x / a.nb) * kFp8Block + threadIdx.x / B::kRowThreads;
    const int b = blockIdx.x % a.nb, n = min(kFp8Block, a.cols - b * kFp8Block);
    const int left = (int)min(a.rows - r0, (int64_t)kFp8Block);  // rows from this thread's first one on
    const X *src = static_cast<const X *>(a.v) + r0 * a.lds + b * kFp8Block;
    uint8_t *dst = a.codes + r0 * a.ldq + b * kFp8Block;
    uint32_t w[B::kPieces][B::kPieceWords];
    uint32_t m = 0;
    grid_dep_wait();
    grid_dep_launch();
#pragma unroll
    for (int i = 0; i < B::kPieces; ++i) {
        B::load(src, t, B::kRows * i < left ? n : 0, w[i]);
        src += B::kRows * a.lds;
    }
#pragma unroll
    for (int i = 0; i < B::kPieces; ++i)
#pragma unroll
        for (int j = 0; j < B::kPieceWords; ++j)
            m = B::kPer == 1 ? max(m, w[i][j] & 0x7FFFFFFFu) : __vmaxu2(m, w[i][j] & 0x7FFF7FFFu);
    if (B::kPer == 2) m = max(m << 16, m & 0xFFFF0000u);
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) part[warp] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, part[i]);
    const BlockScale s = block_scale(m, a.pow2);
    if (threadIdx.x == 0) a.scales[blockIdx.x] = s.scale;
#pragma unroll
    for (int i = 0; i < B::kPieces; ++i) {
        if (B::kRows * i >= left) break;
        B::store(w[i], t, n, s, dst);
        dst += B::kRows * a.ldq;
    }
}

// Vector accesses: rows of a multiple of 8 elements, all 16-byte aligned (codes: 8).
bool vec_ok(const void *p, int64_t ld, int size) {
    return !p || (reinterpret_cast<uintptr_t>(p) % (size == 1 ? 8 : 16) == 0 && ld % 8 == 0);
}

template <typename X, bool VEC>
cudaError_t quant_launch(const QuantArgs &a, int block_rows, cudaStream_t s) {
    constexpr int kSpan = kRowUnits * kUnit;
    const int64_t grid = block_rows == 1 ? (a.rows * ((a.cols + kSpan - 1) / kSpan) + 7) / 8
                                         : (a.rows + kFp8Block - 1) / kFp8Block * a.nb;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    count_launches(1);
    return block_rows == 1 ? cudaLaunchKernelEx(&cfg, fp8_quant_rows_kernel<X, VEC>, a)
                           : cudaLaunchKernelEx(&cfg, fp8_quant_tile_kernel<X, VEC>, a);
}

}  // namespace

cudaError_t launch_rms_norm(const moe_norm_desc &n, const void *x, const void *residual, const void *weight,
                            void *sum, uint16_t *y, uint8_t *codes, float *scales, cudaStream_t s) {
    NormArgs a;
    a.x = x; a.res = residual; a.w = weight; a.sum = sum; a.y = y; a.codes = codes; a.scales = scales;
    a.ldx = n.ldx; a.ldr = n.ldr; a.ldy = n.ldy; a.ldq = n.ldq;
    a.d = n.d; a.nb = ceil_div(n.d, kFp8Block);
    a.w_bf16 = n.w_type == MOE_T_BF16; a.pow2 = n.scale_mode == MOE_SCALE_POW2; a.eps = n.eps;
    const int xs = n.x_type == MOE_T_BF16 ? 2 : 4, rs = n.res_type == MOE_T_BF16 ? 2 : 4;
    const bool vec = n.d % 8 == 0 && vec_ok(x, n.ldx, xs) && vec_ok(residual, n.ldr, rs) && vec_ok(sum, n.ldr, rs) &&
                     vec_ok(weight, 0, a.w_bf16 ? 2 : 4) && vec_ok(y, n.ldy, 2) && vec_ok(codes, n.ldq, 1);
    if (n.x_type == MOE_T_BF16)
        return vec ? norm_res<uint16_t, true>(a, n.T, n.res_type, s) : norm_res<uint16_t, false>(a, n.T, n.res_type, s);
    return vec ? norm_res<float, true>(a, n.T, n.res_type, s) : norm_res<float, false>(a, n.T, n.res_type, s);
}

cudaError_t launch_fp8_quantize(const moe_fp8_quant_desc &q, const void *v, uint8_t *codes, float *scales,
                                cudaStream_t s) {
    QuantArgs a;
    a.v = v; a.codes = codes; a.scales = scales; a.lds = q.ldv; a.ldq = q.ldq; a.rows = q.rows; a.cols = q.cols;
    a.nb = ceil_div(q.cols, kFp8Block); a.pow2 = q.scale_mode == MOE_SCALE_POW2;
    const bool bf = q.v_type == MOE_T_BF16;
    const bool vec = q.cols % 8 == 0 && vec_ok(v, q.ldv, bf ? 2 : 4) && vec_ok(codes, q.ldq, 1);
    if (bf) return vec ? quant_launch<uint16_t, true>(a, q.block_rows, s) : quant_launch<uint16_t, false>(a, q.block_rows, s);
    return vec ? quant_launch<float, true>(a, q.block_rows, s) : quant_launch<float, false>(a, q.block_rows, s);
}

}  // namespace moe
