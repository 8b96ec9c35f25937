// Matrix products of FP8 matrices with a scale per block of 128, and the FP8
// shared expert built on them.
//
//   y[t][n] = sum_b sa[t][b] sw[n / 128][b] sum_{k in block b} a[t][k] w[n][k]
//
// The inner sums are tensor-core products of E4M3 codes (tcgen05.mma,
// kind::f8f6f4, fp32 accumulator in tensor memory); the scales change with
// every 128 of K, so each block's sum leaves tensor memory and is multiplied
// and added in fp32 registers ("promoted"): one fma per 128 multiply-adds.
//
// skinny_kernel (few tokens): the weights stream once, so it is bound by HBM
// and, for the smallest calls, by latency. A = 128 weight rows on the MMA's M
// side, B = BT tokens on its N side (BT = 16 .. 64), so a single token costs
// a 16-column MMA. The grid splits K over a cluster of up to 4 CTAs when there
// are too few tiles for the SMs; the partial sums meet in the cluster's shared
// memory and are added in rank order (deterministic, no scratch, no second
// kernel). Warps: TMA, MMA and four or eight promoting ones (thread = weight
// row = TMEM lane).
//
// wide_kernel (many tokens): tokens on the M side, a pair of SMs per 256 x 256
// tile; bound by the tensor cores' rate and the promotion beside them.
//
// Gate/up (GU): two weight tiles (W1, W3) per stage and two accumulators; the
// 128 rows of a tile are one scale block of h, so silu(g) u is quantised in
// the epilogue and h never exists in wider form.
#include <string.h>

#include <atomic>

#include "common.cuh"
#include "fp8.cuh"
#include "fp8.h"
#include "tc_fp8.cuh"

namespace moe {
namespace {

constexpr int kTile = 128;  // weight rows per tile, and the K block

// The scales are read by ordinary loads, after griddepcontrol.wait: a kernel here
// starts while the one before it, which may be writing them, still runs, so they
// are not read-only for as long as it lives (what a non-coherent load asks for).
struct GemmArgs {
    CUtensorMap a;           // activations E4M3 [T][K]
    CUtensorMap w[2];        // weights E4M3 [N][K] (GU: W1, W3)
    const float *as;         // [T][nkb]
    const float *ws[2];      // [ceil(N / 128)][nkb]
    void *y;                 // plain: [T][ldy]
    uint8_t *h;              // GU: codes [T][ldh]
    float *hs;               // GU: scales [T][ceil(N / 128)]
    int64_t ldy, ldh;
    int T, N, nkb;
    int y_bf16, accumulate, pow2;
    int w_early;             // the weights may be read before the preceding kernel ends
    int *err;
    uint64_t wait_ns;        // limit of the bounded waits
    int extra, extra_got;    // arrivals and bytes waited for in vain (tests of the limit; otherwise 0)
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// An arrival that orders no memory.
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
// The address in CTA `rank` of the cluster that corresponds to this CTA's
// shared address `addr`.
__device__ __forceinline__ uint32_t map_cluster(uint32_t addr, uint32_t rank) {
    uint32_t ra;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(addr), "r"(rank));
    return ra;
}
// A 16-byte store into a CTA of the cluster that completes its bytes on the mbarrier `bar` beside them.
__device__ __forceinline__ void st_async_v4(uint32_t addr, float x, float y, float z, float w, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                     addr),
                 "f"(x), "f"(y), "f"(z), "f"(w), "r"(bar)
                 : "memory");
}
// Bounded wait for what other CTAs of the cluster store.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t *bar, uint32_t parity, uint64_t limit_ns) {
    uint64_t t0 = 0;
    for (int n = 0;; ++n) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((n & 255) == 255) {
            const uint64_t now = globaltimer_ns();
            if (!t0) t0 = now;
            else if (now - t0 > limit_ns) return false;
        }
    }
}
__device__ __forceinline__ void bar_arrive(int id, int threads) {
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_named(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// silu(g) * u, 0 for the rows a tile has beyond the matrix.
__device__ __forceinline__ float swiglu(float g, float u, bool in) { return in ? silu_f32(g) * u : 0.f; }

__device__ __forceinline__ void store_y(const GemmArgs &a, int t, int n, float v) {
    const int64_t o = (int64_t)t * a.ldy + n;
    if (a.y_bf16) {
        static_cast<uint16_t *>(a.y)[o] = (uint16_t)f32x2_to_bf16x2_rn(v, 0.f);
    } else {
        float *p = static_cast<float *>(a.y) + o;
        *p = a.accumulate ? *p + v : v;
    }
}

// ------------------------------------------------------------------ skinny

constexpr int kMaxRanks = 4;  // of a cluster along K

template <int BT, bool GU>
struct SkCfg {
    static constexpr int kMats = GU ? 2 : 1;
    static constexpr int kStage = kMats * kTile * 128 + BT * 128;
    static constexpr int kPromo = BT >= 64 ? 8 : 4;   // promoting warps
    static constexpr int kThreads = 64 + 32 * kPromo;
    static constexpr int kCT = BT * 4 / kPromo;       // tokens (columns) per promoting thread
    static constexpr int kRed = kMats * BT * kTile * 4;  // partial sums sent to this CTA
    static constexpr int kChunk = 2048 / (kMats * BT) < 32 ? 2048 / (kMats * BT) : 32;  // K blocks of scales held
    // two CTAs per SM for the narrow plain tiles (about 110 KB each), one otherwise
    static constexpr int kBudget = (BT <= 32 && !GU ? 104 * 1024 : 212 * 1024) - kRed;
    static constexpr int kStages = kBudget / kStage < 8 ? kBudget / kStage : 8;
    static constexpr int kSlots = kStages < 4 ? kStages : 4;  // accumulators in flight
    static constexpr int kUsed = kSlots * kMats * BT;
    static constexpr int kCols = kUsed <= 64 ? 64 : kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
    static_assert(kUsed <= 512 && kStages >= 3, "tensor or shared memory");
};

template <int BT, bool GU>
struct SkSmem {
    using C = SkCfg<BT, GU>;
    uint8_t ring[C::kStages][C::kStage];    // per stage: weight tile(s), then token rows
    float red[C::kRed / 4];                 // partial sums sent here: [rank][matrix][own tokens / 4][weight row][4]
    float sc[C::kChunk][C::kMats][BT];      // sa * sw of a chunk of K blocks
    uint32_t part[4][BT];                   // GU: per-warp largest |h| of each own token
    uint64_t full[C::kStages], done[C::kStages], acc_empty[C::kSlots], got;
    uint32_t tmem_base;
    volatile int abort;
};

// The end of a skinny tile, four own tokens per step: sums the ranks' partial sums
// in rank order and writes y, or h in FP8. Threads in row order: rpid & 127.
template <int BT, bool GU>
__device__ __forceinline__ void skinny_finish(const GemmArgs &a, SkSmem<BT, GU> &s, int S, int per, int own, int t_own,
                                              int n0, int rpid) {
    using C = SkCfg<BT, GU>;
    constexpr int kGroups = C::kPromo / 4;
    const int r = rpid & 127, grp = rpid >> 7, lane = rpid & 31, n = n0 + r;
    const bool in = n < a.N;
    auto at = [&](int p, int m, int j4) {
        return reinterpret_cast<float4 *>(&s.red[(((p * C::kMats + m) * (per / 4) + j4) * kTile + r) * 4]);
    };
    auto sum = [&](int m, int j4) {
        float4 o = *at(0, m, j4);
#pragma unroll
        for (int p = 1; p < kMaxRanks; ++p)
            if (p < S) {
                const float4 f = *at(p, m, j4);
                o.x += f.x; o.y += f.y; o.z += f.z; o.w += f.w;
            }
        return o;
    };
    const int steps = (own + 3) / 4;
    if constexpr (GU) {
        for (int j4 = grp; j4 < steps; j4 += kGroups) {
            const float4 g = sum(0, j4), u = sum(1, j4);
            const float h[4] = {swiglu(g.x, u.x, in), swiglu(g.y, u.y, in), swiglu(g.z, u.z, in), swiglu(g.w, u.w, in)};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t m = __reduce_max_sync(0xffffffffu, abs_bits(h[e]));
                if (lane == 0) s.part[(rpid >> 5) & 3][j4 * 4 + e] = m;
            }
            // h replaces rank 0's partial sums, which only this thread reads
            *at(0, 0, j4) = make_float4(h[0], h[1], h[2], h[3]);
        }
        bar_named(1, 32 * C::kPromo);
        // a token's scale is one thread's work: two quotients, which every thread computing them for itself
        // made most of this function's time (1600 cycles per four tokens)
        if (rpid < own) {
            const uint32_t m = max(max(s.part[0][rpid], s.part[1][rpid]), max(s.part[2][rpid], s.part[3][rpid]));
            const BlockScale b = block_scale(m, a.pow2);
            s.part[0][rpid] = __float_as_uint(b.hi);
            s.part[1][rpid] = __float_as_uint(b.lo);
            s.part[2][rpid] = __float_as_uint(b.pre);
            a.hs[(int64_t)(t_own + rpid) * gridDim.x + blockIdx.x] = b.scale;
        }
        bar_named(1, 32 * C::kPromo);
        if (in)
#pragma unroll 2
            for (int j4 = grp; j4 < steps; j4 += kGroups) {
                float4 h = *at(0, 0, j4);
                const float4 hi = *reinterpret_cast<const float4 *>(&s.part[0][j4 * 4]);
                const float4 lo = *reinterpret_cast<const float4 *>(&s.part[1][j4 * 4]);
                const float4 pre = *reinterpret_cast<const float4 *>(&s.part[2][j4 * 4]);
                h.x *= pre.x; h.y *= pre.y; h.z *= pre.z; h.w *= pre.w;
                const uint32_t c = f32x4_to_e4m3x4(fmaf(h.x, hi.x, h.x * lo.x), fmaf(h.y, hi.y, h.y * lo.y),
                                                   fmaf(h.z, hi.z, h.z * lo.z), fmaf(h.w, hi.w, h.w * lo.w));
                uint8_t *p = a.h + (int64_t)(t_own + j4 * 4) * a.ldh + n;
#pragma unroll
                for (int e = 0; e < 4; ++e, p += a.ldh)
                    if (j4 * 4 + e < own) *p = (uint8_t)(c >> (8 * e));
            }
    } else if (in) {
        for (int j4 = grp; j4 < steps; j4 += kGroups) {
            const float4 v = sum(0, j4);
            const int t = t_own + j4 * 4, left = own - j4 * 4;
            store_y(a, t, n, v.x);
            if (left > 1) store_y(a, t + 1, n, v.y);
            if (left > 2) store_y(a, t + 2, n, v.z);
            if (left > 3) store_y(a, t + 3, n, v.w);
        }
    }
}

// One CTA per SM as the bound on registers: without it the compiler stops at 56 to
// 168 of them, and everything but the wide calls took 3 to 8% longer (two CTAs of
// the narrow plain tiles fit an SM all the same).
template <int BT, bool GU>
__global__ void __launch_bounds__(SkCfg<BT, GU>::kThreads, 1) skinny_kernel(const __grid_constant__ GemmArgs a) {
    using C = SkCfg<BT, GU>;
    extern __shared__ uint8_t smem_raw[];
    SkSmem<BT, GU> &s =
        *reinterpret_cast<SkSmem<BT, GU> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n0 = blockIdx.x * kTile, t0 = blockIdx.y * BT;
    const int S = gridDim.z, z = blockIdx.z;  // cluster of S CTAs along K, and this CTA's rank
    const int ncols = min(BT, a.T - t0);
    const int per = BT / S, own = min(per, max(0, ncols - z * per));  // tokens this rank finishes, of which exist
    const int kb0 = (int)((int64_t)a.nkb * z / S), kbn = (int)((int64_t)a.nkb * (z + 1) / S) - kb0;

    auto load_w = [&](int i) {
        const int st = i % C::kStages;
        mbar_arrive_expect_tx(&s.full[st], C::kStage);
#pragma unroll
        for (int m = 0; m < C::kMats; ++m)
            tma_load_2d(s.ring[st] + m * kTile * 128, &a.w[m], (kb0 + i) * 128, n0, &s.full[st]);
    };
    auto load_a = [&](int i) {
        const int st = i % C::kStages;
        tma_load_2d(s.ring[st] + C::kMats * kTile * 128, &a.a, (kb0 + i) * 128, t0, &s.full[st]);
    };
    const int ahead = min(kbn, C::kStages);
    const int pid = threadIdx.x - 64;  // promoting thread
    // Scales of up to kChunk K blocks from block i0 on (tokens beyond T: 0). A thread takes one K block
    // (lg bits of its number) of every (threads >> lg)-th token.
    constexpr int kScales = BT * C::kChunk / (32 * C::kPromo);  // tokens per thread, at most
    float sa[kScales], sw[C::kMats];
    const float *as = a.as + (int64_t)t0 * a.nkb + kb0;
    auto chunk_bits = [](int cnt) { return cnt > 1 ? 32 - __clz(cnt - 1) : 0; };
    auto load_scales = [&](int i0) {
        const int cnt = min(C::kChunk, kbn - i0), lg = chunk_bits(cnt), kb = pid & ((1 << lg) - 1);
        if (kb >= cnt) return;
#pragma unroll
        for (int m = 0; m < C::kMats; ++m) sw[m] = a.ws[m][(int64_t)blockIdx.x * a.nkb + kb0 + i0 + kb];
#pragma unroll
        for (int j = 0; j < kScales; ++j) {
            const int c = (pid >> lg) + j * (32 * C::kPromo >> lg);
            sa[j] = c < ncols ? as[(int64_t)c * a.nkb + i0 + kb] : 0.f;
        }
    };
    auto store_scales = [&](int i0) {
        const int cnt = min(C::kChunk, kbn - i0), lg = chunk_bits(cnt), kb = pid & ((1 << lg) - 1);
        if (kb >= cnt) return;
#pragma unroll
        for (int j = 0; j < kScales; ++j) {
            const int c = (pid >> lg) + j * (32 * C::kPromo >> lg);
            if (c < BT)
#pragma unroll
                for (int m = 0; m < C::kMats; ++m) s.sc[kb][m][c] = sa[j] * sw[m];
        }
    };
    // Warp 0 sets the barriers up, arrives and starts to load; the others wait for it and for tensor
    // memory, which the first loads hide (1500 cycles when all waited for all).
    if (warp == 0) {
        if (elect_one()) {
            prefetch_tensormap(&a.w[0]);
            if (GU) prefetch_tensormap(&a.w[1]);
            prefetch_tensormap(&a.a);
            for (int i = 0; i < C::kStages; ++i) {
                mbar_init(&s.full[i], 1);
                mbar_init(&s.done[i], 1);
            }
            for (int i = 0; i < C::kSlots; ++i) mbar_init(&s.acc_empty[i], C::kPromo + a.extra);
            mbar_init(&s.got, 1);
            s.abort = 0;
            fence_mbar_init();
            if (S > 1) mbar_arrive_expect_tx(&s.got, (S - 1) * C::kMats * ((own + 3) / 4) * (kTile * 16) + a.extra_got);
        }
        __syncwarp();
        bar_arrive(2, C::kThreads);
    } else {
        if (warp == 1) {
            tmem_alloc(&s.tmem_base, C::kCols);
            tmem_relinquish();
        }
        tc_fence_before();
        bar_named(2, C::kThreads);
        tc_fence_after();
    }
    if (S > 1) {
        __syncwarp();
        cluster_arrive();
    }
    const uint32_t tmem = warp ? s.tmem_base : 0;
    auto fail = [&]() {
        set_device_error(a.err, MOE_DEVERR_TIMEOUT);
        s.abort = 1;
    };
    const int q = warp & 3, r = 32 * q + lane;        // its tensor-memory lane quarter and weight row
    const int c0 = pid >= 0 ? (pid >> 7) * C::kCT : 0;  // its first token
    float2 acc[C::kMats][C::kCT / 2];

    if (warp == 0) {
        if (elect_one()) {
            if (a.w_early) {
                for (int i = 0; i < ahead; ++i) load_w(i);
                grid_dep_wait();
                for (int i = 0; i < ahead; ++i) load_a(i);
            } else {
                grid_dep_wait();
                for (int i = 0; i < ahead; ++i) {
                    load_w(i);
                    load_a(i);
                }
            }
            int last = ahead;
            for (int i = ahead; i < kbn; ++i) {
                if (!mbar_poll(&s.done[i % C::kStages], ((i / C::kStages) & 1) ^ 1, &s.abort, a.wait_ns)) { fail(); break; }
                load_w(i);
                load_a(i);
                last = i + 1;
            }
            for (int i = max(0, last - C::kStages); i < last; ++i)  // copies land before the CTA exits
                mbar_wait(&s.full[i % C::kStages], (i / C::kStages) & 1);
        }
    } else if (warp == 1) {
        if (elect_one()) {
            constexpr uint32_t idesc = idesc_e4m3(kTile, BT);
            grid_dep_wait();  // the bounded waits count from here, not from an early launch
            int i = 0;
            for (; i < kbn; ++i) {
                const int st = i % C::kStages, slot = i % C::kSlots;
                if (!mbar_poll(&s.acc_empty[slot], ((i / C::kSlots) & 1) ^ 1, &s.abort, a.wait_ns) ||
                    !mbar_poll(&s.full[st], (i / C::kStages) & 1, &s.abort, a.wait_ns)) { fail(); break; }
                tc_fence_after();
                const uint64_t db = sdesc_sw128(s.ring[st] + C::kMats * kTile * 128);
#pragma unroll
                for (int m = 0; m < C::kMats; ++m) {
                    const uint64_t da = sdesc_sw128(s.ring[st] + m * kTile * 128);
                    const uint32_t d = tmem + (uint32_t)((slot * C::kMats + m) * BT);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) tc_mma_f8(d, da + 2 * ks, db + 2 * ks, idesc, ks != 0);
                }
                tc_commit(&s.done[st]);
            }
            // every MMA has finished before the CTA's shared and tensor memory go
            if (i > 0) mbar_wait(&s.done[(i - 1) % C::kStages], ((i - 1) / C::kStages) & 1);
        }
    } else {
        // promoting warps: thread = weight row r of the tile, columns = tokens c0 .. c0 + kCT - 1
        const uint32_t base = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)c0;
        grid_dep_wait();
        if (threadIdx.x == 64) grid_dep_launch();
#pragma unroll
        for (int m = 0; m < C::kMats; ++m)
#pragma unroll
            for (int c = 0; c < C::kCT / 2; ++c) acc[m][c] = make_float2(0.f, 0.f);
        bool live = true;  // until a wait of this warp gives up: then it only keeps the named barriers' counts equal
        for (int i0 = 0; i0 < kbn; i0 += C::kChunk) {
            const int cnt = min(C::kChunk, kbn - i0);
            load_scales(i0);
            if (i0) bar_named(1, 32 * C::kPromo);  // the last chunk's have been read
            store_scales(i0);
            bar_named(1, 32 * C::kPromo);
            for (int k = 0; live && k < cnt; ++k) {
                const int i = i0 + k, st = i % C::kStages, slot = i % C::kSlots;
                live = __all_sync(0xffffffffu, mbar_poll(&s.done[st], (i / C::kStages) & 1, &s.abort, a.wait_ns));
                if (!live) {
                    if (lane == 0) fail();
                    break;
                }
                tc_fence_after();
                constexpr int kV = C::kCT < 32 ? C::kCT : 32, kLoads = C::kCT / kV;
                uint32_t v[C::kMats][kLoads][kV];
#pragma unroll
                for (int m = 0; m < C::kMats; ++m)
#pragma unroll
                    for (int l = 0; l < kLoads; ++l) {
                        const uint32_t at = base + (uint32_t)((slot * C::kMats + m) * BT + l * kV);
                        if constexpr (kV == 16) tmem_ld16(at, v[m][l]);
                        else tmem_ld32(at, v[m][l]);
                    }
#pragma unroll
                for (int m = 0; m < C::kMats; ++m)
#pragma unroll
                    for (int l = 0; l < kLoads; ++l) {
                        if constexpr (kV == 16) tmem_wait_ld16(v[m][l]);
                        else tmem_wait_ld32(v[m][l]);
                    }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.acc_empty[slot]);
#pragma unroll
                for (int m = 0; m < C::kMats; ++m)
#pragma unroll
                    for (int l = 0; l < kLoads; ++l)
#pragma unroll
                        for (int c = 0; c < kV; c += 4) {
                            const float4 f = *reinterpret_cast<const float4 *>(&s.sc[k][m][c0 + l * kV + c]);
                            float2 *d = &acc[m][(l * kV + c) / 2];
                            const uint32_t *x = &v[m][l][c];
                            d[0] = __ffma2_rn(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])),
                                              make_float2(f.x, f.y), d[0]);
                            d[1] = __ffma2_rn(make_float2(__uint_as_float(x[2]), __uint_as_float(x[3])),
                                              make_float2(f.z, f.w), d[1]);
                        }
            }
        }
    }
    // tensor memory goes back before any wait on another CTA
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kCols);
    }
    // Rank z of the cluster finishes the tokens z per .. (z + 1) per - 1. Every rank
    // sends its partial sums there in 16-byte asynchronous stores into the owner's
    // shared memory, counted on the owner's barrier, and the owner adds them in rank
    // order. Plain stores and a cluster barrier (1100 to 1700 cycles) took 1.1 us more
    // in the shared expert of 8 to 32 tokens; bulk copies from shared memory as much.
    if (S > 1) {
        __syncwarp();
        cluster_wait();  // the arrival at the start: every CTA of the cluster runs
    }
    // From here on every thread of every rank arrives at the cluster's second barrier, when it has sent what it
    // sends, and waits there before it leaves, whether a wait gave up or not: what a late rank sends never meets
    // a CTA that is gone. (All threads: warps that had exited were not taken as arrived.)
    auto arrive = [&]() {
        __syncwarp();
        if (S > 1) cluster_arrive_relaxed();
    };
    auto leave = [&]() {
        __syncwarp();
        if (S > 1) cluster_wait();
    };
    if (warp < 2) {
        arrive();
        leave();
        return;
    }
    const int lg = 31 - __clz(per);
    const uint32_t red = smem_u32(s.red), got = smem_u32(&s.got);
#pragma unroll
    for (int c = 0; c < C::kCT; c += 4) {
        const int col = c0 + c, p = col >> lg;
        if (col >= ncols) break;
#pragma unroll
        for (int m = 0; m < C::kMats; ++m) {
            const float2 x = acc[m][c / 2], y = acc[m][c / 2 + 1];
            const uint32_t off = (((z * C::kMats + m) * (per / 4) + ((col & (per - 1)) >> 2)) * kTile + r) * 16;
            if (p == z) reinterpret_cast<float4 *>(s.red)[off / 16] = make_float4(x.x, x.y, y.x, y.y);
            else st_async_v4(map_cluster(red + off, p), x.x, x.y, y.x, y.y, map_cluster(got, p));
        }
    }
    arrive();
    const bool landed = S == 1 || mbar_wait_cluster(&s.got, 0, 2 * a.wait_ns);
    if (!__all_sync(0xffffffffu, landed) && lane == 0) fail();
    bar_named(1, 32 * C::kPromo);  // this rank's own are there, and all of its threads see the same abort flag
    const bool ok = !s.abort;
    const int rpid = (pid & ~127) | r;  // threads in row order
    if (ok) skinny_finish<BT, GU>(a, s, S, per, own, t0 + z * per, n0, rpid);
    leave();
    if (!ok && S > 1) mbar_wait_cluster(&s.got, 0, 10000000);  // what the others sent is on its way: 10 ms for it
}

// SMs of device dev (looked up once per device).
int fp8_num_sms(int dev) {
    static std::atomic<int> sms[64];
    int n = sms[dev].load(std::memory_order_relaxed);
    if (!n) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
        sms[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

// Raises the kernel's shared-memory limit, once per device.
template <typename K>
cudaError_t allow_smem(std::atomic<bool> (&done)[64], int dev, K kernel, int bytes) {
    if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
    return e;
}

// Operand maps: boxes of `a_rows` token rows and of 128 weight rows.
template <bool GU>
bool make_maps(GemmArgs &a, const void *act, int64_t lda, int a_rows, const void *const *w, int64_t ldw, int K) {
    return make_rows_map_u8(&a.a, act, a.T, K, lda, a_rows) && make_rows_map_u8(&a.w[0], w[0], a.N, K, ldw, kTile) &&
           (!GU || make_rows_map_u8(&a.w[1], w[1], a.N, K, ldw, kTile));
}

// Launch of a kernel whose grid is (weight tiles, token tiles, ranks along K).
template <typename K>
cudaError_t launch_split(K kernel, const GemmArgs &a, dim3 grid, int threads, int smem, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = 1;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = grid.z;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Ranks along K: doubled while the SMs hold all clusters at once and a rank keeps a
// K block. Four at most: measured at 4, 5, 6 and 7 ranks, us: 4096 x 4096, one
// token, 4.4, 5.4, 5.3, 5.1; shared expert, 9.6, 10.0, 9.9, 13.1 (gate/up 16
// tiles); 1003 x 1111, 3.2, 3.4, 3.2, 3.3; and 15 clusters of 8 fit where 33 of 4 do.
int split_k(int64_t tiles, int nkb, const int *held) {
    int S = 1, i = 1;
    while (S < kMaxRanks && tiles <= held[i] && nkb >= 2 * S) S *= 2, ++i;
    return S;
}

// Clusters of 1, 2 and 4 CTAs of a kernel that the device holds at one CTA per SM
// (the occupancy query counts no more for kernels with tensor memory).
template <typename K>
cudaError_t clusters_held(std::atomic<int> (&known)[64][3], int dev, K kernel, int threads, int smem, int (&held)[3]) {
    for (int i = 0; i < 3; ++i) {
        int n = known[dev][i].load(std::memory_order_relaxed);
        if (!n) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(1, 1, 1u << i);
            cfg.blockDim = dim3(threads);
            cfg.dynamicSmemBytes = smem;
            cudaLaunchAttribute at[1];
            at[0].id = cudaLaunchAttributeClusterDimension;
            at[0].val.clusterDim.x = 1;
            at[0].val.clusterDim.y = 1;
            at[0].val.clusterDim.z = 1u << i;
            cfg.attrs = at;
            cfg.numAttrs = 1;
            const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
            if (e != cudaSuccess) return e;
            known[dev][i].store(n, std::memory_order_relaxed);
        }
        held[i] = n;
    }
    return cudaSuccess;
}

template <int BT, bool GU>
cudaError_t skinny_launch(GemmArgs &a, const void *act, int64_t lda, const void *const *w, int64_t ldw, int K, int dev,
                          cudaStream_t s) {
    using C = SkCfg<BT, GU>;
    static std::atomic<bool> done[64];
    static std::atomic<int> known[64][3];
    constexpr int smem = (int)sizeof(SkSmem<BT, GU>) + 1024;
    cudaError_t e = allow_smem(done, dev, skinny_kernel<BT, GU>, smem);
    if (e != cudaSuccess) return e;
    int held[3];
    if ((e = clusters_held(known, dev, skinny_kernel<BT, GU>, C::kThreads, smem, held)) != cudaSuccess) return e;
    const int nt = ceil_div(a.N, kTile), tt = ceil_div(a.T, BT);
    if (tt > 65535 || !make_maps<GU>(a, act, lda, BT, w, ldw, K)) return cudaErrorInvalidValue;
    const int S = split_k((int64_t)nt * tt, a.nkb, held);
    return launch_split(skinny_kernel<BT, GU>, a, dim3(nt, tt, S), C::kThreads, smem, s);
}

// -------------------------------------------------------------------- wide

// Many tokens: a pair of CTAs (two SMs) computes 256 tokens x two weight tiles of
// 128 rows (plain: neighbouring tiles; GU: the same tile of W1 and W3) with
// cta_group::2 MMAs (M = 256). Each CTA loads its own 128 tokens and 64 rows of
// each weight tile, 32 KB per K block for the 513 cycles its MMAs take; a single
// CTA's 128 x 256 tile needs 48 KB, and an SM was measured to take in 64 bytes per
// cycle. Persistent, one pair per two SMs over the tiles.
//
// The accumulators of one K block are two of four 128-column slots of tensor
// memory, one per weight tile, each handed back as soon as it has been read, so a
// tile's MMAs can start while the other's is still being read (an N = 128 pair MMA
// runs at the full rate, 257 cycles per K block, TMA and tensor-memory reads
// running beside it).
//
// Eight promoting warps hold the CTA's 128 x 256 fp32 sums in registers (thread =
// token row = TMEM lane; warps 4 .. 7 take columns 0 .. 63 of each weight tile,
// warps 8 .. 11 columns 64 .. 127). Warps 2 and 3 bring the scales: for each row
// and K block the products with the two weight tiles' scales, written to shared
// memory ahead of time, one 8-byte read per thread and K block. Warp 0 loads,
// warp 1 of the even CTA issues.
//
// What bounds it, 4096 x 4096 x 4096 in bursts: loads and MMAs alone 41 us (the
// floor at twice the measured bf16 rate), with the hand-offs between MMAs and
// promotion 50 (an MMA's end is seen about 320 cycles late, and a slot is free
// again 270 to 440 cycles after that), with the promotion 57 (its fmas alone are
// 256 cycles of an SM per K block), with the output 66 to 69. Run back to back for
// seconds the clock falls (power) and it takes 83 us, 1.66 PFLOP/s.
constexpr int kWdThreads = 384;
// Registers: 384 threads are launched with 168 each (64512 in all); warps 0 .. 3
// give theirs up to the promoting warps: 128 x 40 + 256 x 232 = 64512.
constexpr int kWdStages = 6;
constexpr int kWdStage = 2 * kTile * 128;  // per CTA: token tile, weight tile

struct WdSmem {
    uint8_t ring[kWdStages][kWdStage];
    float2 sc[kWdStages][kTile];  // per K block and row: sa * the scales of the two weight tiles
    uint8_t out[8][32 * 64];      // rows on their way out, per promoting warp
    uint32_t part[2][kTile];      // GU: each half's largest |h| of a token
    // done: the K block's MMAs have finished and its scales are there (two warps). full and acc_empty
    // are used in the even CTA, for both CTAs, done in each.
    uint64_t full[kWdStages], done[kWdStages], acc_empty[4], half[4];
    uint32_t tmem_base;
    volatile int abort;
};
constexpr int kWdSmemBytes = (int)sizeof(WdSmem) + 1024;

// Output through shared memory: thread l of a warp holds 64 bytes of row l (four
// 16-byte units); they are written to a buffer of 32 x 64 bytes (unit u of row l
// at unit u ^ (l / 2 % 4): conflict-free both ways) and leave row by row, so a
// store instruction touches 8 rows of 64 bytes instead of 32 rows of 16. A
// tile's direct 16-byte stores took 4 us of an SM's load-store pipe, exposed
// between two tiles.
__device__ __forceinline__ void stage_rows(uint8_t *buf, int lane, const uint4 (&u)[4]) {
    __syncwarp();  // the previous rows have left
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4 *>(buf + lane * 64 + ((i ^ (lane >> 1 & 3)) << 4)) = u[i];
    __syncwarp();
}
__device__ __forceinline__ uint4 staged_unit(const uint8_t *buf, int row, int u) {
    return *reinterpret_cast<const uint4 *>(buf + row * 64 + ((u ^ (row >> 1 & 3)) << 4));
}

// The staged rows t0 .. t0 + 31 to columns n .. of y (16 fp32 or 32 bf16 each).
template <typename TYPE>
__device__ __forceinline__ void store_staged(const GemmArgs &a, const uint8_t *buf, int lane, int t0, int n, bool vec) {
    constexpr int kCols = 64 / (int)sizeof(TYPE);
    TYPE *y = static_cast<TYPE *>(a.y) + (int64_t)t0 * a.ldy + n;
    if (vec && n + kCols <= a.N) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 8 * i + (lane >> 2);
            if (t0 + row >= a.T) break;
            uint4 v = staged_unit(buf, row, lane & 3);
            uint4 *p = reinterpret_cast<uint4 *>(y + (int64_t)row * a.ldy) + (lane & 3);
            if (sizeof(TYPE) == 4 && a.accumulate) {
                const float4 f = *reinterpret_cast<const float4 *>(p);
                v.x = __float_as_uint(f.x + __uint_as_float(v.x));
                v.y = __float_as_uint(f.y + __uint_as_float(v.y));
                v.z = __float_as_uint(f.z + __uint_as_float(v.z));
                v.w = __float_as_uint(f.w + __uint_as_float(v.w));
            }
            *p = v;
        }
    } else {
        const int col = lane & (kCols - 1), rows = min(32, a.T - t0);
        if (n + col < a.N)
#pragma unroll 4
            for (int row = lane / kCols; row < rows; row += 32 / kCols) {
                const int byte = col * (int)sizeof(TYPE);
                const TYPE *q = reinterpret_cast<const TYPE *>(buf + row * 64 + (((byte >> 4) ^ (row >> 1 & 3)) << 4) +
                                                               (byte & 15));
                TYPE *p = y + (int64_t)row * a.ldy + col;
                if constexpr (sizeof(TYPE) == 4) *p = a.accumulate ? *p + *q : *q;
                else *p = *q;
            }
    }
}

// 64 outputs of each of the warp's rows from column n on; v: the thread's row.
__device__ __forceinline__ void store_rows64(const GemmArgs &a, uint8_t *buf, int lane, int t0, int n,
                                             const float2 (&v)[32], bool vec) {
    if (n >= a.N || t0 >= a.T) return;
    if (a.y_bf16) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint4 u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 *f = &v[16 * h + 4 * i];
                u[i] = make_uint4(f32x2_to_bf16x2_rn(f[0].x, f[0].y), f32x2_to_bf16x2_rn(f[1].x, f[1].y),
                                  f32x2_to_bf16x2_rn(f[2].x, f[2].y), f32x2_to_bf16x2_rn(f[3].x, f[3].y));
            }
            stage_rows(buf, lane, u);
            store_staged<uint16_t>(a, buf, lane, t0, n + 32 * h, vec);
        }
    } else {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            uint4 u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = v[8 * h + 2 * i], g = v[8 * h + 2 * i + 1];
                u[i] = make_uint4(__float_as_uint(f.x), __float_as_uint(f.y), __float_as_uint(g.x), __float_as_uint(g.y));
            }
            stage_rows(buf, lane, u);
            store_staged<float>(a, buf, lane, t0, n + 16 * h, vec);
        }
    }
}

// d[at .. at + 15] += v * c, in pairs.
__device__ __forceinline__ void add_scaled(float2 (&d)[32], int at, const uint32_t (&v)[32], float c) {
    const float2 cc = make_float2(c, c);
#pragma unroll
    for (int i = 0; i < 16; ++i)
        d[at + i] = __ffma2_rn(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), cc, d[at + i]);
}

// One K block of a warp's 32 rows and 64 + 64 columns (from tb and tb + 128):
// acc[b] += sc * the accumulator of weight tile b. Four loads of 32 columns, two
// per wait (a wait is for all of a warp's loads, 170 to 190 cycles), the next two
// started as the registers of the first come free; release(b) is called by one
// lane when tile b's columns have been read.
template <typename F>
__device__ __forceinline__ void promote_block(float2 (&acc)[2][32], uint32_t tb, const float2 sc, int lane, F release) {
    uint32_t v[2][32];
    tmem_ld32(tb, v[0]);
    tmem_ld32(tb + 32u, v[1]);
    tmem_wait_ld32(v[0]);
    tmem_wait_ld32(v[1]);
    tc_fence_before();
    __syncwarp();
    if (lane == 0) release(0);
    add_scaled(acc[0], 0, v[0], sc.x);
    tmem_ld32(tb + 128u, v[0]);
    add_scaled(acc[0], 16, v[1], sc.x);
    tmem_ld32(tb + 160u, v[1]);
    tmem_wait_ld32(v[0]);
    tmem_wait_ld32(v[1]);
    tc_fence_before();
    __syncwarp();
    if (lane == 0) release(1);
    add_scaled(acc[1], 0, v[0], sc.y);
    add_scaled(acc[1], 16, v[1], sc.y);
}

// The two scale warps (threads 64 .. 127) of one tile: for its rows t0 .. t0 + 127
// and K blocks kb0 .. kb0 + kbn - 1, the products with the scales of the two
// weight tiles at n0 into sc, and an arrival on done. `it` counts K blocks over
// tiles. False when a wait gave up.
template <int STAGES, bool GU>
__device__ __forceinline__ bool bring_scales(const GemmArgs &a, int t0, int n0, int kb0, int kbn, int &it,
                                             float2 (*sc)[kTile], uint64_t *done, const volatile int *abort) {
    const int r = threadIdx.x - 64, lane = threadIdx.x & 31;  // rows r and r + 64
    // four K blocks per load where they are aligned
    const bool vec = (reinterpret_cast<uintptr_t>(a.as) & 15) == 0 && a.nkb % 4 == 0 && kb0 % 4 == 0 && kbn % 4 == 0;
    const float *as[2];
    for (int i = 0; i < 2; ++i) as[i] = a.as + (int64_t)min(t0 + r + 64 * i, a.T - 1) * a.nkb + kb0;
    const float *w0 = a.ws[0] + (int64_t)(n0 / kTile) * a.nkb + kb0;
    // GU: the same tile of W3; plain: the next row tile (beyond the matrix: this one, never stored)
    const float *w1 = GU ? a.ws[1] + (int64_t)(n0 / kTile) * a.nkb + kb0 : n0 + kTile < a.N ? w0 + a.nkb : w0;
    bool ok = true;
    for (int k0 = 0; k0 < kbn && ok; k0 += 4) {
        float v[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (vec) {
                const float4 f = *reinterpret_cast<const float4 *>(as[i] + k0);
                v[i][0] = f.x; v[i][1] = f.y; v[i][2] = f.z; v[i][3] = f.w;
            } else {
#pragma unroll
                for (int u = 0; u < 4; ++u) v[i][u] = k0 + u < kbn ? as[i][k0 + u] : 0.f;
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (k0 + u >= kbn || !ok) break;
            const int st = it % STAGES, past = it - STAGES + 2;
            const float s0 = w0[k0 + u], s1 = w1[k0 + u];
            // The MMAs of K block `past` were issued after the promotion of past - 2 = it - STAGES, the
            // last reader of this slot, had read its scales.
            if (past >= 0) {
                ok = mbar_poll(&done[past % STAGES], (past / STAGES) & 1, abort, a.wait_ns);
                ok = __all_sync(0xffffffffu, ok);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) sc[st][r + 64 * i] = make_float2(v[i][u] * s0, v[i][u] * s1);
            __syncwarp();
            if (lane == 0) mbar_arrive(&done[st]);
            ++it;
        }
    }
    return ok;
}

template <bool GU>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWdThreads, 1)
    wide_kernel(const __grid_constant__ GemmArgs a) {
    extern __shared__ uint8_t smem_raw[];
    WdSmem &s = *reinterpret_cast<WdSmem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x & 1;            // in the pair
    constexpr int kN = GU ? kTile : 2 * kTile;  // output columns per tile
    const int mt = (a.T + 2 * kTile - 1) / (2 * kTile), nt = (a.N + kN - 1) / kN, tiles = mt * nt;
    const int first = blockIdx.x >> 1, step = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kWdStages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.done[i], 3);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&s.acc_empty[i], 16 + a.extra);
            mbar_init(&s.half[i], 2);  // the promoting warps of one lane quarter
        }
        s.abort = 0;
        fence_mbar_init();
        prefetch_tensormap(&a.a);
        prefetch_tensormap(&a.w[0]);
        if (GU) prefetch_tensormap(&a.w[1]);
    }
    if (warp == 1) tmem_alloc_pair(&s.tmem_base, 512);
    tc_fence_before();
    __syncthreads();
    cluster_arrive();  // the pair's barriers are set up before either CTA signals the other's
    cluster_wait();
    tc_fence_after();
    const uint32_t tmem = s.tmem_base;
    // A wait gave up. Copies and MMAs in flight end well within this time, and no CTA of the pair leaves,
    // nor is anything of it freed, before.
    auto fail = [&]() {
        set_device_error(a.err, MOE_DEVERR_TIMEOUT);
        s.abort = 1;
        for (const uint64_t t0 = globaltimer_ns(); globaltimer_ns() - t0 < 10000000ull;) __nanosleep(1000);
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 0) {
            if (elect_one()) {
                grid_dep_wait();
                int it = 0;
                bool ok = true;
                for (int tile = first; tile < tiles && ok; tile += step) {
                    const int m0 = (tile % mt * 2 + rank) * kTile, n0 = tile / mt * kN + rank * (kTile / 2);
                    for (int kb = 0; kb < a.nkb; ++kb, ++it) {
                        const int st = it % kWdStages;
                        ok = mbar_poll(&s.done[st], ((it / kWdStages) & 1) ^ 1, &s.abort, a.wait_ns);
                        if (!ok) break;
                        if (rank == 0) mbar_arrive_expect_tx(&s.full[st], 2 * kWdStage);
                        const uint32_t full = map_cluster(smem_u32(&s.full[st]), 0);
                        tma_load_2d_pair(s.ring[st], &a.a, kb * 128, m0, full);
                        tma_load_2d_pair(s.ring[st] + kTile * 128, &a.w[0], kb * 128, n0, full);
                        tma_load_2d_pair(s.ring[st] + kTile * 192, &a.w[GU], kb * 128, GU ? n0 : n0 + kTile, full);
                    }
                }
                if (!ok) fail();
                // otherwise the last K block's arrival on done, which every promoting warp waits for,
                // comes after all of the copies
            }
        } else if (warp == 1 && rank == 0) {
            if (elect_one()) {
                constexpr uint32_t idesc = idesc_e4m3(2 * kTile, kTile);
                grid_dep_wait();  // the bounded waits count from here, not from an early launch
                int it = 0;
                bool ok = true;
                for (int tile = first; tile < tiles && ok; tile += step)
                    for (int kb = 0; kb < a.nkb && ok; ++kb, ++it) {
                        const int st = it % kWdStages;
                        ok = mbar_poll(&s.full[st], (it / kWdStages) & 1, &s.abort, a.wait_ns);
                        const uint64_t da = sdesc_sw128(s.ring[st]);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int slot = 2 * (it & 1) + h;
                            ok = ok && mbar_poll(&s.acc_empty[slot], ((it >> 1) & 1) ^ 1, &s.abort, a.wait_ns);
                            if (!ok) break;
                            tc_fence_after();
                            const uint64_t db = sdesc_sw128(s.ring[st] + kTile * (128 + 64 * h));
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                tc_mma_f8_pair(tmem + 128u * slot, da + 2 * ks, db + 2 * ks, idesc, ks != 0);
                            if (h) tc_commit_pair(&s.done[st]);
                        }
                    }
                if (!ok) {
                    fail();
                } else if (it > 0) {
                    // every MMA has finished before the pair's shared and tensor memory go
                    mbar_wait(&s.done[(it - 1) % kWdStages], ((it - 1) / kWdStages) & 1);
                }
            }
        } else if (warp >= 2) {
            grid_dep_wait();
            int it = 0;
            bool ok = true;
            for (int tile = first; tile < tiles && ok; tile += step)
                ok = bring_scales<kWdStages, GU>(a, (tile % mt * 2 + rank) * kTile, tile / mt * kN, 0, a.nkb, it, s.sc,
                                                 s.done, &s.abort);
            if (!ok && lane == 0) fail();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        const int q = warp & 3, j = (warp - 4) >> 2, r = 32 * q + lane;
        const uint32_t base = tmem + ((uint32_t)(32 * q) << 16) + 64u * j;
        const bool vec = (reinterpret_cast<uintptr_t>(a.y) & 15) == 0 && a.ldy % (a.y_bf16 ? 8 : 4) == 0;
        grid_dep_wait();
        if (threadIdx.x == 128) grid_dep_launch();
        const uint32_t acc_empty = map_cluster(smem_u32(&s.acc_empty[0]), 0);
        auto meet = [&](uint32_t parity) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.half[q]);
            return (bool)__all_sync(0xffffffffu, mbar_poll(&s.half[q], parity, &s.abort, a.wait_ns));
        };
        int it = 0;
        for (int tile = first; tile < tiles; tile += step) {
            if (__shfl_sync(0xffffffffu, s.abort, 0)) break;
            const int t = (tile % mt * 2 + rank) * kTile + r, n0 = tile / mt * kN;
            float2 acc[2][32];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 32; ++i) acc[b][i] = make_float2(0.f, 0.f);
            bool ok = true;
            for (int kb = 0; kb < a.nkb; ++kb, ++it) {
                const int st = it % kWdStages;
                ok = mbar_poll(&s.done[st], (it / kWdStages) & 1, &s.abort, a.wait_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint32_t ae = acc_empty + 16 * (it & 1);
                promote_block(acc, base + 256u * (it & 1), s.sc[st][r], lane,
                              [&](int tile_of_two) { mbar_arrive_cluster(ae + 8 * tile_of_two); });
            }
            if (!ok) {
                if (lane == 0) fail();
                break;
            }
            const int t0 = t - lane;  // the warp's rows t0 .. t0 + 31
            if constexpr (!GU) {
                store_rows64(a, s.out[warp - 4], lane, t0, n0 + 64 * j, acc[0], vec);
                store_rows64(a, s.out[warp - 4], lane, t0, n0 + kTile + 64 * j, acc[1], vec);
            } else {
                const int f0 = n0 + 64 * j, nv = a.N - f0;  // this thread's columns of h, and how many exist
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float2 g = acc[0][i], u = acc[1][i];
                    const float h0 = swiglu(g.x, u.x, 2 * i < nv), h1 = swiglu(g.y, u.y, 2 * i + 1 < nv);
                    m = max(m, max(abs_bits(h0), abs_bits(h1)));
                    acc[0][i] = make_float2(h0, h1);
                }
                // the two warps that share these rows meet twice: both have written, and both have read before
                // the next tile writes (a bounded wait: a named barrier would hold one for good if the other
                // had given up)
                s.part[j][r] = m;
                ok = meet(0);
                m = max(m, s.part[1 - j][r]);
                ok = ok && meet(1);
                if (!ok) {
                    if (lane == 0) fail();
                    break;
                }
                const BlockScale b = block_scale(m, a.pow2);
                scale_pairs(acc[0], b);
                if (j == 0 && t < a.T) a.hs[(int64_t)t * nt + n0 / kTile] = b.scale;
                uint4 o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t c[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 x = acc[0][8 * i + 2 * e], y = acc[0][8 * i + 2 * e + 1];
                        c[e] = f32x4_to_e4m3x4(x.x, x.y, y.x, y.y);
                    }
                    o[i] = make_uint4(c[0], c[1], c[2], c[3]);
                }
                uint8_t *buf = s.out[warp - 4];
                stage_rows(buf, lane, o);
                // rows of h are padded to 16 bytes, and columns beyond N hold zeros
                uint8_t *h = a.h + (int64_t)t0 * a.ldh + f0 + 16 * (lane & 3);
                if (16 * (lane & 3) < nv)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = 8 * i + (lane >> 2);
                        if (t0 + row < a.T) *reinterpret_cast<uint4 *>(h + (int64_t)row * a.ldh) = staged_unit(buf, row, lane & 3);
                    }
            }
        }
    }
    // neither CTA leaves while the other's MMAs or arrivals may touch its memory
    tc_fence_before();
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

template <bool GU>
cudaError_t wide_launch(GemmArgs &a, const void *act, int64_t lda, const void *const *w, int64_t ldw, int K, int dev,
                        cudaStream_t s) {
    static std::atomic<bool> done[64];
    const cudaError_t e = allow_smem(done, dev, wide_kernel<GU>, kWdSmemBytes);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (int64_t)ceil_div(a.T, 2 * kTile) * ceil_div(a.N, GU ? kTile : 2 * kTile);
    const int64_t pairs = fp8_num_sms(dev) / 2;
    if (tiles > 0x3FFFFFFF || !make_rows_map_u8(&a.a, act, a.T, K, lda, kTile) ||
        !make_rows_map_u8(&a.w[0], w[0], a.N, K, ldw, kTile / 2) ||
        (GU && !make_rows_map_u8(&a.w[1], w[1], a.N, K, ldw, kTile / 2)))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs)));
    cfg.blockDim = dim3(kWdThreads);
    cfg.dynamicSmemBytes = kWdSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, wide_kernel<GU>, a);
}

// The bounded waits' limit and the tests' arrivals beyond those there are (moe_debug_set_fp8_wait).
std::atomic<uint64_t> g_wait_ns{0};
std::atomic<uint32_t> g_wait_where{0};
void set_waits(GemmArgs &a) {
    const uint64_t ns = g_wait_ns.load(std::memory_order_relaxed);
    a.wait_ns = ns ? ns : kWaitLimitNs;
    const uint32_t where = g_wait_where.load(std::memory_order_relaxed);
    a.extra = where == 1;
    a.extra_got = where == 2 ? 16 : 0;
}

template <bool GU>
cudaError_t gemm_launch(GemmArgs &a, const void *act, int64_t lda, const void *const *w, int64_t ldw, int K,
                        cudaStream_t s) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    // The narrowest token tile that holds all tokens (no weight byte is read twice), or a narrower one
    // whose grid, split four ways along K, the SMs hold at once. Measured, us, with 16, 32 and 64 tokens
    // per tile: 129280 x 4096, T = 16: 91, 95 and 106, and 123 with pairs; T = 32: 171, 103, 112;
    // 4096 x 4096, T = 32 (16: split two ways only): 6.5 and 5.4; 2048 x 4096, T = 64: 6.5 and 5.3;
    // 1003 x 1111, T = 64: 4.0, 5.5 and 5.8; shared expert 4096 x 2048, T = 32: 14.3 and 16.7.
    const int64_t nt = ceil_div(a.N, kTile), sms = fp8_num_sms(dev);
    if (a.T <= 16 || nt * ceil_div(a.T, 16) * 4 <= sms)
        return skinny_launch<16, GU>(a, act, lda, w, ldw, K, dev, s);
    if (a.T <= 32 || nt * ceil_div(a.T, 32) * 4 <= sms) return skinny_launch<32, GU>(a, act, lda, w, ldw, K, dev, s);
    // Above 64 tokens such tiles as long as the grid is one CTA per SM, then pairs of SMs. Measured, us:
    // 4096 x 4096, T = 256 (128 tiles): 14.3 against 18.1, T = 384 (192 tiles): about 30 against 18.7;
    // shared expert 4096 / 2048, T = 256 (64 tiles) 22.1 against 33.0, T = 512 (128 tiles) 32.9 against 33.4;
    // 2048 / 1024, T = 1024 (128 tiles) 21.6 against 23.0.
    if (a.T <= 64 || nt * ceil_div(a.T, 64) <= sms)
        return skinny_launch<64, GU>(a, act, lda, w, ldw, K, dev, s);
    return wide_launch<GU>(a, act, lda, w, ldw, K, dev, s);
}

}  // namespace

void set_fp8_debug_wait(uint64_t limit_ns, uint32_t where) {
    g_wait_ns.store(limit_ns, std::memory_order_relaxed);
    g_wait_where.store(where, std::memory_order_relaxed);
}

cudaError_t launch_fp8_gemm(const moe_fp8_gemm_desc &g, const uint8_t *act, const float *as, const uint8_t *w,
                            const float *ws, void *y, cudaStream_t s, bool w_early) {
    GemmArgs a;
    memset(&a, 0, sizeof a);
    a.as = as; a.ws[0] = ws; a.y = y; a.ldy = g.ldy; a.T = g.T; a.N = g.N; a.nkb = ceil_div(g.K, kTile);
    a.y_bf16 = g.y_type == MOE_T_BF16; a.accumulate = g.accumulate; a.w_early = w_early;
    if (!(a.err = device_error_word())) return cudaErrorInvalidDevice;
    set_waits(a);
    const void *wp[2] = {w, nullptr};
    return gemm_launch<false>(a, act, g.lda, wp, g.ldw, g.K, s);
}

cudaError_t launch_fp8_gate_up(const moe_fp8_ffn_desc &f, const moe_fp8_ffn_weights &w, const uint8_t *x,
                               const float *xs, uint8_t *h, float *hs, int64_t ldh, cudaStream_t s) {
    GemmArgs a;
    memset(&a, 0, sizeof a);
    a.as = xs; a.ws[0] = w.s1; a.ws[1] = w.s3; a.h = h; a.hs = hs; a.ldh = ldh; a.T = f.T; a.N = f.d_ff;
    a.nkb = ceil_div(f.d_model, kTile); a.pow2 = f.scale_mode == MOE_SCALE_POW2;
    if (!(a.err = device_error_word())) return cudaErrorInvalidDevice;
    set_waits(a);
    const void *wp[2] = {w.w1, w.w3};
    return gemm_launch<true>(a, x, f.ldx, wp, f.ld13, f.d_model, s);
}

}  // namespace moe
