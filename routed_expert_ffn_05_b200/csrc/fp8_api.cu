// C ABI entry points of the FP8 operators (moe.h): argument checks, workspace
// carving and launches, and the MoE block that runs them around the layer.
#include <math.h>
#include <stdio.h>

#include "common.cuh"
#include "fp8.h"

namespace moe {
namespace {

bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool valid_type(int32_t t) { return t == MOE_T_BF16 || t == MOE_T_F32; }
bool valid_scale(int32_t m) { return m == MOE_SCALE_F32 || m == MOE_SCALE_POW2; }
int type_size(int32_t t) { return t == MOE_T_BF16 ? 2 : 4; }
int64_t blocks_of(int64_t n) { return (n + 127) / 128; }
int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

moe_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return MOE_OK;
    fprintf(stderr, "libmoe: CUDA error: %s\n", cudaGetErrorString(e));
    return MOE_ERR_CUDA;
}

// A row-major buffer as an address range (empty for a NULL pointer).
struct Span {
    uintptr_t lo, hi;
    Span(const void *p, int64_t rows, int64_t cols, int64_t ld, int size) {
        lo = reinterpret_cast<uintptr_t>(p);
        const unsigned __int128 end = (unsigned __int128)lo + (unsigned __int128)((rows - 1) * (__int128)ld + cols) * size;
        hi = !p || rows <= 0 ? lo : end > UINTPTR_MAX ? UINTPTR_MAX : (uintptr_t)end;
    }
    bool meets(const Span &o) const { return lo < o.hi && o.lo < hi; }
};

// True when out[i] overlaps an input or another output.
bool overlaps(const Span *in, int n_in, const Span *out, int n_out) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j)
            if (out[i].meets(in[j])) return true;
        for (int j = 0; j < i; ++j)
            if (out[i].meets(out[j])) return true;
    }
    return false;
}

constexpr int64_t kMaxLd = (int64_t)1 << 36;  // a TMA row stride stays below 2^40 bytes
constexpr int kMaxNormD = 32768;
constexpr int kMaxDim = 1 << 28;  // of a matrix: every tile and row index of a kernel stays in 32 bits

moe_status check_norm(const moe_norm_desc *n) {
    if (!n) return MOE_ERR_INVALID_ARG;
    if (n->T < 0 || n->d <= 0 || !valid_type(n->x_type) || !valid_type(n->res_type) || !valid_type(n->w_type) ||
        !valid_scale(n->scale_mode) || !(n->eps >= 0.f) || !isfinite(n->eps))
        return MOE_ERR_INVALID_ARG;
    if (n->d > kMaxNormD || n->T > kMaxDim) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

bool valid_ld(int64_t ld, int64_t cols) { return ld >= cols && ld < kMaxLd; }
bool valid_code_ld(int64_t ld, int64_t cols) { return valid_ld(ld, cols) && ld % 16 == 0; }

moe_status check_ffn(const moe_fp8_ffn_desc *f) {
    if (!f) return MOE_ERR_INVALID_ARG;
    if (f->T < 0 || f->d_model <= 0 || f->d_ff <= 0 || !valid_type(f->y_type) || !valid_scale(f->scale_mode) ||
        (f->accumulate != 0 && f->accumulate != 1) || (f->accumulate && f->y_type != MOE_T_F32))
        return MOE_ERR_INVALID_ARG;
    if (!valid_code_ld(f->ldx, f->d_model) || !valid_code_ld(f->ld13, f->d_model) ||
        !valid_code_ld(f->ld2, f->d_ff) || !valid_ld(f->ldy, f->d_model))
        return MOE_ERR_INVALID_ARG;
    if (f->T > kMaxDim || f->d_model > kMaxDim || f->d_ff > kMaxDim) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

bool codes_ok(const uint8_t *codes, const float *scales) {
    return codes && scales && aligned(codes, 16) && aligned(scales, 4);
}

bool ffn_weights_ok(const moe_fp8_ffn_weights *w) {
    return w && codes_ok(w->w1, w->s1) && codes_ok(w->w3, w->s3) && codes_ok(w->w2, w->s2);
}

struct FfnWs {
    int64_t ldh, h, hs, total;
    FfnWs(int64_t T, int64_t d_ff) {
        ldh = up16(d_ff);
        h = 0;
        hs = al256(T * ldh);
        total = al256(hs + T * blocks_of(d_ff) * 4);
    }
};

cudaError_t run_ffn(const moe_fp8_ffn_desc &f, const moe_fp8_ffn_weights &w, const uint8_t *x, const float *xs, void *y,
                    uint8_t *ws, cudaStream_t s) {
    const FfnWs L(f.T, f.d_ff);
    uint8_t *h = ws + L.h;
    float *hs = reinterpret_cast<float *>(ws + L.hs);
    cudaError_t e = launch_fp8_gate_up(f, w, x, xs, h, hs, L.ldh, s);
    if (e != cudaSuccess) return e;
    moe_fp8_gemm_desc g;
    g.T = f.T; g.N = f.d_model; g.K = f.d_ff; g.y_type = f.y_type; g.accumulate = f.accumulate;
    g.lda = L.ldh; g.ldw = f.ld2; g.ldy = f.ldy;
    return launch_fp8_gemm(g, h, hs, w.w2, w.s2, y, s, true);
}

// moe_block: the layer's workspace, then the normed rows and the FFN's.
struct BlockWs {
    int64_t layer, xn, x8, xs, ffn, total;
    explicit BlockWs(const moe_dims &d, int64_t layer_bytes) {
        layer = 0;
        xn = al256(layer_bytes);
        x8 = al256(xn + (int64_t)d.T * d.d_model * 2);
        xs = al256(x8 + (int64_t)d.T * d.d_model);
        ffn = al256(xs + (int64_t)d.T * blocks_of(d.d_model) * 4);
        total = ffn + (d.d_ff_shared > 0 ? FfnWs(d.T, d.d_ff_shared).total : 0);
    }
};

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_rms_norm(const moe_norm_desc *desc, const void *x, const void *residual, const void *weight,
                        void *residual_out, uint16_t *y, uint8_t *codes, float *scales, void *stream) {
    moe_status st = check_norm(desc);
    if (st != MOE_OK) return st;
    const moe_norm_desc &n = *desc;
    const bool any = residual_out || y || codes;
    if (n.T > 0 && (!x || !any)) return MOE_ERR_INVALID_ARG;
    if ((residual_out && !residual) || !codes != !scales) return MOE_ERR_INVALID_ARG;
    if (!valid_ld(n.ldx, n.d) || (residual && !valid_ld(n.ldr, n.d)) || (y && !valid_ld(n.ldy, n.d)) ||
        (codes && !valid_ld(n.ldq, n.d)))
        return MOE_ERR_INVALID_ARG;
    const int xs = type_size(n.x_type), rs = type_size(n.res_type), wsz = type_size(n.w_type);
    if (!aligned(x, xs) || !aligned(residual, rs) || !aligned(residual_out, rs) || !aligned(weight, wsz) ||
        !aligned(y, 2) || !aligned(scales, 4))
        return MOE_ERR_INVALID_ARG;
    if (n.T == 0) return MOE_OK;
    const bool in_place = residual_out == residual;
    const Span in[] = {Span(x, n.T, n.d, n.ldx, xs), Span(weight, 1, n.d, n.d, wsz),
                       Span(in_place ? nullptr : residual, n.T, n.d, n.ldr, rs)};
    const Span out[] = {Span(residual_out, n.T, n.d, n.ldr, rs), Span(y, n.T, n.d, n.ldy, 2),
                        Span(codes, n.T, n.d, n.ldq, 1), Span(scales, n.T, blocks_of(n.d), blocks_of(n.d), 4)};
    if (overlaps(in, 3, out, 4)) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_rms_norm(n, x, residual, weight, residual_out, y, codes, scales,
                                       static_cast<cudaStream_t>(stream)));
}

moe_status moe_fp8_quantize(const moe_fp8_quant_desc *desc, const void *v, uint8_t *codes, float *scales,
                            void *stream) {
    if (!desc) return MOE_ERR_INVALID_ARG;
    const moe_fp8_quant_desc &q = *desc;
    if (q.rows < 0 || q.cols <= 0 || !valid_type(q.v_type) || (q.block_rows != 1 && q.block_rows != 128) ||
        !valid_scale(q.scale_mode) || !valid_ld(q.ldv, q.cols) || !valid_ld(q.ldq, q.cols))
        return MOE_ERR_INVALID_ARG;
    if (q.rows > kMaxDim || q.cols > kMaxDim || (int64_t)q.rows * ((q.cols + 511) / 512) > (int64_t)1 << 30)
        return MOE_ERR_UNSUPPORTED;
    const int vs = type_size(q.v_type);
    if (q.rows == 0) return MOE_OK;
    if (!v || !codes || !scales || !aligned(v, vs) || !aligned(scales, 4)) return MOE_ERR_INVALID_ARG;
    const int64_t nb = blocks_of(q.cols);
    const Span in[] = {Span(v, q.rows, q.cols, q.ldv, vs)};
    const Span out[] = {Span(codes, q.rows, q.cols, q.ldq, 1),
                        Span(scales, q.block_rows == 1 ? q.rows : blocks_of(q.rows), nb, nb, 4)};
    if (overlaps(in, 1, out, 2)) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_fp8_quantize(q, v, codes, scales, static_cast<cudaStream_t>(stream)));
}

moe_status moe_fp8_gemm(const moe_fp8_gemm_desc *desc, const uint8_t *a, const float *a_scales, const uint8_t *w,
                        const float *w_scales, void *y, void *stream) {
    if (!desc) return MOE_ERR_INVALID_ARG;
    const moe_fp8_gemm_desc &g = *desc;
    if (g.T < 0 || g.N <= 0 || g.K <= 0 || !valid_type(g.y_type) || (g.accumulate != 0 && g.accumulate != 1) ||
        (g.accumulate && g.y_type != MOE_T_F32) || !valid_code_ld(g.lda, g.K) || !valid_code_ld(g.ldw, g.K) ||
        !valid_ld(g.ldy, g.N))
        return MOE_ERR_INVALID_ARG;
    if (g.T > kMaxDim || g.N > kMaxDim || g.K > kMaxDim) return MOE_ERR_UNSUPPORTED;
    if (g.T == 0) return MOE_OK;
    const int ys = type_size(g.y_type);
    if (!codes_ok(a, a_scales) || !codes_ok(w, w_scales) || !y || !aligned(y, ys)) return MOE_ERR_INVALID_ARG;
    const int64_t nb = blocks_of(g.K);
    const Span in[] = {Span(a, g.T, g.K, g.lda, 1), Span(w, g.N, g.K, g.ldw, 1), Span(a_scales, g.T, nb, nb, 4),
                       Span(w_scales, blocks_of(g.N), nb, nb, 4)};
    const Span out[] = {Span(y, g.T, g.N, g.ldy, ys)};
    if (overlaps(in, 4, out, 1)) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_fp8_gemm(g, a, a_scales, w, w_scales, y, static_cast<cudaStream_t>(stream)));
}

moe_status moe_fp8_ffn_workspace_size(const moe_fp8_ffn_desc *desc, size_t *bytes) {
    moe_status st = check_ffn(desc);
    if (st != MOE_OK) return st;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = (size_t)FfnWs(desc->T, desc->d_ff).total;
    return MOE_OK;
}

moe_status moe_shared_ffn_fp8(const moe_fp8_ffn_desc *desc, const moe_fp8_ffn_weights *weights, const uint8_t *x,
                              const float *x_scales, void *y, void *ws, void *stream) {
    moe_status st = check_ffn(desc);
    if (st != MOE_OK) return st;
    const moe_fp8_ffn_desc &f = *desc;
    if (f.T == 0) return MOE_OK;
    const int ys = type_size(f.y_type);
    if (!ffn_weights_ok(weights) || !codes_ok(x, x_scales) || !y || !aligned(y, ys) || !ws || !aligned(ws, 256))
        return MOE_ERR_INVALID_ARG;
    const moe_fp8_ffn_weights &w = *weights;
    const int64_t nd = blocks_of(f.d_model), nf = blocks_of(f.d_ff);
    const Span in[] = {Span(x, f.T, f.d_model, f.ldx, 1),       Span(x_scales, f.T, nd, nd, 4),
                       Span(w.w1, f.d_ff, f.d_model, f.ld13, 1), Span(w.s1, nf, nd, nd, 4),
                       Span(w.w3, f.d_ff, f.d_model, f.ld13, 1), Span(w.s3, nf, nd, nd, 4),
                       Span(w.w2, f.d_model, f.d_ff, f.ld2, 1),  Span(w.s2, nd, nf, nf, 4)};
    const Span out[] = {Span(y, f.T, f.d_model, f.ldy, ys), Span(ws, 1, FfnWs(f.T, f.d_ff).total, 0, 1)};
    if (overlaps(in, 8, out, 2)) return MOE_ERR_INVALID_ARG;
    return cuda_status(run_ffn(f, w, x, x_scales, y, static_cast<uint8_t *>(ws), static_cast<cudaStream_t>(stream)));
}

moe_status moe_block_workspace_size(const moe_dims *dims, size_t *bytes) {
    size_t layer = 0;
    moe_status st = moe_workspace_size(dims, &layer);
    if (st != MOE_OK) return st;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = (size_t)BlockWs(*dims, (int64_t)layer).total;
    return MOE_OK;
}

moe_status moe_block(const moe_dims *dims, const moe_weights *weights, const moe_norm_desc *norm,
                     const moe_fp8_ffn_weights *shared, const void *x, const void *residual, const void *norm_weight,
                     void *residual_out, const int32_t *token_ids, float *y, void *ws, void *stream) {
    size_t layer = 0;
    moe_status st = moe_workspace_size(dims, &layer);
    if (st != MOE_OK) return st;
    if ((st = check_norm(norm)) != MOE_OK) return st;
    if (norm->T != dims->T || norm->d != dims->d_model) return MOE_ERR_INVALID_ARG;
    if (dims->T == 0) return MOE_OK;
    if (!ws || !aligned(ws, 256) || !y || !aligned(y, 16)) return MOE_ERR_INVALID_ARG;
    const int64_t T = dims->T, d = dims->d_model, F = dims->d_ff_shared;
    const int64_t nd = blocks_of(d), nf = blocks_of(F);
    if (F > 0 && !ffn_weights_ok(shared)) return MOE_ERR_INVALID_ARG;
    const BlockWs L(*dims, (int64_t)layer);
    uint8_t *w = static_cast<uint8_t *>(ws);
    // nothing is launched before every stage's arguments are known to be good: the norm's by its
    // own checks on the first launch below, the others' here
    const int xs = type_size(norm->x_type), rs = type_size(norm->res_type);
    moe_dims dl = *dims;
    dl.d_ff_shared = 0;  // the layer computes the routed experts only
    if (!weights || !weights->w1 || !weights->w3 || !weights->w2 || !aligned(weights->w1, 256) ||
        !aligned(weights->w3, 256) || !aligned(weights->w2, 256) ||
        (dl.route == MOE_ROUTE_SOFTMAX_TOPK && (!weights->w_router || !aligned(weights->w_router, 16))) ||
        (dl.route == MOE_ROUTE_HASH && !token_ids))
        return MOE_ERR_INVALID_ARG;
    size_t pw[3];
    for (int i = 0; i < 3; ++i)
        if ((st = moe_packed_size(&dl, i == 0 ? MOE_MAT_W1 : i == 1 ? MOE_MAT_W3 : MOE_MAT_W2, &pw[i])) != MOE_OK)
            return st;
    const bool router = dl.route == MOE_ROUTE_SOFTMAX_TOPK;
    const Span none(nullptr, 0, 0, 0, 1);
    const Span in[] = {Span(x, T, d, norm->ldx, xs),
                       Span(residual_out == residual ? nullptr : residual, T, d, norm->ldr, rs),
                       Span(norm_weight, 1, d, d, type_size(norm->w_type)),
                       F > 0 ? Span(shared->w1, F, d, d, 1) : none,
                       F > 0 ? Span(shared->w3, F, d, d, 1) : none,
                       F > 0 ? Span(shared->w2, d, F, F, 1) : none,
                       F > 0 ? Span(shared->s1, nf, nd, nd, 4) : none,
                       F > 0 ? Span(shared->s3, nf, nd, nd, 4) : none,
                       F > 0 ? Span(shared->s2, nd, nf, nf, 4) : none,
                       Span(weights->w1, 1, (int64_t)pw[0], 0, 1),
                       Span(weights->w3, 1, (int64_t)pw[1], 0, 1),
                       Span(weights->w2, 1, (int64_t)pw[2], 0, 1),
                       router ? Span(weights->w_router, dl.E, d, d, 2) : Span(token_ids, 1, T, 0, 4),
                       router ? Span(weights->router_bias, 1, dl.E, 0, 4) : none};
    const Span out[] = {Span(y, T, d, d, 4), Span(ws, 1, L.total, 0, 1), Span(residual_out, T, d, norm->ldr, rs)};
    if (overlaps(in, 14, out, 3)) return MOE_ERR_INVALID_ARG;
    uint16_t *xn = reinterpret_cast<uint16_t *>(w + L.xn);
    uint8_t *x8 = F > 0 ? w + L.x8 : nullptr;
    float *x8s = F > 0 ? reinterpret_cast<float *>(w + L.xs) : nullptr;
    moe_norm_desc n = *norm;
    n.ldy = n.ldq = d;
    if ((st = moe_rms_norm(&n, x, residual, norm_weight, residual_out, xn, x8, x8s, stream)) != MOE_OK) return st;
    if ((st = moe_layer(&dl, weights, xn, token_ids, y, ws, stream)) != MOE_OK || F == 0) return st;
    moe_fp8_ffn_desc f;
    f.T = dims->T; f.d_model = dims->d_model; f.d_ff = dims->d_ff_shared;
    f.y_type = MOE_T_F32; f.accumulate = 1; f.scale_mode = norm->scale_mode;
    f.ldx = f.ld13 = f.ldy = d;
    f.ld2 = F;
    return cuda_status(run_ffn(f, *shared, x8, x8s, y, w + L.ffn, static_cast<cudaStream_t>(stream)));
}

moe_status moe_debug_set_fp8_wait(uint64_t limit_ns, uint32_t where) {
    if (where > 2) return MOE_ERR_INVALID_ARG;
    set_fp8_debug_wait(limit_ns, where);
    return MOE_OK;
}

}  // extern "C"
