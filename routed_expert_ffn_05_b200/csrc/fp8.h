// Internal launchers of the FP8 operators (host side), and their tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"
#include "moe.h"

namespace moe {

// norm.cu, fp8_gemm.cu; arguments already checked (fp8_api.cu).
cudaError_t launch_rms_norm(const moe_norm_desc &n, const void *x, const void *residual, const void *weight,
                            void *sum, uint16_t *y, uint8_t *codes, float *scales, cudaStream_t s);
cudaError_t launch_fp8_quantize(const moe_fp8_quant_desc &q, const void *v, uint8_t *codes, float *scales,
                                cudaStream_t s);
// w_early: the preceding kernel on the stream is one of this library that does
// not write w and lets its dependents start only after its own predecessors
// have ended, so w may be read before it ends.
cudaError_t launch_fp8_gemm(const moe_fp8_gemm_desc &g, const uint8_t *act, const float *as, const uint8_t *w,
                            const float *ws, void *y, cudaStream_t s, bool w_early = false);
// h = FP8 by rows of silu(W1 x) * (W3 x), codes [T][ldh], scales [T][ceil(d_ff / 128)].
cudaError_t launch_fp8_gate_up(const moe_fp8_ffn_desc &f, const moe_fp8_ffn_weights &w, const uint8_t *x,
                               const float *xs, uint8_t *h, float *hs, int64_t ldh, cudaStream_t s);

// Test hook of the products' bounded waits (moe_debug_set_fp8_wait).
void set_fp8_debug_wait(uint64_t limit_ns, uint32_t where);

// Operand tiles: a matrix of `cols` one-byte elements whose rows start `ld`
// bytes apart (ld a multiple of 16, at least cols), in boxes of 128 elements x
// box_rows rows, 128-byte swizzled (rows of 128 bytes in shared memory, the
// K-major layout tcgen05.mma reads). A box reaches beyond cols or rows into
// zeros, never into the bytes between cols and ld. Base 16-byte aligned.
bool make_rows_map_u8(CUtensorMap *map, const void *base, uint64_t rows, uint64_t cols, uint64_t ld,
                      uint32_t box_rows);

}  // namespace moe
