/*
 * bitlinear_block.h -- C ABI of the operators that stand around BitLinear in a
 * BitNet block, for serving and for training on one MI355X (gfx950): layer
 * norm, ReLU^2, and activations kept in 8 bits between the forward and the
 * backward pass.  Part of libbitlinear.so; bitlinear.h holds the ternary
 * products (and the status codes and dtypes used here).
 *
 * [PMV] is the produtoramaxvision.com.br blog article on BitNet b1.58: its
 * section on trade-offs keeps the norm, there RMSNorm, outside BitLinear.  The
 * norm here is layer norm, with a mean and a bias; RMSNorm is not offered.
 * [MBC] is the shadowgraph.io page on a multimodal architecture around
 * bitnet.cpp: its bit_layers.py section gives ReLU^2 as BitNet's activation.
 *
 * A training step of a pre-norm block, with the calls of both headers:
 *   forward   X -> bitlinear_layer_norm (saves X in 8 bits, mean, rstd) -> Y
 *             Y -> bitlinear_quantize_activations, bitlinear_forward_quantized -> H
 *             H -> bitlinear_relu2 (saves H in 8 bits) -> A -> BitLinear (down)
 *   backward  dA (bitlinear_backward of the down projection)
 *             -> bitlinear_relu2_backward (from the saved H) -> dH
 *             -> bitlinear_backward of the up projection -> dY
 *             -> bitlinear_layer_norm_backward (from the saved X) -> dX, dweight, dbias
 *
 * Conventions: those of bitlinear.h.  Device pointers to contiguous row-major
 * arrays owned by the caller, a stream, every argument checked on the host
 * before anything is launched, nothing allocated, no state kept.  The calls
 * may be captured into a graph.  The kernels run on the current device, which
 * the arrays and the stream must belong to.  Arrays are aligned to their
 * element size unless a call says more; rows may have any length.  No output
 * may overlap an input or another output (BITLINEAR_ERR_ARG).
 * Sizes: 1 <= M <= 2^31, 1 <= K <= 2^20, M*K < 2^40.
 * Results do not depend on scheduling: the same call gives the same bits.
 *
 * Activations saved in 8 bits
 * ---------------------------
 * codes:  int8 [M, Kp], Kp = bitlinear_padded_k(K), 16-byte aligned; columns
 *         K..Kp-1 are 0.
 * scales: float32 [M, G], G = bitlinear_saved_groups(K) = Kp / 64: one scale
 *         for each group of 64 consecutive columns of a row.
 * 1 + 4/64 bytes a value.  With amax the largest magnitude of the group:
 *         scale = fp32(amax * fp32(1/127))
 *         s     = fp32(127 / amax)             (an IEEE division)
 *         code  = the integer nearest x * s    (the exact product, ties to even)
 *         x~    = fp32(scale * code)           (the value that is restored)
 * so |x~ - x| <= scale / 2 (1 + 2^-14) (the scale, s and x~ are rounded once
 * each) and |code| <= 127.  The scales follow the group's own values: an
 * outlier channel costs its 63 neighbours resolution and nobody else.  A group
 * whose amax is below 2^-100 is saved as zeros (scale 0, off by amax at most);
 * a group that holds an infinity or a NaN gets a NaN scale and is restored as 64
 * NaNs, so a training loop's check for them still sees it.
 * As an input these arrays are dtype BITLINEAR_SAVED8: the codes are the data
 * pointer, the scales the *_scales pointer beside it (not read for the other
 * dtypes).
 */
#ifndef BITLINEAR_BLOCK_H
#define BITLINEAR_BLOCK_H

#include <stddef.h>
#include <stdint.h>

#include "bitlinear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations saved in 8 bits, as an input dtype beside BITLINEAR_F32 and
 * BITLINEAR_BF16. */
#define BITLINEAR_SAVED8 2

/* G: scales of a saved row of K values, ceil(K / 64). */
int64_t bitlinear_saved_groups(int64_t K);

/* ---- activations saved in 8 bits ---------------------------------------- */
/*
 * codes, scales: see above (outputs).  X: device [M, K], x_dtype
 * BITLINEAR_F32 or _BF16.
 * Errors: BITLINEAR_ERR_NULL, _SHAPE, _DTYPE, _ALIGN, _ARG, _HIP.
 */
int bitlinear_save_activations(const void* X, int x_dtype, int64_t M, int64_t K,
                               int8_t* codes, float* scales, void* stream);

/* X[m, k] = x~ (rounded once, half to even, for BITLINEAR_BF16); x_dtype is
 * the output's, BITLINEAR_F32 or _BF16.  Errors as above. */
int bitlinear_restore_activations(const int8_t* codes, const float* scales, int64_t M, int64_t K,
                                  void* X, int x_dtype, void* stream);

/* ---- layer norm ---------------------------------------------------------- */
/*
 * For each row m of X:
 *   mean = sum_k X / K,  var = sum_k (X - mean)^2 / K,  rstd = 1 / sqrt(var + eps)
 *   Y    = (X - mean) * rstd * weight + bias
 *
 * X:      device [M, K], x_dtype BITLINEAR_F32, _BF16 or _SAVED8 (then
 *         x_scales: its scales; a norm recomputed from saved activations).
 * weight, bias: device float32 [K], each NULL for none (1 and 0).
 * eps:    finite and >= 0.
 * Y:      device [M, K], y_dtype BITLINEAR_F32 or _BF16 (output).
 * mean, rstd: device float32 [M] (outputs, for the backward), both or neither.
 * saved, saved_scales: X in 8 bits (outputs, as bitlinear_save_activations
 *         writes them, from the same read of X), both or neither; not with
 *         BITLINEAR_SAVED8 input (BITLINEAR_ERR_ARG).
 *
 * Arithmetic in float32: the mean first, then the squares of the differences
 * to it; Y is rounded once at the end.  Rows whose mean is 32 or more standard
 * deviations from 0 have it corrected by the sum of the differences, and
 * variance and Y are those about the corrected mean (the one that is stored): a
 * row of one value has that value as its mean and the bias as Y.
 * Errors: BITLINEAR_ERR_NULL (also one of a pair without the other), _SHAPE,
 * _DTYPE, _ALIGN, _ARG, _HIP.
 */
int bitlinear_layer_norm(const void* X, const float* x_scales, int x_dtype, int64_t M, int64_t K,
                         const float* weight, const float* bias, float eps, void* Y, int y_dtype,
                         float* mean, float* rstd, int8_t* saved, float* saved_scales, void* stream);

/* Workspace bytes of bitlinear_layer_norm_backward: partial sums of dweight
 * and dbias (at most 256 rows of 2 K float32; 0 for few rows of at most 16384
 * columns). */
size_t bitlinear_layer_norm_backward_workspace_bytes(int64_t M, int64_t K);

/*
 * With xhat = (X - mean) * rstd and g = dY * weight:
 *   dX      = rstd * (g - sum_k g / K - xhat * sum_k (g * xhat) / K)    [M, K]
 *   dweight = sum_m dY * xhat                                           [K]
 *   dbias   = sum_m dY                                                  [K]
 *
 * dY:     device [M, K], dy_dtype BITLINEAR_F32 (as bitlinear_backward writes
 *         its dX) or _BF16.
 * X, x_scales, x_dtype: the forward's input, whole or as it was saved in 8
 *         bits (BITLINEAR_SAVED8; xhat is then off by scale / 2 * rstd, so rows
 *         that lie many standard deviations from 0 are better kept whole).
 * mean, rstd: device float32 [M], from the forward.
 * weight: device float32 [K], or NULL for none.
 * dX:     device [M, K], dx_dtype BITLINEAR_F32 or _BF16, or NULL.
 * dweight, dbias: device float32 [K], each may be NULL (of dX, dweight and
 *         dbias at least one is given).
 * workspace: >= bitlinear_layer_norm_backward_workspace_bytes(M, K), 256-byte
 *         aligned; may be NULL/0 where that is 0, or without dweight and dbias.
 *         Scratch only: two calls that may overlap need one each.
 *
 * Arithmetic in float32; the sums over m run over fixed sets of rows, one
 * after the other, and over the sets in a fixed order (no atomics).
 * Errors: BITLINEAR_ERR_NULL, _SHAPE, _DTYPE, _ALIGN, _WORKSPACE, _ARG, _HIP.
 */
int bitlinear_layer_norm_backward(const void* dY, int dy_dtype, const void* X, const float* x_scales,
                                  int x_dtype, const float* mean, const float* rstd, int64_t M, int64_t K,
                                  const float* weight, void* dX, int dx_dtype, float* dweight, float* dbias,
                                  void* workspace, size_t workspace_bytes, void* stream);

/* ---- ReLU^2 ---------------------------------------------------------------- */
/*
 * A = max(H, 0)^2: fp32(r * r), r = max(H, 0), as the FFN block forward's
 * hidden layer, but for a NaN: it stays a NaN here (there it becomes 0). [MBC]
 *
 * H:      device [M, K], h_dtype BITLINEAR_F32, _BF16 or _SAVED8 (then
 *         h_scales: its scales).
 * A:      device [M, K], a_dtype BITLINEAR_F32 or _BF16 (output).
 * saved, saved_scales: H in 8 bits (outputs), both or neither; not with
 *         BITLINEAR_SAVED8 input (BITLINEAR_ERR_ARG).
 * Errors: BITLINEAR_ERR_NULL, _SHAPE, _DTYPE, _ALIGN, _ARG, _HIP.
 */
int bitlinear_relu2(const void* H, const float* h_scales, int h_dtype, int64_t M, int64_t K,
                    void* A, int a_dtype, int8_t* saved, float* saved_scales, void* stream);

/*
 * dH = dA * 2 max(H, 0): fp32(dA * fp32(2 r)), rounded once more for a
 * bfloat16 dH (what bitlinear_backward takes as its dY).
 *
 * dA: device [M, K], da_dtype BITLINEAR_F32 or _BF16.  H, h_scales, h_dtype:
 * as for bitlinear_relu2, whole or saved.  dH: device [M, K], dh_dtype
 * BITLINEAR_F32 or _BF16 (output).  Errors as above.
 */
int bitlinear_relu2_backward(const void* dA, int da_dtype, const void* H, const float* h_scales, int h_dtype,
                             int64_t M, int64_t K, void* dH, int dh_dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BITLINEAR_BLOCK_H */
