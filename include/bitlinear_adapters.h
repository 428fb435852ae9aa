/*
 * bitlinear_adapters.h -- C ABI of low-rank adapters beside a BitLinear
 * projection, and of dropout, for serving and for fine-tuning on one MI355X
 * (gfx950).  Part of libbitlinear.so; bitlinear.h holds the ternary products
 * (and the status codes, dtypes and paths used here).
 *
 * A ternary projection is shared and frozen; an adapter adds a product of rank
 * R to it, and every token may have one of its own:
 *   Y[m] = BitLinear(X)[m] + scale[a] (X[m] down[a]^T) up[a]      a = rows[m]
 * With T[m] = X[m] down[a]^T and V[m] = scale[a] dY[m] up[a]^T the gradients are
 *   dX[m]    = ... + V[m] down[a]
 *   ddown[a] = sum over rows[m] = a of V[m]^T X[m]
 *   dup[a]   = scale[a] * sum over rows[m] = a of T[m]^T dY[m]
 *
 * Adapters
 * --------
 * down:   device [A, R, K], up: device [A, R, N], w_dtype BITLINEAR_F32 or _BF16
 *         for both: the R rows of an adapter lie along the input's columns in
 *         `down` and along the output's in `up` (an [N, R] matrix is stored
 *         transposed, once).  Aligned to their element size.
 * scales: device float32 [A].
 * rows:   device int32 [M], the adapter of every token.  A value below 0, or of
 *         A or more, is a token without an adapter.  Tokens of one adapter need
 *         not lie together; where they do (requests one after another), its
 *         weights are read less often.
 * Sizes:  1 <= A <= 65535, 1 <= R <= 256, A * R * K and A * R * N < 2^40, and
 *         those of bitlinear_forward for M, N and K.
 *
 * Arithmetic: products and sums in float32 accuracy whatever the types.
 * float32 values go to the bf16 matrix cores as sums of three bfloat16 numbers,
 * exact for values of 2^-110 and more (smaller ones to 2^-134), and at most
 * 2^-24 (1 + 2^-10) of a product of two of them is left out, with either sign;
 * products with bfloat16 weights or inputs are whole.  Sums are float32; those
 * that come within 2^-8 of the largest float32 on the way may overflow.  T is
 * float32 and is not rounded to fewer bits.  Every sum is over fixed parts in a
 * fixed order (no atomics): results do not depend on scheduling, and the same
 * call gives the same bits.
 * A token's outputs depend on its own row of X (or dY) and its own adapter
 * only: infinities and NaN elsewhere do not reach it.  In a token's own row or
 * adapter they make its outputs non-finite, not always with the same value as
 * in IEEE arithmetic (an infinity may come out as NaN).
 *
 * Conventions: those of bitlinear.h.  Device pointers to contiguous row-major
 * arrays owned by the caller, a stream, every argument checked on the host
 * before anything is launched, nothing allocated, no state kept.  The calls
 * may be captured into a graph.  The kernels run on the current device, which
 * the arrays and the stream must belong to.  No output may overlap an input,
 * another output or the workspace (BITLINEAR_ERR_ARG).  A workspace is scratch
 * only: two calls that may overlap need one each.
 */
#ifndef BITLINEAR_ADAPTERS_H
#define BITLINEAR_ADAPTERS_H

#include <stddef.h>
#include <stdint.h>

#include "bitlinear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- forward --------------------------------------------------------------- */
/*
 * Y[m] += scale[a] (X[m] down[a]^T) up[a]; rows of Y without an adapter are
 * left as they are.
 * X: device [M, K], x_dtype BITLINEAR_F32 or _BF16.  Y: device float32 [M, N],
 * updated.  T: NULL, or device float32 [M, R], receiving X[m] down[a]^T for the
 * backward (zeros for tokens without an adapter).
 * workspace: >= bitlinear_adapters_workspace_bytes(M, K, N, R), 256-byte
 * aligned.  Errors: BITLINEAR_ERR_NULL, _SHAPE, _DTYPE, _ALIGN, _WORKSPACE,
 * _ARG, _HIP.
 */
size_t bitlinear_adapters_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t R);

int bitlinear_adapters_forward(const void* X, int x_dtype, int64_t M, int64_t K, int64_t N, const int32_t* rows,
                               int64_t A, int64_t R, const void* down, const void* up, int w_dtype,
                               const float* scales, float* Y, float* T, void* workspace, size_t workspace_bytes,
                               void* stream);

/*
 * The projection and the adapters: Y = bitlinear_forward(X) and then the above
 * on it.  packed, gamma, path: as for bitlinear_forward_ex.  workspace: >=
 * bitlinear_adapted_workspace_bytes(M, K, N, R), 256-byte aligned (activation
 * codes among it, and parts of the product where its tiles are few).  Up to 16 tokens
 * take two launches, with three exceptions: weights with so many rows that the decode
 * path streams them, tokens whose codes do not fit the decode kernel's LDS in four
 * pieces, fewer than 8 inputs.  Those, more tokens and the prefill path take three or
 * more.  The adapters' sums may be formed in another order than by the two calls one
 * after the other; both are within the accuracy above.
 */
size_t bitlinear_adapted_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t R);

int bitlinear_adapted_forward(const void* X, int x_dtype, int64_t M, int64_t K, const uint32_t* packed, int64_t N,
                              const float* gamma, const int32_t* rows, int64_t A, int64_t R, const void* down,
                              const void* up, int w_dtype, const float* scales, float* Y, float* T, int path,
                              void* workspace, size_t workspace_bytes, void* stream);

/* ---- backward --------------------------------------------------------------- */
/*
 * dY: device [M, N], dy_dtype BITLINEAR_F32 or _BF16.  X: as in the forward
 * (needed for ddown); T: the forward's (needed for dup).
 * dX:    device float32 [M, K], or NULL.  accumulate != 0: the adapters' part is
 *        added to it (to bitlinear_backward's dX) and rows without an adapter
 *        are left as they are; 0: it is written, zeros for those rows.
 * ddown: device float32 [A, R, K], or NULL; dup: device float32 [A, R, N], or
 *        NULL (of the three at least one is given).  Both are written whole:
 *        zeros for an adapter that no token has.
 * workspace: >= bitlinear_adapters_backward_workspace_bytes(M, K, N, A, R),
 *        256-byte aligned.
 * Errors: as above.
 */
size_t bitlinear_adapters_backward_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t A, int64_t R);

int bitlinear_adapters_backward(const void* dY, int dy_dtype, const void* X, int x_dtype, const float* T, int64_t M,
                                int64_t K, int64_t N, const int32_t* rows, int64_t A, int64_t R, const void* down,
                                const void* up, int w_dtype, const float* scales, float* dX, int accumulate,
                                float* ddown, float* dup, void* workspace, size_t workspace_bytes, void* stream);

/* ---- dropout ------------------------------------------------------------------- */
/*
 * For value i = 0 .. n - 1:
 *   Y[i] = (w[i] >= round(p 2^32) ? fp32(X[i] * fp32(1 / (1 - p))) : 0) + residual[i]
 * in float32, rounded once for a bfloat16 Y.  w[i] is 32 random bits that are
 * never stored: word i % 4 of Philox4x32-10 (Salmon et al., "Parallel random
 * numbers: as easy as 1, 2, 3", 2011) with the counter (i / 4, offset) and the
 * key `seed`, each 64 bits, low word first.  The backward pass is the same call
 * on the gradient, with the same p, seed and offset.
 *
 * X: device [n], x_dtype BITLINEAR_F32 or _BF16.  residual: NULL, or device [n],
 * r_dtype BITLINEAR_F32 or _BF16.  Y: device [n], y_dtype likewise (output).
 * Y may be X or the residual itself where the types agree, else it may overlap
 * neither.  0 <= p < 1; p = 0 keeps every value.  1 <= n < 2^40.
 * A dropped value is 0 whatever X holds there.
 * Errors: BITLINEAR_ERR_NULL, _SHAPE, _DTYPE, _ALIGN, _ARG, _HIP.
 */
int bitlinear_dropout(const void* X, int x_dtype, const void* residual, int r_dtype, int64_t n, double p,
                      uint64_t seed, uint64_t offset, void* Y, int y_dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BITLINEAR_ADAPTERS_H */
