/*
 * bitlinear_gated.h -- C ABI of the gated feed-forward block on one MI355X
 * (gfx950), with its backward pass.  Part of libbitlinear.so; bitlinear.h holds
 * the ternary products (and the status codes, dtypes, paths and the packed
 * format used here).
 *
 * The FFN block of bitlinear.h has one up projection.  A gated block has two,
 * from the same activation codes, and multiplies them:
 *   G = BitLinear_gate(X)    U = BitLinear_up(X)    H = act(G) * U
 *   Y = BitLinear_down(H)
 * G and U are formed in float32 exactly as every BitLinear output:
 * fp32(acc) * fp32(fp32(gamma * gamma_A) / 127), acc the exact INT32 sum.
 *   BITLINEAR_ACT_RELU2  H = fp32(fp32(r * r) * U), r = max(G, 0)
 *   BITLINEAR_ACT_SILU   H = G / (1 + exp(-G)) * U, within a few float32 roundings
 * [MBC], the shadowgraph.io page on a multimodal architecture around bitnet.cpp,
 * gives ReLU^2 as BitNet's activation; [PMV], the produtoramaxvision.com.br
 * article on BitNet b1.58, names SwiGLU among the operators that stay outside
 * BitLinear (its section on trade-offs).
 *
 * A training step:
 *   forward   bitlinear_quantize_activations (X) -> codes
 *             bitlinear_gated_forward_quantized (codes) -> H, and G, U kept
 *             H -> BitLinear (down)
 *   backward  dH (bitlinear_backward of the down projection)
 *             -> bitlinear_gated_backward (G, U) -> dG, dU in bfloat16
 *             -> bitlinear_gated_input_backward -> dX
 *             -> bitlinear_backward (dG with the gate's mask, dU with the up
 *                projection's; dX NULL) -> dW of both
 *
 * Conventions: those of bitlinear.h.  Device pointers to contiguous row-major
 * arrays owned by the caller, a stream, every argument checked on the host
 * before anything is launched, nothing allocated, no state kept.  The calls
 * may be captured into a graph.  The kernels run on the current device, which
 * the arrays and the stream must belong to.  No output may overlap an input,
 * another output or the workspace (BITLINEAR_ERR_ARG).
 * Sizes: those of bitlinear_forward for every product.
 * Results do not depend on scheduling: the same call gives the same bits.
 * Non-finite values in X give unspecified results, as everywhere in
 * bitlinear.h; in bitlinear_gated_backward they follow IEEE arithmetic.
 */
#ifndef BITLINEAR_GATED_H
#define BITLINEAR_GATED_H

#include <stddef.h>
#include <stdint.h>

#include "bitlinear.h"

#ifdef __cplusplus
extern "C" {
#endif

#define BITLINEAR_ACT_RELU2 0
#define BITLINEAR_ACT_SILU  1

/* ---- the gated hidden layer ---------------------------------------------- */
/*
 * X:      device [M, D], x_dtype BITLINEAR_F32 or _BF16.
 * packed_gate, packed_up: device packed codes of [F, D] ternary matrices,
 *         16-byte aligned; gamma_gate, gamma_up: device float32[1].
 * act:    BITLINEAR_ACT_RELU2 or _SILU.
 * H:      device [M, F], h_dtype BITLINEAR_F32 or _BF16 (output, rounded once
 *         for bfloat16).
 * G, U:   device [M, F], gu_dtype BITLINEAR_F32 or _BF16 (outputs, kept for the
 *         backward), both or neither.
 * path:   BITLINEAR_PATH_AUTO / _DECODE / _PREFILL; decode takes what
 *         bitlinear_forward's decode path takes ([F, D] as the weights).
 * workspace: >= bitlinear_forward_workspace_bytes(M, D) on the prefill path,
 *         256-byte aligned; may be NULL/0 on the decode path.  Scratch only:
 *         two calls that may overlap need one each.
 * One launch on the decode path; the quantiser and one or two GEMM launches
 * on the prefill path.
 * Errors: BITLINEAR_ERR_NULL, _SHAPE, _DTYPE, _ALIGN, _WORKSPACE, _ARG, _HIP.
 */
int bitlinear_gated_forward(const void* X, int x_dtype, int64_t M, int64_t D, int64_t F, const uint32_t* packed_gate,
                            const float* gamma_gate, const uint32_t* packed_up, const float* gamma_up, int act,
                            void* H, int h_dtype, void* G, void* U, int gu_dtype, int path, void* workspace,
                            size_t workspace_bytes, void* stream);

/* The same from activation codes (Xq int8 [M, padded_k(D)], 16-byte aligned;
 * gamma_a, rowsum: as bitlinear_quantize_activations writes them).  Runs the
 * decode kernel where that fits, else the INT8-MFMA GEMM; the results are the
 * same bits. */
int bitlinear_gated_forward_quantized(const int8_t* Xq, const float* gamma_a, const int32_t* rowsum, int64_t M,
                                      int64_t D, int64_t F, const uint32_t* packed_gate, const float* gamma_gate,
                                      const uint32_t* packed_up, const float* gamma_up, int act, void* H, int h_dtype,
                                      void* G, void* U, int gu_dtype, void* stream);

/* ---- the whole block -------------------------------------------------------- */
/*
 * Y = BitLinear_down(act(G) * U).  packed_down: [D_out, F] ternary; Y: device
 * float32 [M, D_out]; hidden: NULL, or device float32 [M, F], 16-byte aligned,
 * receiving H.  workspace: >= bitlinear_gated_ffn_workspace_bytes(M, D, F, D_out),
 * 256-byte aligned (the hidden layer when `hidden` is NULL, activation
 * codes, and parts of the down product where its tiles are few).  Three launches on the decode path (both its products fit it), four
 * or more on the prefill path.  Errors as above.
 */
size_t bitlinear_gated_ffn_workspace_bytes(int64_t M, int64_t D, int64_t F, int64_t D_out);

int bitlinear_gated_ffn_forward(const void* X, int x_dtype, int64_t M, int64_t D, int64_t F, int64_t D_out,
                                const uint32_t* packed_gate, const float* gamma_gate, const uint32_t* packed_up,
                                const float* gamma_up, int act, const uint32_t* packed_down, const float* gamma_down,
                                float* Y, float* hidden, int path, void* workspace, size_t workspace_bytes,
                                void* stream);

/* ---- backward: through the activation and the product ---------------------- */
/*
 * From dH and the kept G and U, each [M, F] (1 <= M, F; F <= 2^20;
 * M * F < 2^40), dtypes BITLINEAR_F32 or _BF16 (dh_dtype; gu_dtype for both of
 * G and U; d_dtype for both outputs):
 *   RELU2  dG = fp32(dH * fp32(U * fp32(2 r)))    dU = fp32(dH * fp32(r * r))
 *   SILU   dG = dH * U * s (1 + G (1 - s))        dU = dH * G * s     s = 1 / (1 + exp(-G))
 * rounded once more for BITLINEAR_BF16, which is what the products' backward
 * takes.  Arrays are aligned to their element size.
 * Errors: BITLINEAR_ERR_NULL, _SHAPE, _DTYPE, _ALIGN, _ARG, _HIP.
 */
int bitlinear_gated_backward(const void* dH, int dh_dtype, const void* G, const void* U, int gu_dtype, int64_t M,
                             int64_t F, int act, void* dG, void* dU, int d_dtype, void* stream);

/* ---- backward: the input's gradient ----------------------------------------- */
/*
 * dX = gamma_gate (dG W_gate) + gamma_up (dU W_up), W the ternary codes: both
 * products in one launch, float32 accumulation, each scaled and then added; with
 * few rows in parts of F, which a second launch adds in order (the activation
 * clip never binds, as for bitlinear_backward).  A row of dX depends on that row of
 * dG and dU alone: infinities and NaN in others do not reach it.
 * dG, dU: device bfloat16 [M, F] (bit patterns).  packedT_gate, packedT_up:
 * [D, F] matrices as bitlinear_pack_transposed writes them.  dX: device float32
 * [M, D].  workspace: >= bitlinear_gated_input_backward_workspace_bytes(M, F, D,
 * copies), 256-byte aligned, NULL/0 where that is 0.  copies: nonzero where F % 8 != 0
 * or dG or dU is not 16-byte aligned (padded copies of both are made).  Requires
 * M * padded_k(F) < 2^30.
 * Errors: BITLINEAR_ERR_NULL, _SHAPE, _ALIGN, _WORKSPACE, _ARG, _HIP.
 */
size_t bitlinear_gated_input_backward_workspace_bytes(int64_t M, int64_t F, int64_t D, int copies);

int bitlinear_gated_input_backward(const uint16_t* dG, const uint16_t* dU, int64_t M, int64_t F, int64_t D,
                                   const uint32_t* packedT_gate, const float* gamma_gate,
                                   const uint32_t* packedT_up, const float* gamma_up, float* dX, void* workspace,
                                   size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BITLINEAR_GATED_H */
