// C ABI of the gated feed-forward block (include/bitlinear_gated.h): argument
// checks on the host, then the launches.
#include <stdint.h>

#include "../../include/bitlinear_gated.h"
#include "abi_common.hpp"
#include "gated_ops.hpp"
#include "prefill_parts.hpp"

using namespace bitlinear;

namespace {

bool known_path(int path) {
  return path == BITLINEAR_PATH_AUTO || path == BITLINEAR_PATH_DECODE || path == BITLINEAR_PATH_PREFILL;
}
bool known_act(int act) { return act == BITLINEAR_ACT_RELU2 || act == BITLINEAR_ACT_SILU; }

Range packed_range(const uint32_t* p, int64_t N, int64_t K) {
  return {p, static_cast<uint64_t>(N) * static_cast<uint64_t>(padded_k(K)) / 4};
}

// Checks that both forwards share: weights, activation, outputs.
int check_gated(int64_t M, int64_t D, int64_t F, const GatedWeights& w, const GatedOutputs& o) {
  if (!w.gate || !w.gamma_gate || !w.up || !w.gamma_up || !o.H || !o.G != !o.U) return BITLINEAR_ERR_NULL;
  const int st = check_mnk(M, F, D);
  if (st) return st;
  if (!plain_dtype(o.h_dtype) || (o.G && !plain_dtype(o.gu_dtype))) return BITLINEAR_ERR_DTYPE;
  if (!known_act(w.act)) return BITLINEAR_ERR_ARG;
  if (!aligned(w.gate, 16) || !aligned(w.up, 16) || !aligned(w.gamma_gate, 4) || !aligned(w.gamma_up, 4) ||
      !aligned_to(o.H, o.h_dtype) || (o.G && (!aligned_to(o.G, o.gu_dtype) || !aligned_to(o.U, o.gu_dtype))))
    return BITLINEAR_ERR_ALIGN;
  return BITLINEAR_OK;
}

}  // namespace

extern "C" {

int bitlinear_gated_forward(const void* X, int x_dtype, int64_t M, int64_t D, int64_t F, const uint32_t* packed_gate,
                            const float* gamma_gate, const uint32_t* packed_up, const float* gamma_up, int act,
                            void* H, int h_dtype, void* G, void* U, int gu_dtype, int path, void* workspace,
                            size_t workspace_bytes, void* stream) {
  const GatedWeights w = {packed_gate, gamma_gate, packed_up, gamma_up, act};
  const GatedOutputs o = {H, G, U, h_dtype, gu_dtype};
  if (!X) return BITLINEAR_ERR_NULL;
  int st = check_gated(M, D, F, w, o);
  if (st) return st;
  st = check_x(X, x_dtype);
  if (st) return st;
  if (!known_path(path)) return BITLINEAR_ERR_ARG;
  const bool fits = decode_fits(M, D, F);
  if (path == BITLINEAR_PATH_DECODE && !fits) return BITLINEAR_ERR_SHAPE;
  const bool decode = fits && path != BITLINEAR_PATH_PREFILL;
  const size_t need = decode ? 0 : prefill_ws_bytes(M, D);
  if (need) {
    if (!workspace || workspace_bytes < need) return BITLINEAR_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return BITLINEAR_ERR_ALIGN;
  }
  const Range out[] = {array(H, h_dtype, M, F), array(G, gu_dtype, M, F), array(U, gu_dtype, M, F),
                       {need ? workspace : nullptr, need}};
  const Range in[] = {array(X, x_dtype, M, D),    packed_range(packed_gate, F, D), packed_range(packed_up, F, D),
                      floats(gamma_gate, 1),      floats(gamma_up, 1)};
  if (any_overlap(out, in)) return BITLINEAR_ERR_ARG;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (decode) return hip_status(launch_gated_decode(X, x_dtype, nullptr, nullptr, nullptr, M, D, F, w, o, s));
  const PrefillWs c = prefill_ws(workspace, M, D);
  if (launch_act_quant(X, x_dtype, M, D, c.xq, c.ga, c.rs, s) != hipSuccess) return BITLINEAR_ERR_HIP;
  return hip_status(launch_gated_gemm(c.xq, c.ga, c.rs, M, D, F, w, o, s));
}

int bitlinear_gated_forward_quantized(const int8_t* Xq, const float* gamma_a, const int32_t* rowsum, int64_t M,
                                      int64_t D, int64_t F, const uint32_t* packed_gate, const float* gamma_gate,
                                      const uint32_t* packed_up, const float* gamma_up, int act, void* H, int h_dtype,
                                      void* G, void* U, int gu_dtype, void* stream) {
  const GatedWeights w = {packed_gate, gamma_gate, packed_up, gamma_up, act};
  const GatedOutputs o = {H, G, U, h_dtype, gu_dtype};
  if (!Xq || !gamma_a || !rowsum) return BITLINEAR_ERR_NULL;
  const int st = check_gated(M, D, F, w, o);
  if (st) return st;
  if (!aligned(Xq, 16) || !aligned(gamma_a, 4) || !aligned(rowsum, 4)) return BITLINEAR_ERR_ALIGN;
  const Range out[] = {array(H, h_dtype, M, F), array(G, gu_dtype, M, F), array(U, gu_dtype, M, F)};
  const Range in[] = {array(Xq, BITLINEAR_SAVED8, M, D),  floats(gamma_a, M),        {rowsum, 4 * static_cast<uint64_t>(M)},
                      packed_range(packed_gate, F, D),    packed_range(packed_up, F, D), floats(gamma_gate, 1),
                      floats(gamma_up, 1)};
  if (any_overlap(out, in)) return BITLINEAR_ERR_ARG;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (decode_fits(M, D, F)) return hip_status(launch_gated_decode(nullptr, 0, Xq, gamma_a, rowsum, M, D, F, w, o, s));
  return hip_status(launch_gated_gemm(Xq, gamma_a, rowsum, M, D, F, w, o, s));
}

size_t bitlinear_gated_ffn_workspace_bytes(int64_t M, int64_t D, int64_t F, int64_t D_out) {
  if (!size_args_ok(M) || !size_args_ok(D) || !size_args_ok(F) || !size_args_ok(D_out)) return 0;
  const size_t one = prefill_ws_bytes(M, D), two = prefill_ws_bytes(M, F);
  if (one == 0 || two == 0) return 0;
  const size_t all = size_add(align256(size_mul(size_mul(size_t(M), size_t(F)), 4)), one > two ? one : two);
  const size_t parts = prefill_parts_bytes(M, D_out, F);
  return parts ? size_add(all, parts) : all;
}

int bitlinear_gated_ffn_forward(const void* X, int x_dtype, int64_t M, int64_t D, int64_t F, int64_t D_out,
                                const uint32_t* packed_gate, const float* gamma_gate, const uint32_t* packed_up,
                                const float* gamma_up, int act, const uint32_t* packed_down, const float* gamma_down,
                                float* Y, float* hidden, int path, void* workspace, size_t workspace_bytes,
                                void* stream) {
  if (!X || !packed_gate || !gamma_gate || !packed_up || !gamma_up || !packed_down || !gamma_down || !Y)
    return BITLINEAR_ERR_NULL;
  int st = check_mnk(M, F, D);
  if (st) return st;
  st = check_mnk(M, D_out, F);
  if (st) return st;
  st = check_x(X, x_dtype);
  if (st) return st;
  if (!known_path(path) || !known_act(act)) return BITLINEAR_ERR_ARG;
  if (!aligned(packed_gate, 16) || !aligned(packed_up, 16) || !aligned(packed_down, 16) || !aligned(gamma_gate, 4) ||
      !aligned(gamma_up, 4) || !aligned(gamma_down, 4) || !aligned(Y, 4) || !aligned(hidden, 16))
    return BITLINEAR_ERR_ALIGN;
  const bool fits = decode_fits(M, D, F) && decode_fits(M, F, D_out);
  if (path == BITLINEAR_PATH_DECODE && !fits) return BITLINEAR_ERR_SHAPE;
  const bool decode = fits && path != BITLINEAR_PATH_PREFILL;
  const size_t hidden_bytes = hidden ? 0 : align256(static_cast<size_t>(M) * static_cast<size_t>(F) * 4);
  const size_t first = decode ? 0 : prefill_ws_bytes(M, D), second = prefill_ws_bytes(M, F);
  const size_t codes = first > second ? first : second, parts = decode ? 0 : prefill_parts_bytes(M, D_out, F);
  const size_t need = hidden_bytes + codes + parts;
  if (!workspace || workspace_bytes < need) return BITLINEAR_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return BITLINEAR_ERR_ALIGN;
  const Range out[] = {floats(Y, M * D_out), floats(hidden, M * F), {workspace, need}};
  const Range in[] = {array(X, x_dtype, M, D),          packed_range(packed_gate, F, D), packed_range(packed_up, F, D),
                      packed_range(packed_down, D_out, F), floats(gamma_gate, 1),        floats(gamma_up, 1),
                      floats(gamma_down, 1)};
  if (any_overlap(out, in)) return BITLINEAR_ERR_ARG;
  char* ws = static_cast<char*>(workspace);
  float* H = hidden ? hidden : reinterpret_cast<float*>(ws);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const GatedWeights w = {packed_gate, gamma_gate, packed_up, gamma_up, act};
  const GatedOutputs o = {H, nullptr, nullptr, BITLINEAR_F32, BITLINEAR_F32};
  const PrefillWs c = prefill_ws(ws + hidden_bytes, M, decode || F > D ? F : D);
  hipError_t e;
  if (decode) {
    e = launch_gated_decode(X, x_dtype, nullptr, nullptr, nullptr, M, D, F, w, o, s);
  } else {
    e = launch_act_quant(X, x_dtype, M, D, c.xq, c.ga, c.rs, s);
    if (e == hipSuccess) e = launch_gated_gemm(c.xq, c.ga, c.rs, M, D, F, w, o, s);
  }
  if (e == hipSuccess) e = launch_act_quant(H, BITLINEAR_F32, M, F, c.xq, c.ga, c.rs, s);
  if (e != hipSuccess) return BITLINEAR_ERR_HIP;
  if (decode)
    return hip_status(launch_decode_codes(c.xq, c.ga, c.rs, M, F, packed_down, D_out, gamma_down, Y, 1, s));
  if (parts)
    return hip_status(launch_prefill_parts(c.xq, c.ga, c.rs, M, F, packed_down, D_out, gamma_down, Y,
                                           reinterpret_cast<int32_t*>(ws + hidden_bytes + codes), s));
  return hip_status(launch_prefill_gemm(c.xq, c.ga, c.rs, M, F, packed_down, D_out, gamma_down, Y, nullptr, s));
}

int bitlinear_gated_backward(const void* dH, int dh_dtype, const void* G, const void* U, int gu_dtype, int64_t M,
                             int64_t F, int act, void* dG, void* dU, int d_dtype, void* stream) {
  if (!dH || !G || !U || !dG || !dU) return BITLINEAR_ERR_NULL;
  const int st = check_mk(M, F);
  if (st) return st;
  if (!plain_dtype(dh_dtype) || !plain_dtype(gu_dtype) || !plain_dtype(d_dtype)) return BITLINEAR_ERR_DTYPE;
  if (!known_act(act)) return BITLINEAR_ERR_ARG;
  if (!aligned_to(dH, dh_dtype) || !aligned_to(G, gu_dtype) || !aligned_to(U, gu_dtype) || !aligned_to(dG, d_dtype) ||
      !aligned_to(dU, d_dtype))
    return BITLINEAR_ERR_ALIGN;
  const Range out[] = {array(dG, d_dtype, M, F), array(dU, d_dtype, M, F)};
  const Range in[] = {array(dH, dh_dtype, M, F), array(G, gu_dtype, M, F), array(U, gu_dtype, M, F)};
  if (any_overlap(out, in)) return BITLINEAR_ERR_ARG;
  return hip_status(launch_gated_backward(dH, dh_dtype, G, U, gu_dtype, M, F, act, dG, dU, d_dtype,
                                          static_cast<hipStream_t>(stream)));
}

size_t bitlinear_gated_input_backward_workspace_bytes(int64_t M, int64_t F, int64_t D, int copies) {
  return gated_input_backward_ws_bytes(M, F, D, copies != 0);
}

int bitlinear_gated_input_backward(const uint16_t* dG, const uint16_t* dU, int64_t M, int64_t F, int64_t D,
                                   const uint32_t* packedT_gate, const float* gamma_gate,
                                   const uint32_t* packedT_up, const float* gamma_up, float* dX, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  if (!dG || !dU || !packedT_gate || !gamma_gate || !packedT_up || !gamma_up || !dX) return BITLINEAR_ERR_NULL;
  int st = check_mnk(M, F, D);
  if (st) return st;
  st = check_mnk(M, D, F);
  if (st) return st;
  // bf16 operands are addressed with 32-bit byte offsets
  if (M * padded_k(F) >= (int64_t(1) << 30)) return BITLINEAR_ERR_SHAPE;
  if (!aligned(dG, 2) || !aligned(dU, 2) || !aligned(packedT_gate, 16) || !aligned(packedT_up, 16) ||
      !aligned(gamma_gate, 4) || !aligned(gamma_up, 4) || !aligned(dX, 4))
    return BITLINEAR_ERR_ALIGN;
  const bool direct = F % 8 == 0 && aligned(dG, 16) && aligned(dU, 16);
  const size_t need = gated_input_backward_ws_bytes(M, F, D, !direct), sums = gated_dx_parts_bytes(M, F, D);
  if (need) {
    if (!workspace || workspace_bytes < need) return BITLINEAR_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return BITLINEAR_ERR_ALIGN;
  }
  const Range out[] = {floats(dX, M * D), {need ? workspace : nullptr, need}};
  const Range in[] = {array(dG, BITLINEAR_BF16, M, F),    array(dU, BITLINEAR_BF16, M, F),
                      packed_range(packedT_gate, D, F),   packed_range(packedT_up, D, F),
                      floats(gamma_gate, 1),              floats(gamma_up, 1)};
  if (any_overlap(out, in)) return BITLINEAR_ERR_ARG;
  void* copies = direct ? nullptr : static_cast<char*>(workspace) + sums;
  return hip_status(launch_gated_input_backward(dG, dU, M, F, D, packedT_gate, gamma_gate, packedT_up, gamma_up, dX,
                                                static_cast<float*>(workspace), copies,
                                                static_cast<hipStream_t>(stream)));
}

}  // extern "C"
