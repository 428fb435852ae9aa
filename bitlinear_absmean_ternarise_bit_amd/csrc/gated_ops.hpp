// Internal launch interface of the gated feed-forward block
// (include/bitlinear_gated.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sizes.hpp"

namespace bitlinear {

// Both projections' weights and the activation between them.
struct GatedWeights {
  const uint32_t* gate;
  const float* gamma_gate;
  const uint32_t* up;
  const float* gamma_up;
  int act;
};
// Outputs [M, F]; G and U are NULL unless kept.
struct GatedOutputs {
  void* H;
  void* G;
  void* U;
  int h_dtype, gu_dtype;
};

// Padded copies of dG and dU.
inline size_t gated_input_backward_ws_bytes(int64_t M, int64_t F) {
  if (!size_args_ok(M) || !size_args_ok(F)) return 0;
  return size_mul(backward_ws_part(M, padded_k(F)), 2);
}

// decode path: X of x_dtype, or (Xq, ga, rs) codes with X NULL
hipError_t launch_gated_decode(const void* X, int x_dtype, const int8_t* Xq, const float* ga, const int32_t* rs,
                               int64_t M, int64_t D, int64_t F, const GatedWeights& w, const GatedOutputs& out,
                               hipStream_t stream);
// prefill path, from codes
hipError_t launch_gated_gemm(const int8_t* Xq, const float* ga, const int32_t* rs, int64_t M, int64_t D, int64_t F,
                             const GatedWeights& w, const GatedOutputs& out, hipStream_t stream);
hipError_t launch_gated_backward(const void* dH, int dh_dtype, const void* G, const void* U, int gu_dtype, int64_t M,
                                 int64_t F, int act, void* dG, void* dU, int d_dtype, hipStream_t stream);
// copies: the workspace, or NULL where the rows serve as they are
hipError_t launch_gated_input_backward(const uint16_t* dG, const uint16_t* dU, int64_t M, int64_t F, int64_t D,
                                       const uint32_t* packedT_gate, const float* gamma_gate,
                                       const uint32_t* packedT_up, const float* gamma_up, float* dX, void* copies,
                                       hipStream_t stream);

}  // namespace bitlinear
