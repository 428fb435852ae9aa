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

// The input's gradient, M x D over F: tiles of 256 x 128, 128 x 128 or 64 x 64 and F
// in parts of at least 4 stages of 64 columns, which another launch adds: whatever
// is the shortest by what was measured.  A stage of both products takes 1.05 us in a
// round of the largest tiles (one to a CU), 0.75 in one of the middle ones, and
// 0.3 + 0.18 for each of the smallest on a CU; the sum is a launch and its bytes.
// 55x238 over 10688: 157 us in one part, 16 in 41; 512x4096 over 11008: 215 with 128
// middle tiles, 131 in 2 parts of them, 100 with the largest in 4; 16x4096 over
// 11008: 49 with the smallest in 4 parts, 29 in 16, 35 in 32.
struct GatedDxPlan {
  int bm, bn, parts;
};
inline GatedDxPlan gated_dx_plan(int64_t M, int64_t F, int64_t D) {
  GatedDxPlan best = {256, 128, 1};
  const int64_t many = int64_t(1) << 24, stages = padded_k(F) / 64;
  if (M > many || D > many) return best;
  int64_t least = INT64_MAX;
  const GatedDxPlan kinds[] = {{256, 128, 512}, {128, 128, 512}, {64, 64, 1024}};  // (parts: the most workgroups)
  for (const GatedDxPlan& k : kinds) {
    const int64_t tiles = (M + k.bm - 1) / k.bm * ((D + k.bn - 1) / k.bn);
    for (int parts = 1; parts == 1 || (parts <= 64 && parts * 4 <= stages && parts * tiles <= k.parts); ++parts) {
      const int64_t rounds = (tiles * parts + 255) / 256, each = (stages + parts - 1) / parts;
      const int64_t per_stage = k.bm == 256 ? 1050 * rounds : k.bm == 128 ? 750 * rounds : 300 + 180 * rounds;
      const int64_t ns = each * per_stage + (parts > 1 ? 4500 + parts * M * D / 1000 : 0);
      if (ns < least) {
        least = ns;
        best = {k.bm, k.bn, parts};
      }
    }
  }
  return best;
}
// Padded copies of dG and dU, and the parts.
inline size_t gated_dx_parts_bytes(int64_t M, int64_t F, int64_t D) {
  const GatedDxPlan p = gated_dx_plan(M, F, D);
  return p.parts > 1 ? align256(size_mul(size_mul(size_t(M), size_t(D)), size_t(4) * p.parts)) : 0;
}
inline size_t gated_input_backward_ws_bytes(int64_t M, int64_t F, int64_t D, bool copies) {
  if (!size_args_ok(M) || !size_args_ok(F) || !size_args_ok(D)) return 0;
  const size_t parts = gated_dx_parts_bytes(M, F, D), two = copies ? size_mul(backward_ws_part(M, padded_k(F)), 2) : 0;
  return parts == 0 ? two : two == 0 ? (copies ? 0 : parts) : size_add(parts, two);
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
// copies: room for dG's and dU's, or NULL where the rows serve as they are
hipError_t launch_gated_input_backward(const uint16_t* dG, const uint16_t* dU, int64_t M, int64_t F, int64_t D,
                                       const uint32_t* packedT_gate, const float* gamma_gate,
                                       const uint32_t* packedT_up, const float* gamma_up, float* dX, float* parts,
                                       void* copies, hipStream_t stream);

}  // namespace bitlinear
