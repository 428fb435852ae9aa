// Internal launch interface and sizes of the operators around BitLinear
// (include/bitlinear_block.h): layer norm, ReLU^2, 8-bit saved activations.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sizes.hpp"

namespace bitlinear {

// dtypes of the launchers (the header's BITLINEAR_F32, _BF16, _SAVED8)
constexpr int kF32 = 0, kBf16 = 1, kSaved8 = 2;

inline int64_t saved_groups(int64_t K) { return padded_k(K) / 64; }

// An input array: data and, for kSaved8, its scales.
struct BlockIn {
  const void* p;
  const float* scales;
  int dtype;
};

// Sets of rows whose dweight / dbias sums are formed apart, for rows that the
// column kernel sums: 32 columns of 8 to a workgroup, about 1024 workgroups.
inline int64_t ln_param_slabs(int64_t M, int64_t K) {
  const int64_t col_blocks = (padded_k(K) / 8 + 31) / 32;
  int64_t s = 1024 / col_blocks;
  if (s > 256) s = 256;
  if (s > (M + 7) / 8) s = (M + 7) / 8;
  return s < 1 ? 1 : s;
}

inline size_t ln_bwd_workspace_bytes(int64_t M, int64_t K) {
  if (!size_args_ok(M) || !size_args_ok(K)) return 0;
  return align256(size_mul(size_t(ln_param_slabs(M, K)), size_mul(size_t(K), 8)));
}

hipError_t launch_save(const void* X, int x_dtype, int64_t M, int64_t K, int8_t* codes, float* scales,
                       hipStream_t stream);
hipError_t launch_restore(BlockIn codes, int64_t M, int64_t K, void* X, int x_dtype, hipStream_t stream);
hipError_t launch_relu2(BlockIn H, int64_t M, int64_t K, void* A, int a_dtype, int8_t* saved, float* saved_scales,
                        hipStream_t stream);
hipError_t launch_relu2_backward(const void* dA, int da_dtype, BlockIn H, int64_t M, int64_t K, void* dH,
                                 int dh_dtype, hipStream_t stream);
hipError_t launch_layer_norm(BlockIn X, int64_t M, int64_t K, const float* weight, const float* bias, float eps,
                             void* Y, int y_dtype, float* mean, float* rstd, int8_t* saved, float* saved_scales,
                             hipStream_t stream);
hipError_t launch_layer_norm_backward(const void* dY, int dy_dtype, BlockIn X, const float* mean, const float* rstd,
                                      int64_t M, int64_t K, const float* weight, void* dX, int dx_dtype,
                                      float* dweight, float* dbias, void* workspace, hipStream_t stream);

}  // namespace bitlinear
