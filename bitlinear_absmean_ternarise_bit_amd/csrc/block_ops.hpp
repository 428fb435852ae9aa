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

// How layer norm's backward pass is cut up.  Rows of at most kLnBwdMaxChunks
// chunks of 8 (K <= 16384) go through one kernel: `waves` waves to a row,
// `chunks` chunks to a lane, `teams` rows at a time in a workgroup, `groups`
// workgroups.  K <= 8192: one chunk to a lane, as many waves as that takes, 16
// in a workgroup.  Longer: 8 waves with 3 or 4 chunks to a lane, alone in the
// workgroup, which leaves each lane 256 registers; with 7 (kLnLongChunks) a
// kernel of its own.
// About one workgroup to each of the 256 CUs: the parameter gradients leave as
// one partial row from each, and more of them would cost more than they hide.
// So few rows that one workgroup takes them in two turns are left to one: it
// writes the gradients itself, and the second launch (about as long as a turn)
// is saved.
// waves = 0 (rows that neither kernel takes): `groups` sets of rows for the
// column kernel, 32 chunks of columns to a workgroup, about 1024 workgroups.
struct LnBwdPlan {
  int waves, chunks, teams, groups;
};
constexpr int64_t kLnBwdMaxChunks = 2048;
// Rows of up to 28672, 8 waves of 7 chunks to a lane: dx, and with many rows of
// a multiple of 8 values dweight and dbias as well.  An eighth chunk does not
// fit: dweight and two chunks of dbias in LDS are 144 KB of a CU's 160 with 7.
// One pass saves a second read of x and dy but makes 256 partial rows, so it
// gains with rows and with the bytes of a value.  Against two passes, us, at
// 28672 and 16392 columns, M = 512, 768, 1024 and 2048 (types of x, dy, dx):
//   f32 f32 f32      61/67  80/94  98/126  164/228   43/41  53/60  64/76  108/139
//   8 bits f32 bf16  49/41  59/61  69/78   109/147   33/30  43/40  51/51   78/88
//   bf16 bf16 bf16   45/35  54/51  62/68    98/127   30/27  38/33  46/42   69/75
//   8 bits bf16 bf16 43/31  51/42  60/55    91/100   30/26  36/32  44/38   68/67
// They are even at M (bytes of x + bytes of dy) of 4000 to 6500.  The rule is one
// number of rows for all types: from 768 rows to that point it is up to 22%
// slower than two passes where dy is bfloat16, up to 8% from 8 bits with dy
// float32, and float32 rows below 768 miss up to 10%.
constexpr int kLnLongChunks = 7;
constexpr int64_t kLnLongMaxChunks = kLnLongChunks * 512, kLnLongMinRows = 768;

inline LnBwdPlan ln_bwd_plan(int64_t M, int64_t K, bool params) {
  const int64_t cpr = padded_k(K) / 8;
  LnBwdPlan p = {0, 1, 1, 1};
  if (params && cpr > kLnBwdMaxChunks && cpr <= kLnLongMaxChunks && K % 8 == 0 && M >= kLnLongMinRows)
    return {8, kLnLongChunks, 1, 256};
  if (cpr > kLnBwdMaxChunks || K < 8) {
    int64_t s = 1024 / ((cpr + 31) / 32);
    if (s > 256) s = 256;
    if (s > (M + 7) / 8) s = (M + 7) / 8;
    p.groups = static_cast<int>(s < 1 ? 1 : s);
    return p;
  }
  int64_t most = 1;  // teams of a workgroup
  if (cpr <= 1024) {
    p.waves = 1;
    while (64 * p.waves < cpr) p.waves *= 2;
    most = 16 / p.waves;
  } else {
    p.waves = 8;
    p.chunks = cpr <= 1536 ? 3 : 4;
  }
  const bool alone = params && M <= 2 * most;
  const int64_t teams = alone ? M : (M + 255) / 256;
  p.teams = static_cast<int>(teams < most ? teams : most);
  const int64_t groups = (M + p.teams - 1) / p.teams;
  p.groups = static_cast<int>(alone ? 1 : groups < 256 ? groups : 256);
  return p;
}

// One workgroup goes through all rows (rows of fewer than 8 values are one
// workgroup of the column kernel): it writes the gradients themselves.
inline bool ln_bwd_alone(const LnBwdPlan& p, int64_t K) { return p.groups == 1 && (p.waves > 0 || K < 8); }

// Partial rows of dweight and dbias.
inline size_t ln_bwd_workspace_bytes(int64_t M, int64_t K) {
  if (!size_args_ok(M) || !size_args_ok(K)) return 0;
  const LnBwdPlan p = ln_bwd_plan(M, K, true);
  if (ln_bwd_alone(p, K)) return 0;
  return align256(size_mul(size_t(p.groups), size_mul(size_t(K), 8)));
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
