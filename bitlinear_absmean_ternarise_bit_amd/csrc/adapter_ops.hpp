// Internal launch interface and sizes of the low-rank adapters and of dropout
// (include/bitlinear_adapters.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "block_ops.hpp"
#include "sizes.hpp"

namespace bitlinear {

constexpr int64_t kAdapterMaxR = 256, kAdapterMaxA = 65535;

// Adapters of M tokens: ids, and one of the two weight arrays [A, R, C].
struct Adapters {
  const int32_t* rows;
  const float* scales;
  int A, R, w_dtype;
};

inline int64_t padded_r(int64_t R) { return (R + 15) / 16 * 16; }

// The first product, T = X W^T over C columns: `blocks` blocks of 16 tokens to a
// workgroup (4 with 256 tokens or more, so that W is read once for 64), cut along
// the columns where those are few, into parts that are added by whoever reads T.
// `spread`: that many workgroups share the adapters of a group of tokens, each
// taking every spread-th one, where there are fewer than one to a CU without it
// (612x1280, 13 requests of 32 ranks: 17 us alone, 10 with 4).
struct ShrinkPlan {
  int blocks, spread, parts;
};
inline ShrinkPlan shrink_plan(int64_t M, int64_t C) {
  ShrinkPlan p = {M >= 256 ? 4 : 1, 1, 1};
  const int64_t groups = (M + 16 * p.blocks - 1) / (16 * p.blocks);
  if (p.blocks == 1) p.spread = static_cast<int>(M < 16 ? M : 16);
  int64_t parts = (p.blocks == 4 ? 256 : 512) / (groups * p.spread);
  const int64_t most = (C + 255) / 256;  // at least 256 columns, 64 to a wave
  if (parts > most) parts = most;
  if (parts > 16) parts = 16;
  p.parts = static_cast<int>(parts < 1 ? 1 : parts);
  if (p.blocks == 4) {
    const int64_t room = 256 / (groups * p.parts);
    p.spread = static_cast<int>(room < 1 ? 1 : room < 4 ? room : 4);
  }
  return p;
}

// The second product, Y += T W over C columns: 2 blocks of 16 tokens to a
// workgroup of 256 columns where that makes two workgroups for every CU, else 1.
inline int expand_blocks(int64_t M, int64_t C) {
  return (M + 31) / 32 * ((C + 255) / 256) >= 512 ? 2 : 1;
}
// How many workgroups share the adapters of such a group: as for the first product
// while the GPU is not full (each of them adds up T's parts again): 128x11008, one
// request to a group, 16 of them 19.6 us and 2 10.2; 200x5632, a request to a token,
// 16 of them 31 us, one 28 and 3 20.
inline int expand_spread(const ShrinkPlan& p, int64_t items) {
  const int64_t room = (p.blocks == 4 ? 512 : 1024) / items;
  return static_cast<int>(room < 1 ? 1 : room < p.spread ? room : p.spread);
}

// The gradients dW[a] = V^T X over C columns: workgroups of 64 columns, one
// adapter and up to 64 of its R rows, cut along the tokens into parts that a
// second launch adds.
struct GradPlan {
  int64_t tiles;
  int groups, parts;
};
inline GradPlan grad_plan(int64_t M, int64_t C, int64_t A, int64_t R) {
  GradPlan p;
  p.tiles = (C + 63) / 64;
  p.groups = static_cast<int>((R + 63) / 64);
  int64_t parts = 512 / (p.tiles * p.groups * A);
  const int64_t most = (M + 255) / 256;  // at least 64 tokens to a wave
  if (parts > most) parts = most;
  if (parts > 16) parts = 16;
  p.parts = static_cast<int>(parts < 1 ? 1 : parts);
  return p;
}

// Workspaces: T's parts [parts, M, padded_r(R)] float32 and its planes, bf16 [3, M,
// padded_r(R)]; for the backward those of V, V itself, and the parts of whichever
// gradient needs more.
inline size_t parts_ws_bytes(int64_t M, int64_t C, int64_t R) {
  const ShrinkPlan p = shrink_plan(M, C);
  return align256(size_mul(size_mul(size_t(p.parts) * 4, size_t(M)), size_t(padded_r(R))));
}
inline size_t shrink_ws_bytes(int64_t M, int64_t C, int64_t R) {
  return size_add(parts_ws_bytes(M, C, R), align256(size_mul(size_mul(size_t(M), 6), size_t(padded_r(R)))));
}
inline size_t grad_ws_bytes(int64_t M, int64_t C, int64_t A, int64_t R) {
  const GradPlan p = grad_plan(M, C, A, R);
  return p.parts == 1 ? 256 : align256(size_mul(size_mul(size_t(p.parts) * 4, size_t(A)), size_mul(size_t(R), size_t(C))));
}
inline size_t adapters_ws_bytes(int64_t M, int64_t K, int64_t R) {
  if (!size_args_ok(M) || !size_args_ok(K) || !size_args_ok(R) || R > kAdapterMaxR) return 0;
  return shrink_ws_bytes(M, K, R);
}
inline size_t adapters_backward_ws_bytes(int64_t M, int64_t K, int64_t N, int64_t A, int64_t R) {
  if (!size_args_ok(M) || !size_args_ok(K) || !size_args_ok(N) || !size_args_ok(R) || R > kAdapterMaxR || A < 1 ||
      A > kAdapterMaxA)
    return 0;
  const size_t v = align256(size_mul(size_mul(size_t(M), size_t(R)), 4));
  const size_t d = grad_ws_bytes(M, K, A, R), u = grad_ws_bytes(M, N, A, R);
  if (d == 0 || u == 0) return 0;
  return size_add(size_add(shrink_ws_bytes(M, N, R), v), d > u ? d : u);
}

// Tokens of a piece where a decode batch goes through its projection and adapters
// in two launches (adapted_decode.hip), 0 where it does not: more than 16 tokens,
// weights of so many rows that the decode forward streams them in another form,
// rows too long for its LDS.  Xq, ga, rs: as a prefill workspace holds them.
int64_t adapted_decode_piece(int64_t M, int64_t K, int64_t N);
hipError_t launch_adapted_decode(const void* X, int x_dtype, int64_t M, int64_t K, const uint32_t* packed, int64_t N,
                                 const float* gamma, float* Y, const Adapters& ad, const void* down, const void* up,
                                 float* parts, float* T, int64_t piece, int8_t* Xq, float* ga, int32_t* rs,
                                 hipStream_t stream);
// The first product and the tokens' codes in one launch (K >= 8).
hipError_t launch_adapted_first(const void* X, int x_dtype, int64_t M, int64_t K, const Adapters& ad, const void* down,
                                float* parts, int8_t* Xq, float* ga, int32_t* rs, hipStream_t stream);
// The prefill GEMM with the second product in its epilogue: where its 32-bit offsets
// hold and the tokens are so many that those of a tile's wave, 64, are likely of few
// adapters, which it takes one after another (16 ranks: 256x4096x4096 of 1 request 33
// us, as a pass of its own 38; a request for each of its tokens 89 and 75, for each of
// 200x2048x5632 65 and 38).  More ranks take longer there; what is saved is the pass
// over Y, so that has to be large (64 ranks: 2048x4096x4096 67 and 79, 512x4096x4096 44
// and 45, 6852x487x128 36 and 33; more than 64 ranks were not measured); planes:
// launch_join's.  An adapter's R rows of `up` are one buffer resource there: below 2^31
// bytes even of float32, or its size would not fit 32 bits and the offset that stands
// for "nowhere" would lie inside it.
inline bool adapted_gemm_takes(int64_t M, int64_t N, int64_t R) {
  return M >= 256 && N >= 8 && N <= (int64_t(1) << 24) && R * N < (int64_t(1) << 29) &&
         (R <= 16 || (R <= 64 && M * N >= (int64_t(1) << 22)));
}
hipError_t launch_adapted_gemm(const int8_t* Xq, const float* ga, const int32_t* rs, int64_t M, int64_t K,
                               const uint32_t* packed, int64_t N, const float* gamma, float* Y, const uint16_t* planes,
                               const Adapters& ad, const void* up, hipStream_t stream);
// parts of T = X W^T (rows without an adapter are not written)
hipError_t launch_shrink(const void* X, int x_dtype, int64_t M, int64_t C, const Adapters& ad, const void* W,
                         float* parts, hipStream_t stream);
// Y[m] (+)= scale T[m] W from T's parts (of a shrink over C0 columns); planes: room
// for T's; T: NULL, or where the whole T goes ([M, R], zeros for rows without an
// adapter)
hipError_t launch_expand(const float* parts, uint16_t* planes, int64_t M, int64_t C0, int64_t C, const Adapters& ad,
                         const void* W, float* Y, bool accumulate, float* T, hipStream_t stream);
// T and its scaled planes, bf16 [3, M, padded_r(R)]; each may be NULL
hipError_t launch_join(const float* parts, int64_t M, int64_t C0, const Adapters& ad, float* T, uint16_t* planes,
                       hipStream_t stream);
// dW[a] = scale[a] V^T X, V [M, R]; ws: grad_ws_bytes
hipError_t launch_adapter_grad(const float* V, const void* X, int x_dtype, int64_t M, int64_t C, const Adapters& ad,
                               float* dW, float* ws, hipStream_t stream);
hipError_t launch_dropout(const void* X, int x_dtype, const void* residual, int r_dtype, int64_t n, double p,
                          uint64_t seed, uint64_t offset, void* Y, int y_dtype, hipStream_t stream);

}  // namespace bitlinear
