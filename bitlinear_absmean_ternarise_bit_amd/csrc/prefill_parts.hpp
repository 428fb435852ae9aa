// The prefill product cut along K (prefill_parts.hip), for callers whose workspace
// has room for its parts.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sizes.hpp"

namespace bitlinear {

// Parts of Y [M, N] over K, 1 for none, and the time they save in ns.  With few tiles
// of 128 x 128 each CU that has one walks all of K, 0.65 us a stage of 128 whatever
// the tile, while the others idle; parts are INT32 sums, exact in any order, and cost
// a launch and their bytes.  64x4096 over 11008: 47 us in one part, 17 in 8; 43x251
// over 10432: 43 and 12; 777x1003 over 2701 17 either way, so little gain is left out.
// Up to 16 tokens stay in one part: the decode kernel takes them, but for rows too long
// for its LDS (a gated block of 4096 x 11008: 72 us for 6 to 16 tokens, 41 for 17, 24
// for 5).
struct PrefillParts {
  int parts;
  int64_t saved;
};
inline PrefillParts prefill_parts(int64_t M, int64_t N, int64_t K) {
  const int64_t many = int64_t(1) << 24;
  PrefillParts best = {1, 0};
  if (M <= 16 || M > many || N > many || K > (int64_t(1) << 20) || M * padded_k(K) >= (int64_t(1) << 31)) return best;
  const int64_t tiles = (M + 127) / 128 * ((N + 127) / 128), stages = (padded_k(K) + 127) / 128;
  for (int p = 2; p <= 16 && p * tiles <= 256 && 2 * p <= stages; ++p) {
    const int64_t saved = 650 * (stages - (stages + p - 1) / p) - 4500 - p * M * N / 600;
    if (saved > best.saved && saved > 2000) best = {p, saved};
  }
  return best;
}
inline size_t prefill_parts_bytes(int64_t M, int64_t N, int64_t K) {
  const int p = prefill_parts(M, N, K).parts;
  return p > 1 ? align256(size_mul(size_mul(size_t(M), size_t(N)), size_t(4) * p)) : 0;
}
// Y in the parts of prefill_parts, more than one; sums: prefill_parts_bytes
hipError_t launch_prefill_parts(const int8_t* Xq, const float* gamma_a, const int32_t* rowsum, int64_t M, int64_t K,
                                const uint32_t* packed, int64_t N, const float* gamma, float* Y, int32_t* sums,
                                hipStream_t stream);

}  // namespace bitlinear
