// Element-wise passes over flat arrays, eight consecutive values to a thread.
#pragma once

#include "block_device.hpp"

namespace bitlinear {

// The workgroup's place in the array.  Workgroups are dealt round-robin to the
// 8 XCDs; each XCD takes runs of 256 consecutive ones, so that it streams
// through memory (saved.hip has what that measured).
__device__ __forceinline__ uint32_t streaming_block() {
  constexpr uint32_t kRun = 256;
  const uint32_t b = blockIdx.x, in_turn = b % (8 * kRun);
  return b - in_turn + 8 * kRun <= gridDim.x ? b - in_turn + (in_turn & 7) * kRun + (in_turn >> 3) : b;
}

constexpr int64_t kFlatChunks = int64_t(1) << 30;  // chunks of one launch

// n values (8, or fewer at the array's end) at p, aligned to their type only.
template <int DT>
__device__ __forceinline__ void load_flat(const char* p, int n, float (&v)[8]) {
  if (n == 8)
    chunk_f32<DT>(load_chunk<DT, false>(p, nullptr, 8, 0, 8), v);
  else
    chunk_f32<DT>(load_chunk<DT, true>(p, nullptr, n, 0, n), v);
}

}  // namespace bitlinear
