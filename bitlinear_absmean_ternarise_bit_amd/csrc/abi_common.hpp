// Host-side checks shared by the C ABI's source files.  Plain C++ over the
// status codes; nothing here calls HIP.
#pragma once

#include <stdint.h>

#include "../../include/bitlinear_block.h"
#include "block_ops.hpp"
#include "kernels.hpp"

namespace bitlinear {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxK = int64_t(1) << 20;

inline int check_mnk(int64_t M, int64_t N, int64_t K) {
  if (M < 1 || N < 1 || K < 1) return BITLINEAR_ERR_SHAPE;
  if (K > kMaxK) return BITLINEAR_ERR_SHAPE;
  if (N > (int64_t(1) << 31) || M > (int64_t(1) << 31)) return BITLINEAR_ERR_SHAPE;
  if (static_cast<uint64_t>(N) * static_cast<uint64_t>(K) >= (uint64_t(1) << 32)) return BITLINEAR_ERR_SHAPE;
  // the kernels address a packed matrix (N * Kp / 4 bytes; the radix-3 form,
  // N * Kp3 / 5, is never larger) with 32-bit signed byte counts
  if (static_cast<uint64_t>(N) * static_cast<uint64_t>(padded_k(K)) / 4 >= (uint64_t(1) << 31))
    return BITLINEAR_ERR_SHAPE;
  if (static_cast<uint64_t>(M) * static_cast<uint64_t>(N) >= (uint64_t(1) << 40)) return BITLINEAR_ERR_SHAPE;
  if (static_cast<uint64_t>(M) * static_cast<uint64_t>(K) >= (uint64_t(1) << 40)) return BITLINEAR_ERR_SHAPE;
  return BITLINEAR_OK;
}

inline int check_x(const void* X, int x_dtype) {
  if (x_dtype != BITLINEAR_F32 && x_dtype != BITLINEAR_BF16) return BITLINEAR_ERR_DTYPE;
  if (!aligned(X, x_dtype == BITLINEAR_F32 ? 4 : 2)) return BITLINEAR_ERR_ALIGN;
  return BITLINEAR_OK;
}

// The decode kernel keeps all token codes in LDS and addresses a layer's
// outputs with 32-bit offsets.
inline bool decode_fits(int64_t M, int64_t K, int64_t N) {
  return M <= kDecodeMaxM && M * (padded_k(K) + 16) <= kDecodeMaxCodes && M * N < (int64_t(1) << 29);
}

// Parts of a prefill workspace.
struct PrefillWs {
  int8_t* xq;
  float* ga;
  int32_t* rs;
};

inline PrefillWs prefill_ws(void* ws, int64_t M, int64_t K) {
  char* p = static_cast<char*>(ws);
  PrefillWs w;
  w.xq = reinterpret_cast<int8_t*>(p);
  p += align256(static_cast<size_t>(M) * static_cast<size_t>(padded_k(K)));
  w.ga = reinterpret_cast<float*>(p);
  p += align256(static_cast<size_t>(M) * 4);
  w.rs = reinterpret_cast<int32_t*>(p);
  return w;
}

inline int hip_status(hipError_t e) { return e == hipSuccess ? BITLINEAR_OK : BITLINEAR_ERR_HIP; }

inline int check_mk(int64_t M, int64_t K) {
  if (M < 1 || K < 1 || K > (int64_t(1) << 20) || M > (int64_t(1) << 31)) return BITLINEAR_ERR_SHAPE;
  return static_cast<uint64_t>(M) * static_cast<uint64_t>(K) >= (uint64_t(1) << 40) ? BITLINEAR_ERR_SHAPE
                                                                                    : BITLINEAR_OK;
}

inline bool plain_dtype(int dt) { return dt == BITLINEAR_F32 || dt == BITLINEAR_BF16; }

// A memory range of an argument; NULL ranges overlap nothing.
struct Range {
  const void* p;
  uint64_t bytes;
};

inline bool overlap(const Range& a, const Range& b) {
  if (!a.p || !b.p) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y ? y - x < a.bytes : x - y < b.bytes;
}

// Whether an output overlaps an input or another output.
template <int NO, int NI>
inline bool any_overlap(const Range (&out)[NO], const Range (&in)[NI]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < NI; ++j)
      if (overlap(out[i], in[j])) return true;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return true;
  }
  return false;
}

// Sizes of arrays within the limits of check_mk (no overflow in 64 bits).
inline Range array(const void* p, int dt, int64_t M, int64_t K) {
  const uint64_t m = static_cast<uint64_t>(M);
  if (dt == BITLINEAR_SAVED8) return {p, m * static_cast<uint64_t>(padded_k(K))};
  return {p, m * static_cast<uint64_t>(K) * (dt == BITLINEAR_F32 ? 4 : 2)};
}
inline Range floats(const float* p, int64_t n) { return {p, static_cast<uint64_t>(n) * 4}; }
inline Range scale_range(const float* p, int64_t M, int64_t K) { return floats(p, M * saved_groups(K)); }

inline bool aligned_to(const void* p, int dt) {
  return aligned(p, dt == BITLINEAR_F32 ? 4 : dt == BITLINEAR_BF16 ? 2 : 16);
}

}  // namespace bitlinear
