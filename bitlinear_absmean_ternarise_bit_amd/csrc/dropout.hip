// Dropout from a counter-based generator (include/bitlinear_adapters.h), with the
// residual added in the same pass; its mask is formed again wherever it is
// needed.
#include "adapter_ops.hpp"
#include "flat_device.hpp"

namespace bitlinear {

namespace {

// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, 2011): ten rounds of two 32 x 32
// -> 64 bit products, each half exchanged and combined with the key, which steps
// by a constant of its own every round.
__device__ __forceinline__ void philox(uint64_t counter, uint64_t offset, uint64_t seed, uint32_t (&w)[4]) {
  uint32_t a = static_cast<uint32_t>(counter), b = static_cast<uint32_t>(counter >> 32);
  uint32_t c = static_cast<uint32_t>(offset), d = static_cast<uint32_t>(offset >> 32);
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p = static_cast<uint64_t>(0xD2511F53u) * a, q = static_cast<uint64_t>(0xCD9E8D57u) * c;
    a = static_cast<uint32_t>(q >> 32) ^ b ^ k0;
    b = static_cast<uint32_t>(q);
    c = static_cast<uint32_t>(p >> 32) ^ d ^ k1;
    d = static_cast<uint32_t>(p);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  w[0] = a;
  w[1] = b;
  w[2] = c;
  w[3] = d;
}

constexpr int kNone = 3;  // residual type: none

// Bound by memory: 2048x4096 bfloat16 with a residual 9.4 us (5.3 TB/s), 8192x8192
// float32 to bfloat16 66 (6.1), where a copy reaches 5; the generator's 40 wide
// products for 8 values go under it.
// first: the index of the launch's first value.  X, residual and Y may be one
// array: a thread reads its eight values before it writes them.
template <int XT, int RT, int YT>
__global__ __launch_bounds__(256) void dropout_kernel(const char* X, const char* residual, int64_t first, int64_t n,
                                                      uint64_t threshold, float scale, uint64_t seed, uint64_t offset,
                                                      char* Y) {
  const int64_t i = 8 * (static_cast<int64_t>(streaming_block()) * 256 + threadIdx.x);
  if (i >= n) return;
  const int m = static_cast<int>(min(n - i, int64_t(8)));
  float v[8], r[8];
  load_flat<XT>(X + i * kBytes<XT>, m, v);
  if constexpr (RT != kNone) load_flat<RT>(residual + i * kBytes<RT>, m, r);
  uint32_t w[2][4];
  philox(static_cast<uint64_t>(first + i) / 4, offset, seed, w[0]);
  philox(static_cast<uint64_t>(first + i) / 4 + 1, offset, seed, w[1]);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    v[e] = w[e >> 2][e & 3] >= threshold ? __fmul_rn(v[e], scale) : 0.0f;
    if constexpr (RT != kNone) v[e] = __fadd_rn(v[e], r[e]);
  }
  store_chunk<YT>(Y + i * kBytes<YT>, 0, m, v);
}

template <int XT, int RT, int YT>
hipError_t launch_as(const void* X, const void* residual, int64_t n, double p, uint64_t seed, uint64_t offset, void* Y,
                     hipStream_t stream) {
  const uint64_t threshold = static_cast<uint64_t>(p * 4294967296.0 + 0.5);
  const float scale = static_cast<float>(1.0 / (1.0 - p));
  for (int64_t i = 0; i < n; i += 8 * kFlatChunks) {
    const int64_t part = n - i < 8 * kFlatChunks ? n - i : 8 * kFlatChunks;
    dropout_kernel<XT, RT, YT><<<static_cast<unsigned>((part + 2047) / 2048), 256, 0, stream>>>(
        static_cast<const char*>(X) + i * kBytes<XT>,
        residual ? static_cast<const char*>(residual) + i * kBytes<RT> : nullptr, i, part, threshold, scale, seed,
        offset, static_cast<char*>(Y) + i * kBytes<YT>);
  }
  return hipGetLastError();
}

template <int XT, int RT>
hipError_t launch_to(const void* X, const void* residual, int64_t n, double p, uint64_t seed, uint64_t offset, void* Y,
                     int y_dtype, hipStream_t s) {
  return y_dtype == kF32 ? launch_as<XT, RT, kF32>(X, residual, n, p, seed, offset, Y, s)
                         : launch_as<XT, RT, kBf16>(X, residual, n, p, seed, offset, Y, s);
}

template <int XT>
hipError_t launch_with(const void* X, const void* residual, int r_dtype, int64_t n, double p, uint64_t seed,
                       uint64_t offset, void* Y, int y_dtype, hipStream_t s) {
  if (!residual) return launch_to<XT, kNone>(X, nullptr, n, p, seed, offset, Y, y_dtype, s);
  return r_dtype == kF32 ? launch_to<XT, kF32>(X, residual, n, p, seed, offset, Y, y_dtype, s)
                         : launch_to<XT, kBf16>(X, residual, n, p, seed, offset, Y, y_dtype, s);
}

}  // namespace

hipError_t launch_dropout(const void* X, int x_dtype, const void* residual, int r_dtype, int64_t n, double p,
                          uint64_t seed, uint64_t offset, void* Y, int y_dtype, hipStream_t s) {
  return x_dtype == kF32 ? launch_with<kF32>(X, residual, r_dtype, n, p, seed, offset, Y, y_dtype, s)
                         : launch_with<kBf16>(X, residual, r_dtype, n, p, seed, offset, Y, y_dtype, s);
}

}  // namespace bitlinear
