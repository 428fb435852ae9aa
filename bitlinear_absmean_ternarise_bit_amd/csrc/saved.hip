// 8-bit saved activations (save, restore) and ReLU^2 with its backward pass
// (include/bitlinear_block.h): one read of each input, one write of each
// output, chunk by chunk.
#include "block_device.hpp"

namespace bitlinear {

namespace {

// What a pass over [M, K] does with a chunk.
enum Op { kSave, kRestore, kRelu2, kRelu2Backward };

constexpr uint32_t kRun = 256;  // consecutive workgroups of an XCD

// max(h, 0), and a NaN for a NaN
__device__ __forceinline__ float relu(float h) { return h <= 0.0f ? 0.0f : h; }

// One thread to a chunk; row m of the array is chunks m * cpr .. of the grid's
// index (cpr = Kp / 8, so the 8 lanes of a group are neighbours).
//   kSave:          in -> codes, scales
//   kRestore:       in (saved) -> out
//   kRelu2:         in -> out (and codes, scales when SAVE)
//   kRelu2Backward: dA, in -> out
// SHORT: rows of fewer than 8 values.
// Bound by HBM: 5.8 to 6.2 TB/s over 8192x28672 float32, 5.2 to 5.9 over 8192x8192
// bfloat16, 4.4 (restore) to 5.5 over 2048x11008 float32 (a copy reaches 4.9 to 5.1
// with 2 and 1 GiB).  Workgroups are dealt round-robin to the 8 XCDs; each XCD
// takes runs of kRun consecutive workgroups, 2 MiB of float32, so that it
// streams through memory: 8192x28672, save 203 -> 192 us, ReLU^2 325 -> 315, its
// backward 284 -> 274; nothing on arrays below 2048x11008; runs of 4, 1024 or
// 4096 are slower than none.  Two or four chunks to a thread, loaded first, are
// 1% to 35% slower there and slower still on small arrays.  total is 32 bits (at
// most 2^31 chunks to a launch) because a 64-bit division takes about as many
// instructions as the rest of a chunk (2048x4096 bf16: 3% to 8% slower).
template <int OP, int IT, int OT, int DT, bool SAVE, bool SHORT>
__global__ __launch_bounds__(256) void chunk_kernel(const char* __restrict__ in, const float* __restrict__ in_scales,
                                                    const char* __restrict__ dA, uint32_t total, int K, int cpr,
                                                    char* __restrict__ out, int8_t* __restrict__ codes,
                                                    float* __restrict__ scales) {
  const int64_t G = cpr >> 3, Kp = int64_t(cpr) * 8;
  const uint32_t b = blockIdx.x, in_turn = b % (8 * kRun);
  const uint32_t wg = b - in_turn + 8 * kRun <= gridDim.x ? b - in_turn + (in_turn & 7) * kRun + (in_turn >> 3) : b;
  const uint32_t i = wg * 256u + threadIdx.x;
  if (i >= total) return;  // total is a multiple of 8: whole groups leave
  const uint32_t row = i / static_cast<uint32_t>(cpr);
  const int c = static_cast<int>(i - row * static_cast<uint32_t>(cpr)), n = chunk_values(K, c);
  const int64_t m = row;
  float v[8];
  const char* from = in + (IT == kSaved8 ? m * Kp : m * K * kBytes<IT>);
  chunk_f32<IT>(load_chunk<IT, SHORT>(from, in_scales + m * G, K, c, n), v);
  if constexpr (SAVE) save_chunk(v, codes + m * Kp, scales + m * G, c);
  if constexpr (OP == kRelu2) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float r = relu(v[e]);
      v[e] = __fmul_rn(r, r);
    }
  } else if constexpr (OP == kRelu2Backward) {
    float d[8];
    chunk_f32<DT>(load_chunk<DT, SHORT>(dA + m * K * kBytes<DT>, nullptr, K, c, n), d);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __fmul_rn(d[e], 2.0f * relu(v[e]));
  }
  if constexpr (OP != kSave) store_chunk<OT>(out + m * K * kBytes<OT>, c, n, v);
}

template <int OP, int IT, int OT, int DT, bool SAVE>
hipError_t launch(BlockIn in, const void* dA, int64_t M, int64_t K, void* out, int8_t* codes, float* scales,
                  hipStream_t stream) {
  const int64_t cpr = padded_k(K) / 8, G = cpr / 8, Kp = cpr * 8;
  const char* src = static_cast<const char*>(in.p);
  const char* d = static_cast<const char*>(dA);
  char* dst = static_cast<char*>(out);
  const int64_t most = (int64_t(1) << 31) / cpr;  // rows of a launch
  for (int64_t m = 0; m < M; m += most) {
    const int64_t total = (M - m < most ? M - m : most) * cpr;
    // arrays that the operation does not have stay NULL
    auto kernel = K < 8 ? chunk_kernel<OP, IT, OT, DT, SAVE, true> : chunk_kernel<OP, IT, OT, DT, SAVE, false>;
    kernel<<<static_cast<unsigned>((total + 255) / 256), 256, 0, stream>>>(
        src + (IT == kSaved8 ? m * Kp : m * K * kBytes<IT>), in.scales ? in.scales + m * G : nullptr,
        d ? d + m * K * kBytes<DT> : nullptr, static_cast<uint32_t>(total), static_cast<int>(K),
        static_cast<int>(cpr), dst ? dst + m * K * kBytes<OT> : nullptr, codes ? codes + m * Kp : nullptr,
        scales ? scales + m * G : nullptr);
  }
  return hipGetLastError();
}

template <int OP, int OT, int DT>
hipError_t launch_any(BlockIn in, const void* dA, int64_t M, int64_t K, void* out, hipStream_t s) {
  if (in.dtype == kF32) return launch<OP, kF32, OT, DT, false>(in, dA, M, K, out, nullptr, nullptr, s);
  if (in.dtype == kBf16) return launch<OP, kBf16, OT, DT, false>(in, dA, M, K, out, nullptr, nullptr, s);
  return launch<OP, kSaved8, OT, DT, false>(in, dA, M, K, out, nullptr, nullptr, s);
}

template <int OT>
hipError_t launch_relu2_to(BlockIn H, int64_t M, int64_t K, void* A, int8_t* codes, float* scales, hipStream_t s) {
  if (codes && H.dtype == kF32) return launch<kRelu2, kF32, OT, kF32, true>(H, nullptr, M, K, A, codes, scales, s);
  if (codes) return launch<kRelu2, kBf16, OT, kF32, true>(H, nullptr, M, K, A, codes, scales, s);
  return launch_any<kRelu2, OT, kF32>(H, nullptr, M, K, A, s);
}

}  // namespace

hipError_t launch_save(const void* X, int x_dtype, int64_t M, int64_t K, int8_t* codes, float* scales,
                       hipStream_t s) {
  const BlockIn in = {X, nullptr, x_dtype};
  if (x_dtype == kF32) return launch<kSave, kF32, kF32, kF32, true>(in, nullptr, M, K, nullptr, codes, scales, s);
  return launch<kSave, kBf16, kF32, kF32, true>(in, nullptr, M, K, nullptr, codes, scales, s);
}

hipError_t launch_restore(BlockIn in, int64_t M, int64_t K, void* X, int x_dtype, hipStream_t s) {
  if (x_dtype == kF32) return launch<kRestore, kSaved8, kF32, kF32, false>(in, nullptr, M, K, X, nullptr, nullptr, s);
  return launch<kRestore, kSaved8, kBf16, kF32, false>(in, nullptr, M, K, X, nullptr, nullptr, s);
}

hipError_t launch_relu2(BlockIn H, int64_t M, int64_t K, void* A, int a_dtype, int8_t* saved, float* saved_scales,
                        hipStream_t s) {
  if (a_dtype == kF32) return launch_relu2_to<kF32>(H, M, K, A, saved, saved_scales, s);
  return launch_relu2_to<kBf16>(H, M, K, A, saved, saved_scales, s);
}

hipError_t launch_relu2_backward(const void* dA, int da_dtype, BlockIn H, int64_t M, int64_t K, void* dH,
                                 int dh_dtype, hipStream_t s) {
  if (da_dtype == kF32)
    return dh_dtype == kF32 ? launch_any<kRelu2Backward, kF32, kF32>(H, dA, M, K, dH, s)
                            : launch_any<kRelu2Backward, kBf16, kF32>(H, dA, M, K, dH, s);
  return dh_dtype == kF32 ? launch_any<kRelu2Backward, kF32, kBf16>(H, dA, M, K, dH, s)
                          : launch_any<kRelu2Backward, kBf16, kBf16>(H, dA, M, K, dH, s);
}

}  // namespace bitlinear
