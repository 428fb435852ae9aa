// Decode path: launches of the fused kernel (decode_kernel.hpp).
#include "decode_kernel.hpp"

namespace bitlinear {

namespace {

// Radix-3 is held to 128 registers (four waves per SIMD instead of three):
// more waves keep its vector ALU busier.  The 2-bit form is bound by memory
// and keeps the compiler's choice.
template <int FMT, int DT, bool VEC, int EPI, int SPLIT>
__global__ __launch_bounds__(kDecodeThreads) __attribute__((amdgpu_waves_per_eu(FMT == 3 ? 4 : 1))) void decode_kernel(
    const void* __restrict__ X, int M, int64_t K, int64_t Kp, int64_t units,
    const uint32_t* __restrict__ packed, int64_t N, const float* __restrict__ gamma,
    float* __restrict__ Y, int32_t* __restrict__ acc, int blocks_per_layer, int groups, int interleave,
    const float* __restrict__ ga_in, const int32_t* __restrict__ rs_in) {
  decode_body<FMT, DT, VEC, EPI, SPLIT>(X, M, K, Kp, units, packed, N, gamma, Y, acc, blocks_per_layer, groups,
                                        interleave, ga_in, rs_in, WholeGrid{});
}

template <int FMT, int DT, bool VEC>
hipError_t launch_v(const void* X, int64_t M, int64_t K, const uint32_t* packed, int64_t N,
                    const float* gamma, float* Y, int32_t* acc, int64_t L, bool relu2,
                    hipStream_t stream, const float* ga_in = nullptr, const int32_t* rs_in = nullptr) {
  const int64_t Kp = FMT == 2 ? padded_k(K) : r3_padded_k(K);
  const int64_t units = Kp / Format<FMT>::kPerUnit;
  const int groups = pick_groups(L, N);
  const int64_t rows = int64_t(kWaves) * kRowsPerWave * groups;
  const int64_t blocks16 = (N + kRowsPerWave - 1) / kRowsPerWave;  // 16-row blocks per layer
  int bpl = static_cast<int>((N + rows - 1) / rows);
  const bool split = L * bpl < kSplitBelow && blocks16 > bpl;
  if (split) bpl = static_cast<int>(blocks16);
  const unsigned blocks = static_cast<unsigned>(L * bpl);
  // 2-bit weights, one workgroup per layer: the waves take interleaved row
  // groups (1 x 2048 x 2048 layers in a batch: +1.0-1.5%, measured on four
  // boxes; where several workgroups share a layer the contiguous quarters
  // measured as fast or faster)
  const int ilv = FMT == 2 && !split && bpl == 1 && groups > 1;
  const int m = static_cast<int>(M);
  const bool with_acc = acc != nullptr && !relu2;
  const int64_t code_bytes = M * (Kp + 16);
  // after the codes: the waves' staged outputs, or (SPLIT) their partial sums
  const size_t lds = static_cast<size_t>(code_bytes) +
                     (split ? static_cast<size_t>(kDecodeThreads) * sizeof(v4i)
                            : static_cast<size_t>(kWaves) * stage_bytes(m, groups, with_acc, code_bytes));
  auto go = [&](auto split_tag) {
    constexpr int S = decltype(split_tag)::value;
    if constexpr (DT == 2) {
      decode_kernel<FMT, DT, VEC, kEpiY, S><<<blocks, kDecodeThreads, lds, stream>>>(
          X, m, K, Kp, units, packed, N, gamma, Y, nullptr, bpl, groups, ilv, ga_in, rs_in);
    } else {
      if (FMT == 2 && relu2)
        decode_kernel<FMT, DT, VEC, FMT == 2 ? kEpiRelu2 : kEpiY, S><<<blocks, kDecodeThreads, lds, stream>>>(
            X, m, K, Kp, units, packed, N, gamma, Y, nullptr, bpl, groups, ilv, nullptr, nullptr);
      else if (acc)
        decode_kernel<FMT, DT, VEC, kEpiAcc, S><<<blocks, kDecodeThreads, lds, stream>>>(
            X, m, K, Kp, units, packed, N, gamma, Y, acc, bpl, groups, ilv, nullptr, nullptr);
      else
        decode_kernel<FMT, DT, VEC, kEpiY, S><<<blocks, kDecodeThreads, lds, stream>>>(
            X, m, K, Kp, units, packed, N, gamma, Y, acc, bpl, groups, ilv, nullptr, nullptr);
    }
  };
  // split form: 2 loads per batch when a wave's quarter of a row is at most
  // eight load chunks, else 4 (measured on single layers: K = 2048 and 8192
  // are faster with 2, K = 11008 with 4)
  const int64_t chunks = (units + 3) / 4;
  if (split && (chunks + kWaves - 1) / kWaves <= 8) go(std::integral_constant<int, 2>());
  else if (split) go(std::integral_constant<int, 4>());
  else go(std::integral_constant<int, 0>());
  return hipGetLastError();
}

template <int FMT>
hipError_t launch_fmt(const void* X, int x_dtype, int64_t M, int64_t K, const uint32_t* packed,
                      int64_t N, const float* gamma, float* Y, int32_t* acc, int64_t L, bool relu2,
                      hipStream_t stream) {
  const int esize = x_dtype == 0 ? 4 : 2;
  const bool vec = (reinterpret_cast<uintptr_t>(X) % 16 == 0) && ((K * esize) % 16 == 0);
  if (x_dtype == 0)
    return vec ? launch_v<FMT, 0, true>(X, M, K, packed, N, gamma, Y, acc, L, relu2, stream)
               : launch_v<FMT, 0, false>(X, M, K, packed, N, gamma, Y, acc, L, relu2, stream);
  return vec ? launch_v<FMT, 1, true>(X, M, K, packed, N, gamma, Y, acc, L, relu2, stream)
             : launch_v<FMT, 1, false>(X, M, K, packed, N, gamma, Y, acc, L, relu2, stream);
}

}  // namespace

hipError_t launch_decode(const void* X, int x_dtype, int64_t M, int64_t K, const uint32_t* packed,
                         int64_t N, const float* gamma, float* Y, int32_t* acc, int64_t L,
                         hipStream_t stream, bool relu2) {
  return launch_fmt<2>(X, x_dtype, M, K, packed, N, gamma, Y, acc, L, relu2, stream);
}

hipError_t launch_decode_codes(const int8_t* Xq, const float* gamma_a, const int32_t* rowsum, int64_t M,
                              int64_t K, const uint32_t* packed, int64_t N, const float* gamma, float* Y,
                              int64_t L, hipStream_t stream) {
  return launch_v<2, 2, true>(Xq, M, K, packed, N, gamma, Y, nullptr, L, false, stream, gamma_a, rowsum);
}

hipError_t launch_decode_r3(const void* X, int x_dtype, int64_t M, int64_t K, const uint8_t* packed,
                            int64_t N, const float* gamma, float* Y, int32_t* acc, int64_t L,
                            hipStream_t stream) {
  return launch_fmt<3>(X, x_dtype, M, K, reinterpret_cast<const uint32_t*>(packed), N, gamma, Y,
                       acc, L, false, stream);
}

}  // namespace bitlinear
