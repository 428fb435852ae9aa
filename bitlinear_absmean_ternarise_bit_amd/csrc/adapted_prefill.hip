// Prefill through a projection and its adapters (include/bitlinear_adapters.h): the
// INT8-MFMA GEMM with the adapters' second product in its epilogue
// (prefill_gemm.hpp, EPI 4 to 7), for up to 64 ranks.  Y is written once; as a pass
// of its own the second product reads and writes it again, 180 MB for 2048 tokens
// of 11008 outputs (4096 inputs, 16 ranks: 106 us, the GEMM alone 88).  Part of the
// difference is scratch memory: Y's tile, T's planes, two sets of weights and a block's
// product exceed a lane's 256 registers with 256 x 256 tiles, by 59 with 16 ranks of
// bfloat16, 76 of float32, 136 and 150 with more ranks (128 x 256 tiles: none, none, 2
// and 11; 128 x 128 none).  The main loop has none of it.
#include <algorithm>

#include "prefill_gemm.hpp"

namespace bitlinear {

namespace {

constexpr int64_t kCUs = 256;

template <int BM, int BN, int WM, int WN, int EPI>
__global__ __launch_bounds__(64 * WM * WN, 1) void adapted_gemm_kernel(
    const int8_t* __restrict__ Xq, const float* __restrict__ gamma_a, const int32_t* __restrict__ rowsum, int64_t M,
    int64_t Kp, const uint32_t* __restrict__ packed, int64_t N, int64_t ldy, const float* __restrict__ gamma,
    float* __restrict__ Y, int tiles_m, int tiles_n, int bytes_a, int bytes_b, AdapterOut ao) {
  prefill_gemm_body<BM, BN, WM, WN, EPI>(Xq, gamma_a, rowsum, M, Kp, packed, N, ldy, gamma, Y, nullptr, tiles_m, tiles_n,
                                       bytes_a, bytes_b, GatedOut{}, ao);
}

// Columns [n0, n0 + N) of Y.
template <int BM, int BN, int WM, int WN>
hipError_t launch_tile(const int8_t* Xq, const float* ga, const int32_t* rs, int64_t M, int64_t Kp,
                       const uint32_t* packed, int64_t n0, int64_t N, int64_t ldy, const float* gamma, float* Y,
                       AdapterOut ao, int w_dtype, hipStream_t stream) {
  // buffer offsets are 32-bit: the tokens go in chunks of < 2^31 code bytes
  const int64_t chunk = ((int64_t(1) << 31) - 1) / Kp / BM * BM;
  ao.up += n0 * (w_dtype == kF32 ? 4 : 2);
  for (int64_t r0 = 0; r0 < M; r0 += chunk) {
    const int64_t Mc = std::min(M - r0, chunk);
    const int tiles_m = static_cast<int>((Mc + BM - 1) / BM), tiles_n = static_cast<int>((N + BN - 1) / BN);
    const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(int64_t(tiles_m) * tiles_n, kCUs));
    AdapterOut at = ao;
    at.planes += r0 * padded_r(ao.R);
    at.rows += r0;
    const bool f32 = w_dtype == kF32;
    auto kernel = ao.R <= 16
                      ? (f32 ? adapted_gemm_kernel<BM, BN, WM, WN, 5> : adapted_gemm_kernel<BM, BN, WM, WN, 4>)
                      : (f32 ? adapted_gemm_kernel<BM, BN, WM, WN, 7> : adapted_gemm_kernel<BM, BN, WM, WN, 6>);
    kernel<<<blocks, 64 * WM * WN, 0, stream>>>(
        Xq + r0 * Kp, ga + r0, rs + r0, Mc, Kp, packed + n0 * (Kp / 16), N, ldy, gamma, Y + r0 * ldy + n0, tiles_m,
        tiles_n, static_cast<int>(Mc * Kp), static_cast<int>(N * (Kp / 4)), at);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_adapted_gemm(const int8_t* Xq, const float* ga, const int32_t* rs, int64_t M, int64_t K,
                               const uint32_t* packed, int64_t N, const float* gamma, float* Y, const uint16_t* planes,
                               const Adapters& ad, const void* up, hipStream_t stream) {
  const int64_t Kp = padded_k(K);
  const AdapterOut ao = {planes, M * padded_r(ad.R), ad.rows, static_cast<const char*>(up), N, ad.A, ad.R};
  const int wt = ad.w_dtype;
  // Tiles of 256 tokens x 256 columns, 128 x 256 or 128 x 128 by weighed rounds, as
  // for the gated GEMM (gated.hip, where the weights and what they decide stand).
  auto tiles = [&](int64_t bm, int64_t bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); };
  auto rounds = [&](int64_t n) { return (n + kCUs - 1) / kCUs; };
  if (tiles(128, 128) <= kCUs)
    return launch_tile<128, 128, 2, 2>(Xq, ga, rs, M, Kp, packed, 0, N, N, gamma, Y, ao, wt, stream);
  const int64_t large = 7 * rounds(tiles(256, 256)), middle = 4 * rounds(tiles(128, 256));
  const int64_t whole = tiles(256, 256) / kCUs, per_column = (M + 255) / 256;
  const int64_t n = whole * kCUs / per_column * 256;
  if (n > 0 && n < N && (M + 127) / 128 * ((N - n + 255) / 256) <= kCUs && 7 * whole + 4 < std::min(large, middle)) {
    const hipError_t e = launch_tile<256, 256, 4, 2>(Xq, ga, rs, M, Kp, packed, 0, n, N, gamma, Y, ao, wt, stream);
    return e != hipSuccess ? e
                           : launch_tile<128, 256, 2, 4>(Xq, ga, rs, M, Kp, packed, n, N - n, N, gamma, Y, ao, wt, stream);
  }
  if (middle < large) return launch_tile<128, 256, 2, 4>(Xq, ga, rs, M, Kp, packed, 0, N, N, gamma, Y, ao, wt, stream);
  return launch_tile<256, 256, 4, 2>(Xq, ga, rs, M, Kp, packed, 0, N, N, gamma, Y, ao, wt, stream);
}

}  // namespace bitlinear
