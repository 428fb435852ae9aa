// The prefill product of few tiles, cut along K: the INT8-MFMA GEMM writes the INT32
// sums of each part (prefill_gemm.hpp, EPI 8) and a second launch adds and rescales
// them.  The sums are exact, so Y has the bits of the product in one piece.
#include "prefill_parts.hpp"
#include "prefill_gemm.hpp"

namespace bitlinear {

namespace {

__global__ __launch_bounds__(256, 1) void prefill_parts_kernel(const int8_t* __restrict__ Xq,
                                                               const float* __restrict__ gamma_a,
                                                               const int32_t* __restrict__ rowsum, int64_t M, int64_t Kp,
                                                               const uint32_t* __restrict__ packed, int64_t N,
                                                               const float* __restrict__ gamma, int32_t* __restrict__ sums,
                                                               int tiles_m, int tiles_n, int bytes_a, int bytes_b) {
  const int stages = static_cast<int>((Kp + 127) / 128), part = blockIdx.y, parts = gridDim.y;
  const int first = part * stages / parts;
  prefill_gemm_body<128, 128, 2, 2, 8>(Xq, gamma_a, rowsum, M, Kp, packed, N, N, gamma, nullptr, sums + part * M * N,
                                       tiles_m, tiles_n, bytes_a, bytes_b, GatedOut{}, AdapterOut{}, first,
                                       (part + 1) * stages / parts - first);
}

__global__ __launch_bounds__(256) void join_parts_kernel(const int32_t* __restrict__ sums, int nparts, int64_t M, int64_t N,
                                                         const float* __restrict__ gamma_a,
                                                         const int32_t* __restrict__ rowsum,
                                                         const float* __restrict__ gamma, float* __restrict__ Y) {
  const int64_t n = M * N, i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n) return;
  const int64_t m = i / N;
  int v = sums[i];
#pragma unroll 4
  for (int s = 1; s < nparts; ++s) v += sums[s * n + i];
  Y[i] = __fmul_rn(static_cast<float>(v - rowsum[m]), __fdiv_rn(__fmul_rn(gamma[0], gamma_a[m]), 127.0f));
}

}  // namespace

hipError_t launch_prefill_parts(const int8_t* Xq, const float* gamma_a, const int32_t* rowsum, int64_t M, int64_t K,
                                const uint32_t* packed, int64_t N, const float* gamma, float* Y, int32_t* sums,
                                hipStream_t stream) {
  const int64_t Kp = padded_k(K);
  const int parts = prefill_parts(M, N, K).parts;
  const int tiles_m = static_cast<int>((M + 127) / 128), tiles_n = static_cast<int>((N + 127) / 128);
  prefill_parts_kernel<<<dim3(static_cast<unsigned>(tiles_m * tiles_n), parts), 256, 0, stream>>>(
      Xq, gamma_a, rowsum, M, Kp, packed, N, gamma, sums, tiles_m, tiles_n, static_cast<int>(M * Kp),
      static_cast<int>(N * (Kp / 4)));
  join_parts_kernel<<<static_cast<unsigned>((M * N + 255) / 256), 256, 0, stream>>>(sums, parts, M, N, gamma_a, rowsum,
                                                                                  gamma, Y);
  return hipGetLastError();
}

}  // namespace bitlinear
