// Backward of the gated feed-forward block (include/bitlinear_gated.h):
// through act(G) * U, element by element, and the input's gradient, the sum of
// two products on the bf16 matrix cores.
#include "bf16_gemm.hpp"
#include "flat_device.hpp"
#include "gated_device.hpp"
#include "gated_ops.hpp"

namespace bitlinear {

namespace {

// dG and dU from dH, G and U, each read once, each written once: bound by memory
// (2048x11008, dH float32, the others bfloat16: 42 us, 6.4 TB/s).
template <int HT, int GT, int OT>
__global__ __launch_bounds__(256) void gated_backward_kernel(const char* dH, const char* G, const char* U, int64_t n,
                                                             int act, char* dG, char* dU) {
  const int64_t first = 8 * (static_cast<int64_t>(streaming_block()) * 256 + threadIdx.x);
  if (first >= n) return;
  const int m = static_cast<int>(min(n - first, int64_t(8)));
  float d[8], g[8], u[8];
  load_flat<HT>(dH + first * kBytes<HT>, m, d);
  load_flat<GT>(G + first * kBytes<GT>, m, g);
  load_flat<GT>(U + first * kBytes<GT>, m, u);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (act == kActRelu2) {
      const float r = g[i] <= 0.0f ? 0.0f : g[i];
      g[i] = __fmul_rn(d[i], __fmul_rn(u[i], 2.0f * r));
      u[i] = __fmul_rn(d[i], __fmul_rn(r, r));
    } else {
      const float s = sigmoid(g[i]);
      const float slope = __fmul_rn(s, __fmaf_rn(g[i], __fsub_rn(1.0f, s), 1.0f));
      const float a = __fmul_rn(g[i], s);
      g[i] = __fmul_rn(__fmul_rn(d[i], u[i]), slope);
      u[i] = __fmul_rn(d[i], a);
    }
  }
  store_chunk<OT>(dG + first * kBytes<OT>, 0, m, g);
  store_chunk<OT>(dU + first * kBytes<OT>, 0, m, u);
}

template <int HT, int GT, int OT>
hipError_t launch_as(const void* dH, const void* G, const void* U, int64_t n, int act, void* dG, void* dU,
                     hipStream_t stream) {
  for (int64_t i = 0; i < n; i += 8 * kFlatChunks) {
    const int64_t part = n - i < 8 * kFlatChunks ? n - i : 8 * kFlatChunks;
    gated_backward_kernel<HT, GT, OT><<<static_cast<unsigned>((part + 2047) / 2048), 256, 0, stream>>>(
        static_cast<const char*>(dH) + i * kBytes<HT>, static_cast<const char*>(G) + i * kBytes<GT>,
        static_cast<const char*>(U) + i * kBytes<GT>, part, act, static_cast<char*>(dG) + i * kBytes<OT>,
        static_cast<char*>(dU) + i * kBytes<OT>);
  }
  return hipGetLastError();
}

template <int HT, int GT>
hipError_t launch_to(const void* dH, const void* G, const void* U, int64_t n, int act, void* dG, void* dU, int d_dtype,
                     hipStream_t s) {
  return d_dtype == kF32 ? launch_as<HT, GT, kF32>(dH, G, U, n, act, dG, dU, s)
                         : launch_as<HT, GT, kBf16>(dH, G, U, n, act, dG, dU, s);
}

// C[p, q] = gamma A B^T + gamma2 A2 B2^T (bf16_gemm.hpp, EPI 2): 2048x4096 over 11008
// 310 to 330 us, 1.12 to 1.19 PFLOP/s, where the library's large bfloat16 product
// reaches 1.4; one launch for both saves writing and reading dX between.  Part blockIdx.y of
// the contraction, each with a C of its own
template <int BM, int BN, int WM, int WN, int BMODE>
__global__ __launch_bounds__(64 * WM * WN, 1) void bf16_two_products_kernel(
    const uint16_t* __restrict__ A, int64_t P, int64_t lda, const void* __restrict__ B, int64_t Q, int64_t Rp,
    float* __restrict__ C, const float* __restrict__ gamma, int bytes_a, int bytes_b, int tiles_p, int tiles_q,
    SecondProduct second) {
  const int stages = static_cast<int>(Rp / 64), part = blockIdx.y, parts = gridDim.y;
  second.first = static_cast<int>(static_cast<int64_t>(part) * stages / parts);
  second.count = static_cast<int>(static_cast<int64_t>(part + 1) * stages / parts) - second.first;
  bf16_gemm_nt_body<BM, BN, WM, WN, BMODE, 2>(A, P, lda, B, Q, Rp, C + part * P * Q, Q, gamma, nullptr, 0, bytes_a,
                                              bytes_b, tiles_p, tiles_q, second);
}

// dX = the sum of its parts, in order
__global__ __launch_bounds__(256) void sum_parts_kernel(const float* __restrict__ parts, int nparts, int64_t n,
                                                        float* __restrict__ dX) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    float v = parts[i];
#pragma unroll 8
    for (int s = 1; s < nparts; ++s) v += parts[s * n + i];
    dX[i] = v;
  }
}

}  // namespace

hipError_t launch_gated_backward(const void* dH, int dh_dtype, const void* G, const void* U, int gu_dtype, int64_t M,
                                 int64_t F, int act, void* dG, void* dU, int d_dtype, hipStream_t s) {
  const int64_t n = M * F;
  if (dh_dtype == kF32)
    return gu_dtype == kF32 ? launch_to<kF32, kF32>(dH, G, U, n, act, dG, dU, d_dtype, s)
                            : launch_to<kF32, kBf16>(dH, G, U, n, act, dG, dU, d_dtype, s);
  return gu_dtype == kF32 ? launch_to<kBf16, kF32>(dH, G, U, n, act, dG, dU, d_dtype, s)
                          : launch_to<kBf16, kBf16>(dH, G, U, n, act, dG, dU, d_dtype, s);
}

hipError_t launch_gated_input_backward(const uint16_t* dG, const uint16_t* dU, int64_t M, int64_t F, int64_t D,
                                       const uint32_t* packedT_gate, const float* gamma_gate,
                                       const uint32_t* packedT_up, const float* gamma_up, float* dX, float* parts,
                                       void* copies, hipStream_t stream) {
  const int64_t Fp = padded_k(F);
  int64_t lda = F;
  if (copies) {
    uint16_t* a = static_cast<uint16_t*>(copies);
    uint16_t* b = a + backward_ws_part(M, Fp) / 2;
    int64_t blocks = (M * (Fp / 8) + 255) / 256;
    if (blocks > 65536) blocks = 65536;
    pad_rows_bf16_kernel<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(dG, M, F, a, Fp);
    pad_rows_bf16_kernel<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(dU, M, F, b, Fp);
    dG = a;
    dU = b;
    lda = Fp;
  }
  const int bytes_a = static_cast<int>(M * lda * 2), bytes_b = static_cast<int>(D * (Fp / 4));
  const SecondProduct second = {dU, packedT_up, gamma_up, 0, 0};
  const GatedDxPlan plan = gated_dx_plan(M, F, D);
  auto go = [&](auto kernel, int bm, int bn, int threads) {
    const int tiles_p = static_cast<int>((M + bm - 1) / bm), tiles_q = static_cast<int>((D + bn - 1) / bn);
    kernel<<<dim3(static_cast<unsigned>(tiles_p * tiles_q), plan.parts), threads, 0, stream>>>(
        dG, M, lda, packedT_gate, D, Fp, plan.parts > 1 ? parts : dX, gamma_gate, bytes_a, bytes_b, tiles_p, tiles_q,
        second);
  };
  const bool whole = lda == Fp;
  if (plan.bm == 256)
    go(whole ? bf16_two_products_kernel<256, 128, 4, 2, 1> : bf16_two_products_kernel<256, 128, 4, 2, 2>, 256, 128, 512);
  else if (plan.bm == 128)
    go(whole ? bf16_two_products_kernel<128, 128, 2, 2, 1> : bf16_two_products_kernel<128, 128, 2, 2, 2>, 128, 128, 256);
  else
    go(whole ? bf16_two_products_kernel<64, 64, 1, 2, 1> : bf16_two_products_kernel<64, 64, 1, 2, 2>, 64, 64, 128);
  if (plan.parts > 1) {
    const int64_t blocks = (M * D + 255) / 256;
    sum_parts_kernel<<<static_cast<unsigned>(blocks < 65536 ? blocks : 65536), 256, 0, stream>>>(parts, plan.parts, M * D,
                                                                                             dX);
  }
  return hipGetLastError();
}

}  // namespace bitlinear
