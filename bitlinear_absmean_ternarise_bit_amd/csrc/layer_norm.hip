// Layer norm's forward pass (include/bitlinear_block.h):
//   mean = sum x / K, var = sum (x - mean)^2 / K, rstd = 1 / sqrt(var + eps)
//   y = (x - mean) rstd w + b
// in float32, with the row's 8-bit copy written from the same read.
#include "block_device.hpp"

namespace bitlinear {

namespace {

// One workgroup per row, rows gridDim.x apart; the row is read from memory
// (the caches after the first time) for the mean, the variance and the output.
template <int XT, int YT, bool SAVE>
__global__ __launch_bounds__(256) void layer_norm_rows_kernel(
    const char* __restrict__ X, const float* __restrict__ x_scales, int64_t M, int K, int cpr,
    const float* __restrict__ weight, const float* __restrict__ bias, float eps, char* __restrict__ Y,
    float* __restrict__ mean_out, float* __restrict__ rstd_out, int8_t* __restrict__ codes,
    float* __restrict__ scales) {
  __shared__ float slots[2][4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t G = cpr >> 3, Kp = int64_t(cpr) * 8;
  for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
    const char* row = X + (XT == kSaved8 ? m * Kp : m * K * kBytes<XT>);
    const float* rs = x_scales + m * G;
    float sum[1] = {0.0f};
    for (int c = tid; c < cpr; c += 256) {
      float v[8];
      chunk_f32<XT>(load_chunk<XT>(row, rs, K, c, chunk_values(K, c)), v);
      if constexpr (SAVE) save_chunk(v, codes + m * Kp, scales + m * G, c);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[0] += v[e];
    }
    team_sum<4>(sum, slots[0], wave, lane);
    const float mean = sum[0] / static_cast<float>(K);
    float sq[1] = {0.0f};
    for (int c = tid; c < cpr; c += 256) {
      const int n = chunk_values(K, c);
      float v[8];
      chunk_f32<XT>(load_chunk<XT>(row, rs, K, c, n), v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = e < n ? v[e] - mean : 0.0f;
        sq[0] = __fmaf_rn(d, d, sq[0]);
      }
    }
    team_sum<4>(sq, slots[1], wave, lane);
    const float rstd = 1.0f / sqrtf(sq[0] / static_cast<float>(K) + eps);
    for (int c = tid; c < cpr; c += 256) {
      const int n = chunk_values(K, c);
      float v[8], w[8], b[8];
      chunk_f32<XT>(load_chunk<XT>(row, rs, K, c, n), v);
      if (weight) chunk_f32<kF32>(load_chunk<kF32>(reinterpret_cast<const char*>(weight), nullptr, K, c, n), w);
      if (bias) chunk_f32<kF32>(load_chunk<kF32>(reinterpret_cast<const char*>(bias), nullptr, K, c, n), b);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xh = (v[e] - mean) * rstd;
        v[e] = __fmaf_rn(xh, weight ? w[e] : 1.0f, bias ? b[e] : 0.0f);
      }
      store_chunk<YT>(Y + m * K * kBytes<YT>, c, n, v);
    }
    if (tid == 0 && mean_out) {
      mean_out[m] = mean;
      rstd_out[m] = rstd;
    }
  }
}

struct Args {
  BlockIn X;
  int64_t M, K;
  const float *weight, *bias;
  float eps;
  void* Y;
  float *mean, *rstd;
  int8_t* saved;
  float* saved_scales;
};

template <int XT, int YT, bool SAVE>
hipError_t launch(const Args& a, hipStream_t stream) {
  const int cpr = static_cast<int>(padded_k(a.K) / 8);
  const unsigned blocks = static_cast<unsigned>(a.M < (1 << 20) ? a.M : (1 << 20));
  layer_norm_rows_kernel<XT, YT, SAVE><<<blocks, 256, 0, stream>>>(
      static_cast<const char*>(a.X.p), a.X.scales, a.M, static_cast<int>(a.K), cpr, a.weight, a.bias, a.eps,
      static_cast<char*>(a.Y), a.mean, a.rstd, a.saved, a.saved_scales);
  return hipGetLastError();
}

template <int YT>
hipError_t launch_to(const Args& a, hipStream_t s) {
  if (a.X.dtype == kF32) return a.saved ? launch<kF32, YT, true>(a, s) : launch<kF32, YT, false>(a, s);
  if (a.X.dtype == kBf16) return a.saved ? launch<kBf16, YT, true>(a, s) : launch<kBf16, YT, false>(a, s);
  return launch<kSaved8, YT, false>(a, s);
}

}  // namespace

hipError_t launch_layer_norm(BlockIn X, int64_t M, int64_t K, const float* weight, const float* bias, float eps,
                             void* Y, int y_dtype, float* mean, float* rstd, int8_t* saved, float* saved_scales,
                             hipStream_t stream) {
  const Args a = {X, M, K, weight, bias, eps, Y, mean, rstd, saved, saved_scales};
  return y_dtype == kF32 ? launch_to<kF32>(a, stream) : launch_to<kBf16>(a, stream);
}

}  // namespace bitlinear
