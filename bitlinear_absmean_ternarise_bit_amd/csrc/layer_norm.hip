// Layer norm's forward pass (include/bitlinear_block.h):
//   mean = sum x / K, var = sum (x - mean)^2 / K, rstd = 1 / sqrt(var + eps)
//   y = (x - mean) rstd w + b
// in float32, with the row's 8-bit copy written from the same read.  Bound by
// the bytes of x and y (and the copy): layer_norm_kernel reads a row once and
// keeps it in registers; rows over kLnMaxChunks chunks, and rows of fewer than 8
// values, take the kernel below it, which reads them three times.
#include "block_device.hpp"

namespace bitlinear {

namespace {

// A float32 sum of K values leaves the mean some ulps off, and where a row's
// values lie far from 0 and close together rstd makes much of them: a constant
// row of 8000.1 has x - mean = 0.002 for 0 at K = 28672, and xhat = 0.5.  There
// the sum `diff` of d = x - first gives what the first mean lacks:
//   mean = first + diff / K,  shift = mean - first (exact: they are ulps apart)
//   var  = sum (d - shift)^2 / K = (sq - shift (2 diff - K shift)) / K
// with sq = sum d^2, both about the mean that is stored.  A first mean that is
// not finite, or a sum that overflows, stays as it is.
struct RowMean {
  float mean, shift, var;
};
__device__ __forceinline__ RowMean corrected_mean(float first, float diff, float sq, float K, float inv_k) {
  const float moved = __fmaf_rn(diff, inv_k, first);
  const float mean = fabsf(moved) < __builtin_inff() ? moved : first;
  const float shift = mean == first ? 0.0f : mean - first;
  const float left = shift == 0.0f ? sq : __fmaf_rn(-shift, __fmaf_rn(-K, shift, 2.0f * diff), sq);
  return {mean, shift, (left < 0.0f ? 0.0f : left) * inv_k};
}
// The rows that are corrected: those whose mean is 32 standard deviations or
// more.  Below, an ulp of the mean is at most 2^-18 of xhat.  Corrected always,
// with the sum beside that of the squares, 2048x4096 bfloat16 takes 9.5 us
// instead of 8.6 and 8192x8192 49.9 instead of 48.8.
__device__ __forceinline__ bool far_from_zero(float mean, float var) {
  return mean != 0.0f && var <= mean * (mean * 0x1p-10f);
}

constexpr int kLnMaxChunks = 4096;  // K <= 32768

// Waves that a SIMD holds at once: 64 or 128 registers to a lane.  As many
// waves as the row needs with one chunk to a lane and all eight resident beat
// half the waves with two chunks and six resident (8192 rows of 1024 to 8192,
// bfloat16: equal to 4% slower; float32 with the 8-bit copy, where the two
// chunks spill: 23% to 67% slower).
template <int NC>
constexpr int kLnWavesPerSimd = NC == 1 ? 8 : 4;

// A team of W waves holds a row, NC chunks of 8 columns to a lane, between the
// mean, the variance and the output.  W > 1: a team is a workgroup; W = 1: four
// teams to a workgroup, without barriers.  Rows are gridDim.x T apart, about as
// many teams as the card holds at once; each loads its next row before it works
// on the current one, and keeps weight and bias in registers (NC <= 2), so that
// nothing but that load is waited for; with NC = 4 the weight lies in LDS and the
// bias is read again (2048x28672, against both read again: float32 8% faster,
// bfloat16 12%; 5% slower where a team has one row).  8192x8192 bfloat16: 49 us,
// 5.4 TB/s, about 150 vector instructions for a wave's 512 columns, two thirds of
// what the SIMDs issue in that time; with the 8-bit copy 63 us, 5.4 TB/s, 200.
// WHOLE: K is a multiple of 8.
template <int XT, int YT, bool SAVE, int W, int NC, bool WHOLE>
__global__ __launch_bounds__(W > 1 ? 64 * W : 256, kLnWavesPerSimd<NC>) void layer_norm_kernel(
    const char* __restrict__ X, const float* __restrict__ x_scales, int64_t M, int K, int cpr,
    const float* __restrict__ weight, const float* __restrict__ bias, float eps, char* __restrict__ Y,
    float* __restrict__ mean_out, float* __restrict__ rstd_out, int8_t* __restrict__ codes,
    float* __restrict__ scales) {
  constexpr bool kHoldWeights = NC <= 2;
  constexpr int T = W > 1 ? 1 : 4;
  __shared__ float slots[3][W];
  __shared__ __align__(16) float lds_w[kHoldWeights ? 4 : 64 * W * NC * 8];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int team = W > 1 ? 0 : wave, wt = W > 1 ? wave : 0;
  const int64_t G = cpr >> 3, Kp = int64_t(cpr) * 8;
  const float inv_k = 1.0f / static_cast<float>(K);
  int c[NC], n[NC];
  float w[kHoldWeights ? NC : 1][8], b[kHoldWeights ? NC : 1][8];
  // chunk j of weight or bias (`none` where it is NULL)
  auto load_vector = [&](const float* from, float none, int j, float (&o)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = none;
    if (!from) return;
    Raw<kF32> rv = fetch_chunk<kF32, WHOLE>(reinterpret_cast<const char*>(from), nullptr, K, cpr, c[j]);
    if constexpr (!WHOLE) settle_chunk<kF32>(rv, n[j]);
    chunk_f32<kF32>(rv, o);
  };
  // this lane's place in the weight's LDS area: 8 floats in two halves, so that
  // a wave's 16-byte accesses are consecutive
  auto place = [&](int j, int half) { return ((j * 2 + half) * 64 * W + wt * 64 + lane) * 4; };
  Raw<XT> r[NC];
  auto load_row = [&](int64_t m) {
    m = m < M ? m : 0;  // behind the last row: any row, not used
    const char* row = X + (XT == kSaved8 ? m * Kp : m * K * kBytes<XT>);
#pragma unroll
    for (int j = 0; j < NC; ++j) r[j] = fetch_chunk<XT, WHOLE>(row, x_scales + m * G, K, cpr, c[j]);
  };
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    c[j] = wt * 64 + lane + j * 64 * W;
    n[j] = c[j] < cpr ? chunk_values(K, c[j]) : 0;
  }
  const int64_t stride = static_cast<int64_t>(gridDim.x) * T;
  int64_t m = static_cast<int64_t>(blockIdx.x) * T + team;
  if (m >= M) return;  // W = 1 only: a grid has no more workgroups than rows
  load_row(m);
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    if constexpr (kHoldWeights) {
      load_vector(weight, 1.0f, j, w[j]);
      load_vector(bias, 0.0f, j, b[j]);
    } else {
      load_vector(weight, 1.0f, j, w[0]);
#pragma unroll
      for (int e = 0; e < 8; ++e) lds_w[place(j, e >> 2) + (e & 3)] = w[0][e];  // read by this lane alone
    }
  }
#pragma unroll
  for (int j = 0; j < NC; ++j) arrive(r[j]);
  for (; m < M; m += stride) {
    float v[NC][8], sum[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      if constexpr (!WHOLE) settle_chunk<XT>(r[j], n[j]);
      chunk_f32<XT>(r[j], v[j]);
    }
    load_row(m + stride);
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[0] += v[j][e];
    team_sum<W>(sum, slots[0], wt, lane);
    float mean = sum[0] * inv_k;
    if constexpr (SAVE) {
      const __amdgpu_buffer_rsrc_t to_codes = row_resource(codes + m * Kp, static_cast<int>(Kp));
      const __amdgpu_buffer_rsrc_t to_scales = row_resource(scales + m * G, static_cast<int>(4 * G));
#pragma unroll
      for (int j = 0; j < NC; ++j) save_chunk(v[j], to_codes, to_scales, c[j]);
    }
    float sq[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NC; ++j) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[j][e] -= mean;
      if (n[j] < 8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] = (WHOLE ? n[j] > 0 : e < n[j]) ? v[j][e] : 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sq[0] = __fmaf_rn(v[j][e], v[j][e], sq[0]);
    }
    team_sum<W>(sq, slots[1], wt, lane);
    float var = sq[0] * inv_k;
    if (far_from_zero(mean, var)) {  // the same for the whole team
      float diff[1] = {0.0f};
#pragma unroll
      for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) diff[0] += v[j][e];
      team_sum<W>(diff, slots[2], wt, lane);
      const RowMean row = corrected_mean(mean, diff[0], sq[0], static_cast<float>(K), inv_k);
#pragma unroll
      for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] -= row.shift;
      mean = row.mean;
      var = row.var;
    }
    const float rstd = 1.0f / sqrtf(var + eps);
    const __amdgpu_buffer_rsrc_t to_y = row_resource(Y + m * K * kBytes<YT>, K * kBytes<YT>);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int held = kHoldWeights ? j : 0;
      if constexpr (!kHoldWeights) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[0][e] = lds_w[place(j, e >> 2) + (e & 3)];
        load_vector(bias, 0.0f, j, b[0]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) v[j][e] = __fmaf_rn(v[j][e] * rstd, w[held][e], b[held][e]);
      put_chunk<YT, WHOLE>(to_y, c[j], n[j], v[j]);
    }
    // by the team's first lane: the others fall behind 4 bytes
    const int stats = mean_out && wt == 0 ? 4 : 0;
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(mean), row_resource(mean_out + m, stats), 4u * lane, 0, 0);
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(rstd), row_resource(rstd_out + m, stats), 4u * lane, 0, 0);
  }
}

// Long rows, and rows of fewer than 8 values (SHORT): one workgroup per row,
// rows gridDim.x apart; the row is read from memory (the caches after the first
// time) for the mean, the variance and the output.  That costs: 2048x53248
// bfloat16 179 us, 2.4 TB/s of x and y once (2048x32768, held in registers, 56 us;
// 2048x32776 105).
template <int XT, int YT, bool SAVE, bool SHORT>
__global__ __launch_bounds__(256) void layer_norm_rows_kernel(
    const char* __restrict__ X, const float* __restrict__ x_scales, int64_t M, int K, int cpr,
    const float* __restrict__ weight, const float* __restrict__ bias, float eps, char* __restrict__ Y,
    float* __restrict__ mean_out, float* __restrict__ rstd_out, int8_t* __restrict__ codes,
    float* __restrict__ scales) {
  __shared__ float slots[3][4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t G = cpr >> 3, Kp = int64_t(cpr) * 8;
  const float inv_k = 1.0f / static_cast<float>(K);
  for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
    const char* row = X + (XT == kSaved8 ? m * Kp : m * K * kBytes<XT>);
    const float* rs = x_scales + m * G;
    float sum[1] = {0.0f};
    for (int c = tid; c < cpr; c += 256) {
      float v[8];
      chunk_f32<XT>(load_chunk<XT, SHORT>(row, rs, K, c, chunk_values(K, c)), v);
      if constexpr (SAVE) save_chunk(v, codes + m * Kp, scales + m * G, c);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[0] += v[e];
    }
    team_sum<4>(sum, slots[0], wave, lane);
    float mean = sum[0] * inv_k;
    float sq[1] = {0.0f};
    for (int c = tid; c < cpr; c += 256) {
      const int n = chunk_values(K, c);
      float v[8];
      chunk_f32<XT>(load_chunk<XT, SHORT>(row, rs, K, c, n), v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = e < n ? v[e] - mean : 0.0f;
        sq[0] = __fmaf_rn(d, d, sq[0]);
      }
    }
    team_sum<4>(sq, slots[1], wave, lane);
    float var = sq[0] * inv_k;
    if (far_from_zero(mean, var)) {  // the same for the whole workgroup
      float diff[1] = {0.0f};
      for (int c = tid; c < cpr; c += 256) {
        const int n = chunk_values(K, c);
        float v[8];
        chunk_f32<XT>(load_chunk<XT, SHORT>(row, rs, K, c, n), v);
#pragma unroll
        for (int e = 0; e < 8; ++e) diff[0] += e < n ? v[e] - mean : 0.0f;
      }
      team_sum<4>(diff, slots[2], wave, lane);
      const RowMean of = corrected_mean(mean, diff[0], sq[0], static_cast<float>(K), inv_k);
      mean = of.mean;
      var = of.var;
    }
    const float rstd = 1.0f / sqrtf(var + eps);
    for (int c = tid; c < cpr; c += 256) {
      const int n = chunk_values(K, c);
      float v[8], w[8], b[8];
      chunk_f32<XT>(load_chunk<XT, SHORT>(row, rs, K, c, n), v);
      if (weight) chunk_f32<kF32>(load_chunk<kF32, SHORT>(reinterpret_cast<const char*>(weight), nullptr, K, c, n), w);
      if (bias) chunk_f32<kF32>(load_chunk<kF32, SHORT>(reinterpret_cast<const char*>(bias), nullptr, K, c, n), b);
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

template <int XT, int YT, bool SAVE, int W, int NC>
void launch_held(const Args& a, hipStream_t stream) {
  constexpr int64_t T = W > 1 ? 1 : 4;  // rows at a time of a workgroup
  constexpr int64_t most = 256 * (4 * kLnWavesPerSimd<NC> / (W > 1 ? W : 4));  // workgroups that 256 CUs hold
  const int64_t wgs = (a.M + T - 1) / T, turns = (wgs + most - 1) / most;
  const int64_t blocks = (wgs + turns - 1) / turns;  // as many turns for each
  auto kernel = a.K % 8 == 0 ? layer_norm_kernel<XT, YT, SAVE, W, NC, true>
                             : layer_norm_kernel<XT, YT, SAVE, W, NC, false>;
  kernel<<<static_cast<unsigned>(blocks), W > 1 ? 64 * W : 256, 0, stream>>>(
      static_cast<const char*>(a.X.p), a.X.scales, a.M, static_cast<int>(a.K), static_cast<int>(padded_k(a.K) / 8),
      a.weight, a.bias, a.eps, static_cast<char*>(a.Y), a.mean, a.rstd, a.saved, a.saved_scales);
}

template <int XT, int YT, bool SAVE>
hipError_t launch(const Args& a, hipStream_t stream) {
  const int cpr = static_cast<int>(padded_k(a.K) / 8);
  if (a.K < 8 || cpr > kLnMaxChunks) {
    const unsigned blocks = static_cast<unsigned>(a.M < (1 << 20) ? a.M : (1 << 20));
    auto kernel = a.K < 8 ? layer_norm_rows_kernel<XT, YT, SAVE, true> : layer_norm_rows_kernel<XT, YT, SAVE, false>;
    kernel<<<blocks, 256, 0, stream>>>(static_cast<const char*>(a.X.p), a.X.scales, a.M, static_cast<int>(a.K), cpr,
                                       a.weight, a.bias, a.eps, static_cast<char*>(a.Y), a.mean, a.rstd, a.saved,
                                       a.saved_scales);
  } else if (cpr <= 64) {
    launch_held<XT, YT, SAVE, 1, 1>(a, stream);
  } else if (cpr <= 128) {
    launch_held<XT, YT, SAVE, 2, 1>(a, stream);
  } else if (cpr <= 256) {
    launch_held<XT, YT, SAVE, 4, 1>(a, stream);
  } else if (cpr <= 512) {
    launch_held<XT, YT, SAVE, 8, 1>(a, stream);
  } else if (cpr <= 1024) {
    launch_held<XT, YT, SAVE, 16, 1>(a, stream);
  } else if (cpr <= 2048) {
    launch_held<XT, YT, SAVE, 16, 2>(a, stream);
  } else {
    launch_held<XT, YT, SAVE, 16, 4>(a, stream);
  }
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
