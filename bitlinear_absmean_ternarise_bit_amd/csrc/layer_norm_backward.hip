// Layer norm's backward pass (include/bitlinear_block.h).  With
// xhat = (x - mean) rstd and g = dy w:
//   dx = rstd (g - sum_k g / K - xhat sum_k (g xhat) / K)
//   dw = sum_m dy xhat,  db = sum_m dy
// in float32, from x as it was or from its 8-bit copy.
#include "block_device.hpp"

namespace bitlinear {

namespace {

// dx: one workgroup per row, rows gridDim.x apart; the row is read for the two
// sums and again for the output.
template <int XT, int DT, int OT>
__global__ __launch_bounds__(256) void ln_dx_rows_kernel(
    const char* __restrict__ dY, const char* __restrict__ X, const float* __restrict__ x_scales,
    const float* __restrict__ mean_in, const float* __restrict__ rstd_in, int64_t M, int K, int cpr,
    const float* __restrict__ weight, char* __restrict__ dX) {
  __shared__ float slots[2][8];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t G = cpr >> 3, Kp = int64_t(cpr) * 8;
  const float inv_k = 1.0f / static_cast<float>(K);
  int turn = 0;
  for (int64_t m = blockIdx.x; m < M; m += gridDim.x, turn ^= 1) {
    const char* row = X + (XT == kSaved8 ? m * Kp : m * K * kBytes<XT>);
    const char* drow = dY + m * K * kBytes<DT>;
    const float mean = mean_in[m], rstd = rstd_in[m];
    auto chunk = [&](int c, int n, float (&g)[8], float (&xh)[8]) {
      chunk_f32<XT>(load_chunk<XT>(row, x_scales + m * G, c, n), xh);
      chunk_f32<DT>(load_chunk<DT>(drow, nullptr, c, n), g);
      if (weight) {
        float w[8];
        chunk_f32<kF32>(load_chunk<kF32>(reinterpret_cast<const char*>(weight), nullptr, c, n), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] *= w[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) xh[e] = (xh[e] - mean) * rstd;
    };
    float s[2] = {0.0f, 0.0f};
    for (int c = tid; c < cpr; c += 256) {
      float g[8], xh[8];
      chunk(c, chunk_values(K, c), g, xh);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s[0] += g[e];
        s[1] = __fmaf_rn(g[e], xh[e], s[1]);
      }
    }
    team_sum<4>(s, slots[turn], wave, lane);
    const float c1 = s[0] * inv_k, c2 = s[1] * inv_k;
    for (int c = tid; c < cpr; c += 256) {
      const int n = chunk_values(K, c);
      float g[8], xh[8];
      chunk(c, n, g, xh);
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = rstd * (g[e] - __fmaf_rn(xh[e], c2, c1));
      store_chunk<OT>(dX + m * K * kBytes<OT>, c, n, g);
    }
  }
}

// Partial dw and db of slab blockIdx.y (rows slab, slab + slabs, ... in groups
// of 8): 32 chunks of columns by 8 rows at a time.
template <int XT, int DT>
__global__ __launch_bounds__(256) void ln_param_cols_kernel(
    const char* __restrict__ dY, const char* __restrict__ X, const float* __restrict__ x_scales,
    const float* __restrict__ mean_in, const float* __restrict__ rstd_in, int64_t M, int K, int cpr,
    float* __restrict__ partial) {
  __shared__ float sums[8][32 * 8];
  const int tid = threadIdx.x, cl = tid & 31, r = tid >> 5;
  const int c = blockIdx.x * 32 + cl;
  const int64_t G = cpr >> 3, Kp = int64_t(cpr) * 8;
  const int n = c < cpr ? chunk_values(K, c) : 0;
  float dw[8] = {}, db[8] = {};
  for (int64_t m = blockIdx.y * 8 + r; m < M; m += int64_t(gridDim.y) * 8) {
    float xh[8], d[8];
    chunk_f32<XT>(load_chunk<XT>(X + (XT == kSaved8 ? m * Kp : m * K * kBytes<XT>), x_scales + m * G, c, n), xh);
    chunk_f32<DT>(load_chunk<DT>(dY + m * K * kBytes<DT>, nullptr, c, n), d);
    const float mean = mean_in[m], rstd = rstd_in[m];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      db[e] += d[e];
      dw[e] = __fmaf_rn(d[e], (xh[e] - mean) * rstd, dw[e]);
    }
  }
  float* out = partial + static_cast<int64_t>(blockIdx.y) * 2 * K;
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[r][cl * 8 + e] = a ? db[e] : dw[e];
    __syncthreads();
    const int k = blockIdx.x * 256 + tid;
    if (k < K) {
      float t = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) t += sums[i][tid];
      out[a * K + k] = t;
    }
  }
}

// dw[k] = sum over the slabs of partial[slab][0][k], db likewise from [1].
__global__ __launch_bounds__(256) void ln_param_sum_kernel(const float* __restrict__ partial, int slabs, int K,
                                                           float* __restrict__ dw, float* __restrict__ db) {
  const int k = blockIdx.x * 256 + threadIdx.x;
  float* out = blockIdx.y ? db : dw;
  if (k >= K || !out) return;
  const float* p = partial + static_cast<int64_t>(blockIdx.y) * K + k;
  float t = 0.0f;
  for (int s = 0; s < slabs; ++s) t += p[static_cast<int64_t>(s) * 2 * K];
  out[k] = t;
}

struct Args {
  const void* dY;
  BlockIn X;
  const float *mean, *rstd;
  int64_t M, K;
  const float* weight;
  void* dX;
  float *dweight, *dbias;
  float* partial;
};

template <int XT, int DT>
hipError_t launch(const Args& a, int dx_dtype, hipStream_t stream) {
  const int cpr = static_cast<int>(padded_k(a.K) / 8), K = static_cast<int>(a.K);
  const char* dY = static_cast<const char*>(a.dY);
  const char* X = static_cast<const char*>(a.X.p);
  if (a.dX) {
    const unsigned blocks = static_cast<unsigned>(a.M < (1 << 20) ? a.M : (1 << 20));
    if (dx_dtype == kF32)
      ln_dx_rows_kernel<XT, DT, kF32><<<blocks, 256, 0, stream>>>(dY, X, a.X.scales, a.mean, a.rstd, a.M, K, cpr,
                                                                 a.weight, static_cast<char*>(a.dX));
    else
      ln_dx_rows_kernel<XT, DT, kBf16><<<blocks, 256, 0, stream>>>(dY, X, a.X.scales, a.mean, a.rstd, a.M, K, cpr,
                                                                  a.weight, static_cast<char*>(a.dX));
  }
  if (a.dweight || a.dbias) {
    const int slabs = static_cast<int>(ln_param_slabs(a.M, a.K));
    ln_param_cols_kernel<XT, DT><<<dim3((cpr + 31) / 32, slabs), 256, 0, stream>>>(dY, X, a.X.scales, a.mean, a.rstd,
                                                                                  a.M, K, cpr, a.partial);
    ln_param_sum_kernel<<<dim3((K + 255) / 256, 2), 256, 0, stream>>>(a.partial, slabs, K, a.dweight, a.dbias);
  }
  return hipGetLastError();
}

template <int DT>
hipError_t launch_from(const Args& a, int dx_dtype, hipStream_t s) {
  if (a.X.dtype == kF32) return launch<kF32, DT>(a, dx_dtype, s);
  if (a.X.dtype == kBf16) return launch<kBf16, DT>(a, dx_dtype, s);
  return launch<kSaved8, DT>(a, dx_dtype, s);
}

}  // namespace

hipError_t launch_layer_norm_backward(const void* dY, int dy_dtype, BlockIn X, const float* mean, const float* rstd,
                                      int64_t M, int64_t K, const float* weight, void* dX, int dx_dtype,
                                      float* dweight, float* dbias, void* workspace, hipStream_t stream) {
  const Args a = {dY, X, mean, rstd, M, K, weight, dX, dweight, dbias, static_cast<float*>(workspace)};
  return dy_dtype == kF32 ? launch_from<kF32>(a, dx_dtype, stream) : launch_from<kBf16>(a, dx_dtype, stream);
}

}  // namespace bitlinear
