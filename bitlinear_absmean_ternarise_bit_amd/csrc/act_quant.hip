// Standalone per-token AbsMax INT8 quantiser (the prefill path's first
// kernel): one wavefront per token, four tokens per 256-thread workgroup.
#include "block_device.hpp"
#include "kernels.hpp"
#include "quant_act.hpp"

namespace bitlinear {

namespace {

// RC: 16-byte chunks per lane kept in registers (rows of up to RC * 64 chunks
// are read once)
template <int DT, bool VEC, int RC>
__global__ __launch_bounds__(256) void act_quant_kernel(const void* __restrict__ X, int64_t M, int64_t K,
                                                        int64_t Kp, int8_t* __restrict__ Xq,
                                                        float* __restrict__ gamma_a,
                                                        int32_t* __restrict__ rowsum) {
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t m = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (m >= M) return;  // whole wave leaves together
  constexpr int esize = DT == 0 ? 4 : 2;
  const char* row = static_cast<const char*>(X) + m * K * esize;
  float ga;
  int rs;
  quantize_row_wave<DT, VEC, RC>(row, K, Kp, lane, Xq + m * Kp, ga, rs);
  if (lane == 0) {
    gamma_a[m] = ga;
    rowsum[m] = rs;
  }
}

// Rows too long for one wave's registers: one 256-thread workgroup per
// token, RC 16-byte chunks per thread kept in registers between the max and
// the codes, so X is read once (the wave-per-token kernel would read such a
// row twice, and with many rows in flight the second read misses L2).
template <int DT, int RC>
__global__ __launch_bounds__(256) void act_quant_row_kernel(const void* __restrict__ X, int64_t K, int64_t Kp,
                                                            int8_t* __restrict__ Xq, float* __restrict__ gamma_a,
                                                            int32_t* __restrict__ rowsum) {
  constexpr int P = ActTraits<DT>::kPerChunk;
  constexpr int esize = DT == 0 ? 4 : 2;
  __shared__ float s_max[4];
  __shared__ int s_sum[4];
  const int tid = threadIdx.x;
  const int lane = tid & (kWave - 1), wave = tid >> 6;
  const int64_t m = blockIdx.x;
  const uint4* r4 = reinterpret_cast<const uint4*>(static_cast<const char*>(X) + m * K * esize);
  const int64_t nc = K / P;
  uint4 v[RC];
#pragma unroll
  for (int u = 0; u < RC; ++u) {
    const int64_t c = tid + u * 256;
    v[u] = r4[c < nc ? c : nc - 1];
  }
  float mx = 0.0f;
#pragma unroll
  for (int u = 0; u < RC; ++u) {
    float f[P];
    chunk_to_f32<DT>(v[u], f);
    float mu = 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i) mu = fmaxf(mu, fabsf(f[i]));
    mx = (tid + u * 256 < nc) ? fmaxf(mx, mu) : mx;
  }
  mx = wave_max(mx);
  if (lane == 0) s_max[wave] = mx;
  __syncthreads();
  mx = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
  const float s = __fdiv_rn(127.0f, __fadd_rn(mx, kEps));
  int8_t* dst = Xq + m * Kp;
  int sum = 0;
#pragma unroll
  for (int u = 0; u < RC; ++u) {
    const int64_t c = tid + u * 256;
    if (c < nc) sum += quantize_chunk<DT>(v[u], s, dst + c * P);
  }
  for (int64_t k = K + tid; k < Kp; k += 256) dst[k] = 0;
  sum = wave_sum(sum);
  if (lane == 0) s_sum[wave] = sum;
  __syncthreads();
  if (tid == 0) {
    gamma_a[m] = mx;
    rowsum[m] = s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3];
  }
}

// Rows at any address, of any length from 8 up (longer ones are given to it): one lane to a chunk of 8
// values (block_device.hpp), RC of them in its registers, W waves to a row, so X
// is read once with 16-byte loads.  The chunk that the row's end cuts is moved
// into place and filled with zeros, which are the codes of the padding.  Value by
// value, 2048 rows of 4095 bfloat16 took 38 us; this takes 8.
template <int DT, int RC, int W>
__global__ __launch_bounds__(256) void act_quant_any_kernel(const char* __restrict__ X, int64_t M, int K, int Kp,
                                                            int8_t* __restrict__ Xq, float* __restrict__ gamma_a,
                                                            int32_t* __restrict__ rowsum) {
  __shared__ float s_max[4];
  __shared__ int s_sum[4];
  const int lane = threadIdx.x & (kWave - 1), wave = wave_id();
  const int first = W == 1 ? lane : static_cast<int>(threadIdx.x);
  const int64_t m = W == 1 ? static_cast<int64_t>(blockIdx.x) * 4 + wave : blockIdx.x;
  if (m >= M) return;  // (W = 1) whole waves leave together
  const char* row = X + m * K * kBytes<DT>;
  float v[RC][8];
  float mx = 0.0f;
#pragma unroll
  for (int u = 0; u < RC; ++u) {
    const int c = first + u * 64 * W;
    chunk_f32<DT>(load_chunk<DT, false>(row, nullptr, K, c, chunk_values(K, c)), v[u]);
  }
#pragma unroll
  for (int u = 0; u < RC; ++u)
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(v[u][i]));
  mx = quant_wave_max(mx);
  if constexpr (W > 1) {
    if (lane == 0) s_max[wave] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
  }
  const float s = __fdiv_rn(127.0f, __fadd_rn(mx, kEps));
  int8_t* dst = Xq + m * Kp;
  int sum = 0;
#pragma unroll
  for (int u = 0; u < RC; ++u) {
    const int c = first + u * 64 * W;
    if (8 * c >= Kp) continue;
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int code = act_code(v[u][i], s);
      sum += code;
      w[i >> 2] |= (static_cast<uint32_t>(code) & 0xffu) << (8 * (i & 3));
    }
    *reinterpret_cast<uint2*>(dst + 8 * c) = make_uint2(w[0], w[1]);
  }
  sum = quant_wave_sum(sum);
  if constexpr (W > 1) {
    if (lane == 0) s_sum[wave] = sum;
    __syncthreads();
    sum = s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3];
  }
  if (first == 0) {
    gamma_a[m] = mx;
    rowsum[m] = sum;
  }
}

template <int DT>
hipError_t launch_dt(const void* X, int64_t M, int64_t K, int8_t* Xq, float* gamma_a,
                     int32_t* rowsum, hipStream_t stream) {
  const int64_t Kp = padded_k(K);
  const int blocks = static_cast<int>((M + 3) / 4);
  constexpr int esize = DT == 0 ? 4 : 2;
  const bool vec = (reinterpret_cast<uintptr_t>(X) % 16 == 0) && ((K * esize) % 16 == 0);
  const int64_t chunks_per_lane = (K * esize / 16 + kWave - 1) / kWave;
  const char* rows = static_cast<const char*>(X);
  const int k = static_cast<int>(K), kp = static_cast<int>(Kp);
  const bool a_group_each = M < (int64_t(1) << 24);  // a launch holds fewer than 2^32 threads
  // Short rows go value by value, up to four to a lane: 20000x63 bfloat16 5.1 us, in
  // chunks 8.5, 20000x191 7.2 and 8.8, 2048x255 float32 3.3 and 3.5; only of very many
  // rows do chunks take those of 193 to 256 faster (60000x255 25 and 21).
  const bool short_rows = Kp <= 192 || (Kp <= 256 && M < 32768);
  if (!vec && !short_rows && Kp <= 2048)
    act_quant_any_kernel<DT, 4, 1><<<blocks, 256, 0, stream>>>(rows, M, k, kp, Xq, gamma_a, rowsum);
  else if (!vec && Kp > 2048 && Kp <= 8192 && a_group_each)
    act_quant_any_kernel<DT, 4, 4><<<static_cast<unsigned>(M), 256, 0, stream>>>(rows, M, k, kp, Xq, gamma_a, rowsum);
  else if (!vec && Kp > 8192 && Kp <= 28672 && a_group_each)
    act_quant_any_kernel<DT, 14, 4><<<static_cast<unsigned>(M), 256, 0, stream>>>(rows, M, k, kp, Xq, gamma_a, rowsum);
  else if (!vec)
    act_quant_kernel<DT, false, 4><<<blocks, 256, 0, stream>>>(X, M, K, Kp, Xq, gamma_a, rowsum);
  else if (chunks_per_lane <= 4)
    act_quant_kernel<DT, true, 4><<<blocks, 256, 0, stream>>>(X, M, K, Kp, Xq, gamma_a, rowsum);
  else if (chunks_per_lane <= 8)
    act_quant_kernel<DT, true, 8><<<blocks, 256, 0, stream>>>(X, M, K, Kp, Xq, gamma_a, rowsum);
  else if (chunks_per_lane <= 16)
    act_quant_kernel<DT, true, 16><<<blocks, 256, 0, stream>>>(X, M, K, Kp, Xq, gamma_a, rowsum);
  else if (chunks_per_lane <= 32)  // a workgroup per token: at most 8 chunks per thread
    act_quant_row_kernel<DT, 8><<<static_cast<unsigned>(M), 256, 0, stream>>>(X, K, Kp, Xq, gamma_a, rowsum);
  else if (chunks_per_lane <= 64)
    act_quant_row_kernel<DT, 16><<<static_cast<unsigned>(M), 256, 0, stream>>>(X, K, Kp, Xq, gamma_a, rowsum);
  else  // rows over 64 KiB: two passes, the second from L2
    act_quant_kernel<DT, true, 16><<<blocks, 256, 0, stream>>>(X, M, K, Kp, Xq, gamma_a, rowsum);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_act_quant(const void* X, int x_dtype, int64_t M, int64_t K, int8_t* Xq,
                            float* gamma_a, int32_t* rowsum, hipStream_t stream) {
  if (x_dtype == 0) return launch_dt<0>(X, M, K, Xq, gamma_a, rowsum, stream);
  return launch_dt<1>(X, M, K, Xq, gamma_a, rowsum, stream);
}

}  // namespace bitlinear
