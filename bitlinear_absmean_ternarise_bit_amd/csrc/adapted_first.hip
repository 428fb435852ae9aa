// What a projection with adapters does with X alone, in one launch
// (include/bitlinear_adapters.h): the adapters' first product and the tokens'
// codes.  Either leaves most of the GPU waiting for its loads; together they read X
// from memory once and are one launch (2048x4096 bf16, 16 ranks: 16.5 us, apart 11
// and 8.2; one token of 2048 columns 4.8).  With more than 32 ranks of float32 for 64
// tokens a workgroup, 12 of a lane's registers go to scratch memory, 26 with X of
// float32.
#include <algorithm>

#include "adapter_device.hpp"
#include "quant_act.hpp"

namespace bitlinear {

namespace {

// The codes of a token: chunks of 8 values, up to 4 to a lane in registers.  W = 4: a
// workgroup to a token, rows over 8192 values read twice; W = 1: a wave to a token of
// up to 2048 (3656x80 float32, 16 ranks, with the first product: a workgroup to a
// token 20 us, a wave 11).
template <int DT, int W>
__device__ __forceinline__ void token_codes(const char* row, int K, int Kp, int8_t* dst, float* gamma_a,
                                            int32_t* rowsum) {
  __shared__ float s_max[kAdapterWaves];
  __shared__ int s_sum[kAdapterWaves];
  constexpr int RC = 4, kLanes = W * kWave;
  const int lane = threadIdx.x & (kWave - 1), wave = wave_id(), me = W == 1 ? lane : static_cast<int>(threadIdx.x);
  float v[RC][8];
  float mx = 0.0f;
  auto load = [&](int c, float (&f)[8]) { chunk_f32<DT>(load_chunk<DT, false>(row, nullptr, K, c, chunk_values(K, c)), f); };
  auto widen = [&](const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(f[i]));
  };
#pragma unroll
  for (int u = 0; u < RC; ++u) load(me + u * kLanes, v[u]);
#pragma unroll
  for (int u = 0; u < RC; ++u) widen(v[u]);
  if constexpr (W > 1) {
    for (int c = me + RC * kLanes; 8 * c < K; c += kLanes) {
      float f[8];
      load(c, f);
      widen(f);
    }
  }
  mx = quant_wave_max(mx);
  if constexpr (W > 1) {
    if (lane == 0) s_max[wave] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
  }
  const float s = __fdiv_rn(127.0f, __fadd_rn(mx, kEps));
  int sum = 0;
  auto store = [&](int c, const float (&f)[8]) {
    if (8 * c >= Kp) return;
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int code = act_code(f[i], s);
      sum += code;
      w[i >> 2] |= (static_cast<uint32_t>(code) & 0xffu) << (8 * (i & 3));
    }
    *reinterpret_cast<uint2*>(dst + 8 * c) = make_uint2(w[0], w[1]);
  };
#pragma unroll
  for (int u = 0; u < RC; ++u) store(me + u * kLanes, v[u]);
  if constexpr (W > 1) {
    for (int c = me + RC * kLanes; 8 * c < Kp; c += kLanes) {
      float f[8];
      load(c, f);
      store(c, f);
    }
  }
  sum = quant_wave_sum(sum);
  if constexpr (W > 1) {
    if (lane == 0) s_sum[wave] = sum;
    __syncthreads();
    sum = s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3];
    __syncthreads();  // the next token's maxima and sums overwrite these
  }
  if (me == 0) {
    *gamma_a = mx;
    *rowsum = sum;
  }
}

constexpr int kWaveRow = 2048;  // codes of a row that a wave takes

// The first workgroups take the first product (groups x parts x spread of them),
// the others the codes of a token each, or of four.
template <int DT, int WT, int RB, int RT>
__global__ __launch_bounds__(kAdapterThreads, 2) void adapted_first_kernel(const char* X, int64_t M, int K, int Kp,
                                                                           Adapters ad, const char* down, float* parts,
                                                                           int nparts, int spread, int64_t shrinks,
                                                                           int64_t items, int64_t groups, int8_t* Xq,
                                                                           float* gamma_a, int32_t* rowsum) {
  for (int64_t b = blockIdx.x; b < items; b += gridDim.x) {
    if (b < shrinks) {
      const int64_t rest = b / nparts;
      shrink_body<DT, WT, RB, RT>(X, M, K, ad, down, parts, groups, rest / spread, groups, static_cast<int>(b % nparts),
                                  nparts, static_cast<int>(rest % spread), spread);
    } else if (Kp <= kWaveRow) {
      const int64_t m = kAdapterWaves * (b - shrinks) + wave_id();
      if (m < M) token_codes<DT, 1>(X + m * K * kBytes<DT>, K, Kp, Xq + m * Kp, gamma_a + m, rowsum + m);
    } else {
      const int64_t m = b - shrinks;
      token_codes<DT, 4>(X + m * K * kBytes<DT>, K, Kp, Xq + m * Kp, gamma_a + m, rowsum + m);
    }
  }
}

template <int DT, int WT, int RB>
hipError_t launch_as(const void* X, int64_t M, int64_t K, const Adapters& ad, const void* down, float* parts, int8_t* Xq,
                     float* ga, int32_t* rs, hipStream_t stream) {
  const ShrinkPlan p = shrink_plan(M, K);
  const int64_t groups = (M + 16 * RB - 1) / (16 * RB), shrinks = groups * p.parts * p.spread;
  const int64_t Kp = padded_k(K), items = shrinks + (Kp <= kWaveRow ? (M + kAdapterWaves - 1) / kAdapterWaves : M);
  auto kernel = ad.R <= 16   ? adapted_first_kernel<DT, WT, RB, 1>
                : ad.R <= 32 ? adapted_first_kernel<DT, WT, RB, 2>
                             : adapted_first_kernel<DT, WT, RB, 4>;
  kernel<<<static_cast<unsigned>(std::min(items, kMaxGrid)), kAdapterThreads, 0, stream>>>(
      static_cast<const char*>(X), M, static_cast<int>(K), static_cast<int>(Kp), ad, static_cast<const char*>(down),
      parts, p.parts, p.spread, shrinks, items, groups, Xq, ga, rs);
  return hipGetLastError();
}

template <int DT, int WT>
hipError_t launch_any(const void* X, int64_t M, int64_t K, const Adapters& ad, const void* down, float* parts, int8_t* Xq,
                      float* ga, int32_t* rs, hipStream_t stream) {
  return shrink_plan(M, K).blocks == 4 ? launch_as<DT, WT, 4>(X, M, K, ad, down, parts, Xq, ga, rs, stream)
                                       : launch_as<DT, WT, 1>(X, M, K, ad, down, parts, Xq, ga, rs, stream);
}

}  // namespace

hipError_t launch_adapted_first(const void* X, int x_dtype, int64_t M, int64_t K, const Adapters& ad, const void* down,
                                float* parts, int8_t* Xq, float* ga, int32_t* rs, hipStream_t stream) {
  if (x_dtype == kF32)
    return ad.w_dtype == kF32 ? launch_any<kF32, kF32>(X, M, K, ad, down, parts, Xq, ga, rs, stream)
                              : launch_any<kF32, kBf16>(X, M, K, ad, down, parts, Xq, ga, rs, stream);
  return ad.w_dtype == kF32 ? launch_any<kBf16, kF32>(X, M, K, ad, down, parts, Xq, ga, rs, stream)
                            : launch_any<kBf16, kBf16>(X, M, K, ad, down, parts, Xq, ga, rs, stream);
}

}  // namespace bitlinear
