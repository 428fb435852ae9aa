// Low-rank adapters (include/bitlinear_adapters.h) as three products on the bf16
// matrix cores:
//   shrink  T[m] = X[m] W[a]^T          contraction along the rows of W
//   expand  Y[m] += scale T[m] W[a]     contraction over the R rows of W
//   grad    dW[a] = scale V^T X         contraction over an adapter's tokens
// Forward: shrink with down, expand with up.  Backward: shrink of dY with up,
// expand with down, grad of both.
//
// Accuracy: a float32 operand is the exact sum of three bfloat16 planes (its
// upper 8 significant bits, the next 8, the rest), and the products of planes p
// and q with p + q <= 2 are formed; what is left out is below 2^-24 of the
// product.  The matrix cores are far from the bound (at R = 16 each value of X or
// Y that passes takes part in 16 multiplications), so this costs nothing that
// shows and T needs no rounding.
//
// Tokens of different adapters: a block of 16 tokens goes through each adapter
// that it holds, all 16 rows at once, and keeps the rows that are the adapter's
// own.  A row of a matrix-core product depends on its own operand row only, so
// what other rows hold (another request's infinities, memory that nothing has
// written) cannot reach it.  In the contraction over tokens (grad) rows of other
// adapters are zeros on both sides by selection, not by multiplication.
#include <algorithm>

#include "adapter_ops.hpp"
#include "block_device.hpp"

namespace bitlinear {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256, kWaves = 4;
constexpr int kBlock = 16;      // tokens of a block
constexpr int kTileCols = 128;  // columns of a wave in expand and grad
constexpr int64_t kMaxGrid = int64_t(1) << 20;  // workgroups; each walks every gridDim.x-th item

template <int DT>
constexpr int kPlanes = DT == kF32 ? 3 : 1;

// upper or lower halves of two words, the first one's in the lower half
__device__ __forceinline__ uint32_t upper(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }
__device__ __forceinline__ uint32_t lower(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }

// Planes of two float32: what truncation leaves is exact each time, and the third
// plane holds the last 8 bits.
__device__ __forceinline__ void split(float a, float b, uint32_t (&p)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
    p[i] = upper(ua, ub);
    a = __fsub_rn(a, __uint_as_float(ua & 0xffff0000u));
    b = __fsub_rn(b, __uint_as_float(ub & 0xffff0000u));
  }
}

// Chunk c (eight columns) of a row of C, zeros behind it.
template <int DT>
__device__ __forceinline__ Raw<DT> any_chunk(const char* row, int64_t C, int64_t c) {
  const int n = static_cast<int>(max(int64_t(0), min(int64_t(8), C - 8 * c)));
  // the row's last 16 columns are enough to place what is left of it
  const int64_t skip = C > 16 ? (C - 9) / 8 * 8 : 0;  // a multiple of 8; 9 to 16 columns follow, or all of a short row
  if (n == 8 || C <= 16) {
    const int K = n == 8 ? 8 : static_cast<int>(C);
    const char* at = n == 8 ? row + 8 * c * kBytes<DT> : row;
    const int cc = n == 8 ? 0 : static_cast<int>(c);
    return K >= 8 ? load_chunk<DT, false>(at, nullptr, K, cc, n) : load_chunk<DT, true>(at, nullptr, K, cc, n);
  }
  return load_chunk<DT, false>(row + skip * kBytes<DT>, nullptr, static_cast<int>(C - skip),
                               static_cast<int>(c - skip / 8), n);
}
template <int DT>
__device__ __forceinline__ Raw<DT> whole_chunk(const char* row, int64_t c) {
  return fetch_chunk<DT, false>(row + 8 * c * kBytes<DT>, nullptr, 8, 1, 0);
}

// Eight consecutive values of a row as operand planes (shrink).
template <int DT>
__device__ __forceinline__ void row_planes(const Raw<DT>& r, bf16x8 (&p)[kPlanes<DT>]) {
  if constexpr (DT == kBf16) {
    p[0] = __builtin_bit_cast(bf16x8, r.a);
  } else {
    float v[8];
    chunk_f32<DT>(r, v);
    v4u w[3];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t s[3];
      split(v[2 * i], v[2 * i + 1], s);
#pragma unroll
      for (int q = 0; q < 3; ++q) w[q][i] = s[q];
    }
#pragma unroll
    for (int q = 0; q < 3; ++q) p[q] = __builtin_bit_cast(bf16x8, w[q]);
  }
}

// Four rows of eight columns as the operand planes of each column: element i of
// plane q of column j is row i's (expand, grad: rows are the contraction).
template <int DT>
__device__ __forceinline__ void column_planes(const Raw<DT> (&r)[4], s16x4 (&p)[kPlanes<DT>][8]) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  if constexpr (DT == kBf16) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      p[0][2 * h] = __builtin_bit_cast(s16x4, u32x2{lower(r[0].a[h], r[1].a[h]), lower(r[2].a[h], r[3].a[h])});
      p[0][2 * h + 1] = __builtin_bit_cast(s16x4, u32x2{upper(r[0].a[h], r[1].a[h]), upper(r[2].a[h], r[3].a[h])});
    }
  } else {
    float v[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) chunk_f32<DT>(r[i], v[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t lo[3], hi[3];
      split(v[0][j], v[1][j], lo);
      split(v[2][j], v[3][j], hi);
#pragma unroll
      for (int q = 0; q < 3; ++q) p[q][j] = __builtin_bit_cast(s16x4, u32x2{lo[q], hi[q]});
    }
  }
}

// Four float32 as operand planes.
__device__ __forceinline__ void value_planes(const f32x4& v, s16x4 (&p)[3]) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  uint32_t lo[3], hi[3];
  split(v[0], v[1], lo);
  split(v[2], v[3], hi);
#pragma unroll
  for (int q = 0; q < 3; ++q) p[q] = __builtin_bit_cast(s16x4, u32x2{lo[q], hi[q]});
}

// The adapter of token m0 + lane (lanes 0 to 15), -1 for none.
__device__ __forceinline__ int token_adapter(const Adapters& ad, int64_t m0, int64_t M, int lane) {
  const int64_t m = m0 + lane;
  const int id = lane < kBlock && m < M ? ad.rows[m] : -1;
  return id >= 0 && id < ad.A ? id : -1;
}

// Calls f(a, mine) for the adapters of a block, every `spread`-th one from
// `from`: mine has bit t set where token t is a's.  The same for all lanes.
template <typename F>
__device__ __forceinline__ void each_adapter(int id, int spread, int from, F&& f) {
  uint32_t todo = static_cast<uint32_t>(__ballot(id >= 0)) & 0xffffu;
  for (int n = 0; todo; ++n) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
    const uint32_t mine = static_cast<uint32_t>(__ballot(id == a)) & 0xffffu;
    todo &= ~mine;
    if (n % spread == from) f(a, mine);
  }
}

// ---- shrink ---------------------------------------------------------------------
// A workgroup takes a block of 16 tokens, one part of the columns and every
// spread-th adapter of the block; its four waves share the part's columns in
// steps of 32 (v_mfma_f32_16x16x32_bf16: lane l holds token or rank row l % 16,
// columns 8 (l / 16) .. + 7) and add their sums in LDS.  RT tiles of 16 ranks at
// a time.
template <int XT, int WT, int RT>
__global__ __launch_bounds__(kThreads) void shrink_kernel(const char* __restrict__ X, int64_t M, int64_t C, Adapters ad,
                                                          const char* __restrict__ W, float* __restrict__ parts,
                                                          int64_t blocks) {
  __shared__ f32x4 sums[kWaves][RT][kWave];
  const int wave = wave_id(), lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const int Rp = (ad.R + 15) & ~15;
  const int64_t steps = (C + 31) / 32, whole = C / 32;
  const int64_t q = static_cast<int64_t>(blockIdx.y) * kWaves + wave, Q = static_cast<int64_t>(gridDim.y) * kWaves;
  const int64_t lo = q * steps / Q, hi = (q + 1) * steps / Q;
  for (int64_t block = blockIdx.x; block < blocks; block += gridDim.x) {
    const int64_t m0 = block * kBlock;
    const char* xrow = X + min(m0 + l, M - 1) * C * kBytes<XT>;
    float* out = parts + (static_cast<int64_t>(blockIdx.y) * M + m0) * Rp;
    each_adapter(token_adapter(ad, m0, M, lane), gridDim.z, blockIdx.z, [&](int a, uint32_t mine) {
      for (int r0 = 0; r0 < ad.R; r0 += 16 * RT) {
        f32x4 acc[RT];
        const char* wrow[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
          wrow[t] = W + (static_cast<int64_t>(a) * ad.R + min(r0 + 16 * t + l, ad.R - 1)) * C * kBytes<WT>;
        }
        auto add = [&](const Raw<XT>& xr, const Raw<WT> (&wr)[RT]) {
          bf16x8 x[kPlanes<XT>];
          row_planes<XT>(xr, x);
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            bf16x8 w[kPlanes<WT>];
            row_planes<WT>(wr[t], w);
#pragma unroll
            for (int p = 0; p < kPlanes<XT>; ++p)
#pragma unroll
              for (int s = 0; s < kPlanes<WT>; ++s)
                if (p + s <= 2) acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[p], w[s], acc[t], 0, 0, 0);
          }
        };
        const int64_t end = min(hi, whole);
#pragma unroll 4
        for (int64_t st = lo; st < end; ++st) {
          const int64_t c = 4 * st + g;
          Raw<WT> wr[RT];
          const Raw<XT> xr = whole_chunk<XT>(xrow, c);
#pragma unroll
          for (int t = 0; t < RT; ++t) wr[t] = whole_chunk<WT>(wrow[t], c);
          add(xr, wr);
        }
        if (whole >= lo && whole < hi) {  // the step that the row's end cuts
          const int64_t c = 4 * whole + g;
          Raw<WT> wr[RT];
          const Raw<XT> xr = any_chunk<XT>(xrow, C, c);
#pragma unroll
          for (int t = 0; t < RT; ++t) wr[t] = any_chunk<WT>(wrow[t], C, c);
          add(xr, wr);
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) sums[wave][t][lane] = acc[t];
        __syncthreads();
        if (wave < RT) {
          f32x4 v = sums[0][wave][lane];
#pragma unroll
          for (int w = 1; w < kWaves; ++w) v += sums[w][wave][lane];
          const int r = r0 + 16 * wave + l;
          if (r < Rp) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (mine >> (4 * g + i) & 1u) out[static_cast<int64_t>(4 * g + i) * Rp + r] = r < ad.R ? v[i] : 0.0f;
          }
        }
        __syncthreads();
      }
    });
  }
}

// ---- expand ---------------------------------------------------------------------
// A wave takes a block of 16 tokens and 128 columns; four waves to a workgroup.
// v_mfma_f32_16x16x16_bf16 with T as the rows (lane l: token l % 16, ranks
// 4 (l / 16) .. + 3) and W as the columns: lane l loads eight consecutive columns
// 8 (l % 16) .. + 7 of its four rank rows, 16 or 32 bytes a load, and column j of
// each lane's eight is an operand of its own, so no transposition through LDS is
// needed and a lane ends with eight consecutive columns of four tokens.
template <int WT>
__global__ __launch_bounds__(kThreads) void expand_kernel(const float* __restrict__ parts, int nparts, int64_t M,
                                                          int64_t C, Adapters ad, const char* __restrict__ W, float* Y,
                                                          int accumulate, float* __restrict__ T, int64_t items,
                                                          int64_t tiles) {
  const int wave = wave_id(), lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const int Rp = (ad.R + 15) & ~15;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t block = item / tiles, m0 = block * kBlock;
    const int64_t n0 = ((item - block * tiles) * kWaves + wave) * kTileCols;
    const bool low_out = T != nullptr && n0 == 0;  // this wave also writes T
    if (n0 >= C) continue;
    const int64_t c = n0 / 8 + l;  // the lane's chunk of eight columns
    const int n = static_cast<int>(max(int64_t(0), min(int64_t(8), C - 8 * c)));
    const int id = token_adapter(ad, m0, M, lane);
    const float* trow = parts + min(m0 + l, M - 1) * Rp + 4 * g;
    auto add_row = [&](int64_t m, const float (&d)[8]) {
      char* y = reinterpret_cast<char*>(Y + m * C + n0) + 32 * l;
      float v[8];
      if (accumulate && n > 0) {
        chunk_f32<kF32>(n == 8 ? load_chunk<kF32, false>(y, nullptr, 8, 0, 8) : load_chunk<kF32, true>(y, nullptr, n, 0, n), v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __fadd_rn(v[j], d[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = d[j];
      }
      store_chunk<kF32>(y, 0, n, v);
    };
    each_adapter(id, gridDim.y, blockIdx.y, [&](int a, uint32_t mine) {
      const float scale = ad.scales[a];
      f32x4 d[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      for (int r0 = 0; r0 < ad.R; r0 += 16) {
        Raw<WT> w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = r0 + 4 * g + i;
          const char* row = W + (static_cast<int64_t>(a) * ad.R + min(r, ad.R - 1)) * C * kBytes<WT>;
          w[i] = any_chunk<WT>(row, C, c);
          if (r >= ad.R) w[i] = Raw<WT>{};
        }
        f32x4 t = *reinterpret_cast<const f32x4*>(trow + r0);
        for (int s = 1; s < nparts; ++s) t += *reinterpret_cast<const f32x4*>(trow + static_cast<int64_t>(s) * M * Rp + r0);
        if (low_out && (mine >> l & 1u)) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (r0 + 4 * g + i < ad.R) T[(m0 + l) * ad.R + r0 + 4 * g + i] = t[i];
        }
        s16x4 tp[3], wp[kPlanes<WT>][8];
        value_planes(t * scale, tp);
        column_planes<WT>(w, wp);
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
          for (int s = 0; s < kPlanes<WT>; ++s)
            if (p + s <= 2) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                d[j] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(tp[p], wp[s][j], d[j], 0, 0, 0);
            }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v[8] = {d[0][i], d[1][i], d[2][i], d[3][i], d[4][i], d[5][i], d[6][i], d[7][i]};
        if (mine >> (4 * g + i) & 1u) add_row(m0 + 4 * g + i, v);
      }
    });
    if (blockIdx.y == 0 && (low_out || !accumulate)) {  // tokens without an adapter
      const uint32_t none = ~static_cast<uint32_t>(__ballot(id >= 0));
      const float zero[8] = {};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + 4 * g + i;
        if (!accumulate && m < M && (none >> (4 * g + i) & 1u)) add_row(m, zero);
      }
      if (low_out && m0 + l < M && (none >> l & 1u))
        for (int r = g; r < ad.R; r += 4) T[(m0 + l) * ad.R + r] = 0.0f;
    }
  }
}

// T[m, r] from its parts, zeros for rows without an adapter.
__global__ __launch_bounds__(kThreads) void join_kernel(const float* __restrict__ parts, int nparts, int64_t M,
                                                        Adapters ad, float* __restrict__ T) {
  const int Rp = (ad.R + 15) & ~15;
  const int64_t n = M * ad.R;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t m = i / ad.R;
    const int id = ad.rows[m];
    float v = 0.0f;
    if (id >= 0 && id < ad.A)
      for (int s = 0; s < nparts; ++s) v += parts[(s * M + m) * Rp + (i - m * ad.R)];
    T[i] = v;
  }
}

// ---- grad -----------------------------------------------------------------------
// A workgroup takes 128 columns, one adapter, RT tiles of 16 ranks and one part
// of the tokens; each of its four waves a quarter of those, 16 tokens at a time
// (blocks without one of the adapter's are passed over).  V is the row operand
// (lane l: rank l % 16, tokens 4 (l / 16) .. + 3), X the columns as in expand.
// The waves' sums meet in LDS, and each wave then writes one of every four ranks,
// eight consecutive columns to a lane.
template <int XT, int RT>
__global__ __launch_bounds__(kThreads) void grad_kernel(const float* __restrict__ V, const char* __restrict__ X,
                                                        int64_t M, int64_t C, Adapters ad, float* __restrict__ out,
                                                        int scaled, int nparts, int64_t items, int64_t tiles,
                                                        int groups) {
  __shared__ f32x4 sums[kWaves][8][kWave];
  const int wave = wave_id(), lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const int64_t blocks = (M + kBlock - 1) / kBlock;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    int64_t rest = item;
    const int64_t tile = rest % tiles;
    rest /= tiles;
    const int group = static_cast<int>(rest % groups);
    rest /= groups;
    const int a = static_cast<int>(rest % ad.A), part = static_cast<int>(rest / ad.A);
    const int r0 = group * 16 * RT;
    const int64_t c = tile * (kTileCols / 8) + l;
    const int64_t q = static_cast<int64_t>(part) * kWaves + wave, Q = static_cast<int64_t>(nparts) * kWaves;
    const int64_t lo = q * blocks / Q, hi = (q + 1) * blocks / Q;
    f32x4 acc[RT][8];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[t][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t b = lo; b < hi; b += 4) {
      const int64_t mine_at = b * kBlock + lane;
      const uint64_t here = __ballot(mine_at < min(hi * kBlock, M) && ad.rows[mine_at < M ? mine_at : M - 1] == a);
      for (int sub = 0; sub < 4; ++sub) {
        const uint32_t mine = static_cast<uint32_t>(here >> (16 * sub)) & 0xffffu;
        if (!mine) continue;
        const int64_t m0 = (b + sub) * kBlock;
        Raw<XT> x[4];
        f32x4 v[RT];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t m = min(m0 + 4 * g + i, M - 1);
          const bool use = mine >> (4 * g + i) & 1u;
          x[i] = any_chunk<XT>(X + m * C * kBytes<XT>, C, c);
          if (!use) x[i] = Raw<XT>{};
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            const int r = r0 + 16 * t + l;
            const float e = V[m * ad.R + min(r, ad.R - 1)];
            v[t][i] = use && r < ad.R ? e : 0.0f;
          }
        }
        s16x4 xp[kPlanes<XT>][8];
        column_planes<XT>(x, xp);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          s16x4 vp[3];
          value_planes(v[t], vp);
#pragma unroll
          for (int p = 0; p < 3; ++p)
#pragma unroll
            for (int s = 0; s < kPlanes<XT>; ++s)
              if (p + s <= 2) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  acc[t][j] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(vp[p], xp[s][j], acc[t][j], 0, 0, 0);
              }
        }
      }
    }
    const float scale = scaled ? ad.scales[a] : 1.0f;
    const int n = static_cast<int>(max(int64_t(0), min(int64_t(8), C - 8 * c)));
    for (int t = 0; t < RT; ++t) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        f32x4 mine = acc[0][j];
#pragma unroll
        for (int s = 1; s < RT; ++s) mine = t == s ? acc[s][j] : mine;
        sums[wave][j][lane] = mine;
      }
      __syncthreads();
      const int r = r0 + 16 * t + 4 * g + wave;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float s = reinterpret_cast<const float*>(&sums[0][j][lane])[wave];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) s += reinterpret_cast<const float*>(&sums[w][j][lane])[wave];
        v[j] = __fmul_rn(s, scale);
      }
      if (r < ad.R && n > 0) {
        float* to = out + ((static_cast<int64_t>(part) * ad.A + a) * ad.R + r) * C + 8 * c;
        store_chunk<kF32>(reinterpret_cast<char*>(to), 0, n, v);
      }
    }
    __syncthreads();
  }
}

// dW = scale * the sum of its parts
__global__ __launch_bounds__(kThreads) void grad_join_kernel(const float* __restrict__ parts, int nparts, int64_t n,
                                                             int64_t per_adapter, const float* __restrict__ scales,
                                                             float* __restrict__ dW) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    float v = parts[i];
    for (int s = 1; s < nparts; ++s) v += parts[s * n + i];
    dW[i] = __fmul_rn(v, scales[i / per_adapter]);
  }
}

unsigned flat_grid(int64_t n) {
  return static_cast<unsigned>(std::min<int64_t>((n + kThreads - 1) / kThreads, int64_t(1) << 16));
}

template <int XT, int WT>
hipError_t shrink_as(const void* X, int64_t M, int64_t C, const Adapters& ad, const void* W, float* parts,
                     hipStream_t s) {
  const ShrinkPlan p = shrink_plan(M, C);
  const int64_t blocks = (M + kBlock - 1) / kBlock;
  const dim3 grid(static_cast<unsigned>(std::min(blocks, kMaxGrid)), p.parts, p.spread);
  auto kernel = ad.R <= 16 ? shrink_kernel<XT, WT, 1> : ad.R <= 32 ? shrink_kernel<XT, WT, 2> : shrink_kernel<XT, WT, 4>;
  kernel<<<grid, kThreads, 0, s>>>(static_cast<const char*>(X), M, C, ad, static_cast<const char*>(W), parts, blocks);
  return hipGetLastError();
}

template <int XT>
hipError_t grad_as(const float* V, const void* X, int64_t M, int64_t C, const Adapters& ad, float* dW, float* ws,
                   hipStream_t s) {
  const GradPlan p = grad_plan(M, C, ad.A, ad.R);
  const int64_t items = int64_t(p.tiles) * p.groups * ad.A * p.parts;
  const unsigned grid = static_cast<unsigned>(std::min(items, kMaxGrid));
  const bool one = p.parts == 1;
  auto kernel = ad.R <= 16 ? grad_kernel<XT, 1> : ad.R <= 32 ? grad_kernel<XT, 2> : grad_kernel<XT, 4>;
  kernel<<<grid, kThreads, 0, s>>>(V, static_cast<const char*>(X), M, C, ad, one ? dW : ws, one, p.parts, items, p.tiles,
                                   p.groups);
  if (!one) {
    const int64_t per = int64_t(ad.R) * C, n = per * ad.A;
    grad_join_kernel<<<flat_grid(n), kThreads, 0, s>>>(ws, p.parts, n, per, ad.scales, dW);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_shrink(const void* X, int x_dtype, int64_t M, int64_t C, const Adapters& ad, const void* W,
                         float* parts, hipStream_t s) {
  if (x_dtype == kF32)
    return ad.w_dtype == kF32 ? shrink_as<kF32, kF32>(X, M, C, ad, W, parts, s)
                              : shrink_as<kF32, kBf16>(X, M, C, ad, W, parts, s);
  return ad.w_dtype == kF32 ? shrink_as<kBf16, kF32>(X, M, C, ad, W, parts, s)
                            : shrink_as<kBf16, kBf16>(X, M, C, ad, W, parts, s);
}

hipError_t launch_expand(const float* parts, int64_t M, int64_t C0, int64_t C, const Adapters& ad, const void* W,
                         float* Y, bool accumulate, float* T, hipStream_t s) {
  const ShrinkPlan p = shrink_plan(M, C0);
  const int64_t blocks = (M + kBlock - 1) / kBlock, tiles = (C + kWaves * kTileCols - 1) / (kWaves * kTileCols);
  const int64_t items = blocks * tiles;
  const dim3 grid(static_cast<unsigned>(std::min(items, kMaxGrid)), p.spread);
  auto kernel = ad.w_dtype == kF32 ? expand_kernel<kF32> : expand_kernel<kBf16>;
  kernel<<<grid, kThreads, 0, s>>>(parts, p.parts, M, C, ad, static_cast<const char*>(W), Y, accumulate, T, items,
                                   tiles);
  return hipGetLastError();
}

hipError_t launch_join(const float* parts, int64_t M, int64_t C0, const Adapters& ad, float* T, hipStream_t s) {
  join_kernel<<<flat_grid(M * ad.R), kThreads, 0, s>>>(parts, shrink_plan(M, C0).parts, M, ad, T);
  return hipGetLastError();
}

hipError_t launch_adapter_grad(const float* V, const void* X, int x_dtype, int64_t M, int64_t C, const Adapters& ad,
                               float* dW, float* ws, hipStream_t s) {
  return x_dtype == kF32 ? grad_as<kF32>(V, X, M, C, ad, dW, ws, s) : grad_as<kBf16>(V, X, M, C, ad, dW, ws, s);
}

}  // namespace bitlinear
