// Low-rank adapters (include/bitlinear_adapters.h) as three products on the bf16
// matrix cores:
//   shrink  T[m] = X[m] W[a]^T          contraction along the rows of W
//   expand  Y[m] += scale T[m] W[a]     contraction over the R rows of W
//   grad    dW[a] = scale V^T X         contraction over an adapter's tokens
// Forward: shrink with down, expand with up.  Backward: shrink of dY with up,
// expand with down, grad of both.
//
// Accuracy: a float32 operand is the sum of three bfloat16 planes, each what is left
// of it rounded to nearest, and the products of planes p and q with p + q <= 2 are
// formed.  The second plane is at most 2^-8 and the third 2^-17 of the value's power
// of two, so what is left out is at most 2^-24 (1 + 2^-10) of the product and as often
// above as below; planes cut off instead leave out up to 2^-21, always towards zero,
// and are no faster (55 calls of 9 sizes in both types: 0.98 to 1.03 times as long).
// The matrix cores are far from the bound (at R = 16 each value of X or Y that passes
// takes part in 16 multiplications), so this costs nothing that shows and T needs no
// rounding.
//
// Tokens of different adapters: a block of 16 tokens goes through each adapter
// that it holds, all 16 rows at once, and keeps the rows that are the adapter's
// own.  A row of a matrix-core product depends on its own operand row only, so
// what other rows hold (another request's infinities, memory that nothing has
// written) cannot reach it.  In the contraction over tokens (grad) rows of other
// adapters are zeros on both sides by selection, not by multiplication.
#include <algorithm>

#include "adapter_device.hpp"

namespace bitlinear {

namespace {

template <int XT, int WT, int RB, int RT>
__global__ __launch_bounds__(kAdapterThreads, 2) void shrink_kernel(const char* __restrict__ X, int64_t M, int64_t C,
                                                                    Adapters ad, const char* __restrict__ W,
                                                                    float* __restrict__ parts, int64_t groups) {
  shrink_body<XT, WT, RB, RT>(X, M, C, ad, W, parts, groups, blockIdx.x, gridDim.x, blockIdx.y, gridDim.y, blockIdx.z,
                              gridDim.z);
}

// ---- expand ---------------------------------------------------------------------
// A workgroup takes RB blocks of 16 tokens and 64 CW columns, 16 CW to a wave.
// T's planes come into LDS, with many tokens as join_kernel wrote them; with few
// the parts are added, scaled and split here, which saves a launch, and T itself
// leaves from the workgroups of the first columns, if the caller wants it.  (With
// many tokens each of a row's workgroups would read all parts again: at
// 2048x4096 and 64 ranks as much as Y itself.)
// v_mfma_f32_16x16x16_bf16 with T as the rows (lane l: token l % 16, ranks
// 4 (l / 16) .. + 3) and W as the columns: lane l loads CW consecutive columns
// of its four rank rows, 8 or 16 bytes a load, and column j of each lane's
// is an operand of its own, so no transposition through LDS is needed and a lane
// ends with CW consecutive columns of four tokens of each block, which it adds
// to Y.  2048x4096, 64 ranks of float32: 25 us for 67 MB of Y, of which a copy takes
// 13: a workgroup's loads, products and stores follow each other, and two of them
// fit a CU.
template <int WT, int RB, int CW>
__global__ __launch_bounds__(kAdapterThreads, 2) void expand_kernel(const float* __restrict__ parts, int nparts,
                                                          const uint16_t* __restrict__ planes, int64_t M, int64_t C, Adapters ad, const char* __restrict__ W, float* Y,
                                                          int accumulate, float* __restrict__ T, int64_t items,
                                                          int64_t tiles) {
  extern __shared__ __align__(16) short low[];  // [3 planes][RB * 16 tokens][Rp + 4]
  const int wave = wave_id(), lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const int Rp = (ad.R + 15) & ~15, stride = Rp + 4, plane = RB * kBlock * stride;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t group = item / tiles, tile = item - group * tiles, m0 = group * (RB * kBlock);
    if (planes != nullptr) {  // formed by join_kernel
      const int per_row = Rp / 8, n = RB * kBlock * per_row;
      for (int i = threadIdx.x; i < 3 * n; i += kAdapterThreads) {
        const int s = i / n, token = (i - s * n) / per_row, r = 8 * (i - s * n - token * per_row);
        const u32x2* from = reinterpret_cast<const u32x2*>(planes + (s * M + min(m0 + token, M - 1)) * Rp + r);
        u32x2* to = reinterpret_cast<u32x2*>(low + s * plane + token * stride + r);
        to[0] = from[0];
        to[1] = from[1];
      }
    } else {
      for (int i = threadIdx.x; i < RB * kBlock * (Rp / 4); i += kAdapterThreads) {
        const int token = i / (Rp / 4), r = 4 * (i - token * (Rp / 4));
        const int64_t m = m0 + token;
        const int id = m < M ? ad.rows[m] : -1;
        const bool has = id >= 0 && id < ad.A;
        f32x4 t = {0.0f, 0.0f, 0.0f, 0.0f};
        if (has) {
          const float* from = parts + m * Rp + r;
          t = *reinterpret_cast<const f32x4*>(from);
#pragma unroll 4
          for (int s = 1; s < nparts; ++s) t += *reinterpret_cast<const f32x4*>(from + static_cast<int64_t>(s) * M * Rp);
        }
        if (T != nullptr && tile == 0 && blockIdx.y == 0 && m < M) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (r + k < ad.R) T[m * ad.R + r + k] = t[k];
        }
        s16x4 p[3];
        value_planes(t * (has ? ad.scales[id] : 0.0f), p);
#pragma unroll
        for (int s = 0; s < 3; ++s) *reinterpret_cast<s16x4*>(low + s * plane + token * stride + r) = p[s];
      }
    }
    __syncthreads();
    const int64_t n0 = (tile * kAdapterWaves + wave) * (16 * CW);
    if (n0 < C) {
      const Columns at = lane_columns<CW>(C, n0 / CW + l);
      const bool inside = n0 + 16 * CW <= C;
      const int id = token_adapter(ad, m0, M, RB * kBlock, lane);
      // The group's rows of Y as a buffer resource: rows and columns that are not
      // to be touched lie at an offset past it, where loads give zeros and stores
      // are dropped, so no row takes a branch.
      const __amdgpu_buffer_rsrc_t yres = __builtin_amdgcn_make_buffer_rsrc(
          Y + m0 * C, 0, static_cast<int>(min(M - m0, int64_t(RB * kBlock)) * C * 4), 0x00020000);
      const uint32_t row_bytes = static_cast<uint32_t>(C) * 4u, y_col = static_cast<uint32_t>(at.first) * 4u;
      auto y_at = [&](int token, uint64_t rows) {
        return rows >> token & 1u ? static_cast<uint32_t>(token) * row_bytes + y_col : kNowhere;
      };
      auto store_row = [&](uint32_t off, const float (&v)[CW]) {
        if (inside) {
#pragma unroll
          for (int h = 0; h < CW / 4; ++h)
            __builtin_amdgcn_raw_buffer_store_b128(v4u{__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]),
                                                       __float_as_uint(v[4 * h + 2]), __float_as_uint(v[4 * h + 3])},
                                                   yres, off + 16u * h, 0, 0);
        } else {
#pragma unroll
          for (int j = 0; j < CW; ++j)
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[j]), yres, j >= at.skip ? off + 4u * j : kNowhere, 0,
                                                  0);
        }
      };
      auto load_w = [&](int a, int r0, Some<WT, CW> (&w)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = load_some<WT, CW>(W + ((static_cast<int64_t>(a) * ad.R + min(r0 + 4 * g + i, ad.R - 1)) * C + at.first) *
                                          kBytes<WT>);
      };
      each_adapter(id, gridDim.y, blockIdx.y, [&](int a, uint64_t mine) {
        Some<WT, CW> w[4];
        load_w(a, 0, w);
        v4u y[RB][4][CW / 4];  // asked for ahead of the products
        auto load_y = [&](int b, v4u (&v)[4][CW / 4]) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t off = y_at(kBlock * b + 4 * g + i, mine);
#pragma unroll
            for (int h = 0; h < CW / 4; ++h) v[i][h] = __builtin_amdgcn_raw_buffer_load_b128(yres, off + 16u * h, 0, 0);
          }
        };
        if (accumulate) {
#pragma unroll
          for (int b = 0; b < RB; ++b) load_y(b, y[b]);
        }
        f32x4 d[RB][CW];
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
          for (int j = 0; j < CW; ++j) d[b][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int r0 = 0; r0 < ad.R; r0 += 16) {
          if (r0 + 16 > ad.R) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (r0 + 4 * g + i >= ad.R) w[i] = Some<WT, CW>{};
          }
          s16x4 wp[kPlanes<WT>][CW];
          column_planes<WT, CW>(w, wp);
          if (r0 + 16 < ad.R) load_w(a, r0 + 16, w);
#pragma unroll
          for (int b = 0; b < RB; ++b) {
            s16x4 tp[3];
#pragma unroll
            for (int s = 0; s < 3; ++s)
              tp[s] = *reinterpret_cast<const s16x4*>(low + s * plane + (kBlock * b + l) * stride + r0 + 4 * g);
#pragma unroll
            for (int p = 0; p < 3; ++p)
#pragma unroll
              for (int s = 0; s < kPlanes<WT>; ++s)
                if (p + s <= 2) {
#pragma unroll
                  for (int j = 0; j < CW; ++j)
                    d[b][j] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(tp[p], wp[s][j], d[b][j], 0, 0, 0);
                }
          }
        }
#pragma unroll
        for (int b = 0; b < RB; ++b) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v[CW];
#pragma unroll
            for (int j = 0; j < CW; ++j)
              v[j] = accumulate ? __fadd_rn(__uint_as_float(y[b][i][j >> 2][j & 3]), d[b][j][i]) : d[b][j][i];
            store_row(y_at(kBlock * b + 4 * g + i, mine), v);
          }
        }
      });
      if (!accumulate && blockIdx.y == 0) {  // tokens without an adapter (the resource ends with the last token)
        const uint64_t none = ~__ballot(id >= 0);
        const float zero[CW] = {};
        for (int b = 0; b < RB; ++b)
          for (int i = 0; i < 4; ++i) store_row(y_at(kBlock * b + 4 * g + i, none), zero);
      }
    }
    __syncthreads();  // the next item's planes overwrite these
  }
}

// T [M, R] from its parts, and its planes, scaled, [3][M][Rp] (zeros for rows
// without an adapter); either may be NULL.  Four ranks to a thread.
__global__ __launch_bounds__(kAdapterThreads) void join_kernel(const float* __restrict__ parts, int nparts, int64_t M,
                                                               Adapters ad, float* __restrict__ T,
                                                               uint16_t* __restrict__ planes) {
  const int Rp = (ad.R + 15) & ~15, quads = Rp / 4;
  const int64_t n = M * quads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kAdapterThreads + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * kAdapterThreads) {
    const int64_t m = i / quads;
    const int r = 4 * static_cast<int>(i - m * quads), id = ad.rows[m];
    const bool has = id >= 0 && id < ad.A;
    f32x4 t = {0.0f, 0.0f, 0.0f, 0.0f};
    if (has) {
      const float* from = parts + m * Rp + r;
      t = *reinterpret_cast<const f32x4*>(from);
#pragma unroll 4
      for (int s = 1; s < nparts; ++s) t += *reinterpret_cast<const f32x4*>(from + static_cast<int64_t>(s) * M * Rp);
    }
    if (T != nullptr) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (r + k < ad.R) T[m * ad.R + r + k] = t[k];
    }
    if (planes != nullptr) {
      s16x4 p[3];
      value_planes(t * (has ? ad.scales[id] : 0.0f), p);
#pragma unroll
      for (int s = 0; s < 3; ++s) *reinterpret_cast<s16x4*>(planes + (s * M + m) * Rp + r) = p[s];
    }
  }
}

// ---- grad -----------------------------------------------------------------------
// A workgroup takes 64 columns, one adapter, RT tiles of 16 ranks and one part
// of the tokens; each of its four waves a quarter of those, 16 tokens at a time
// (blocks without one of the adapter's are passed over), with the next block's
// loads on their way.  Parts and waves take blocks in turn, so that a request's
// tokens, which lie together, are shared by all of them (2048x4096 of 8 requests, 64
// ranks, both gradients: 83 us with consecutive blocks to a wave, 53 in turn).  V is
// the row operand (lane l: rank l % 16, tokens 4 (l / 16) .. + 3), X the columns as in
// expand.  The waves' sums meet in LDS, and each wave then writes one of every four
// ranks.  With more than 32 ranks (RT = 4) two blocks of X and V beside 64 sums exceed a
// lane's 256 registers: 24 of them go to scratch memory in the token loop, 69 with X of
// float32.
template <int XT, int RT>
__global__ __launch_bounds__(kAdapterThreads, 2) void grad_kernel(const float* __restrict__ V, const char* __restrict__ X,
                                                        int64_t M, int64_t C, Adapters ad, float* __restrict__ out,
                                                        int scaled, int nparts, int64_t items, int64_t tiles,
                                                        int groups) {
  constexpr int CW = kGradCols;
  __shared__ f32x4 sums[kAdapterWaves][CW][kWave];
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
    const Columns at = lane_columns<CW>(C, tile * 16 + l);
    const int64_t q = static_cast<int64_t>(part) * kAdapterWaves + wave, Q = static_cast<int64_t>(nparts) * kAdapterWaves;
    f32x4 acc[RT][CW];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int j = 0; j < CW; ++j) acc[t][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // The adapter's tokens in blocks q, q + Q, q + 2 Q ..., four blocks at a time, the
    // ids of the next four already loaded.
    auto ids_at = [&](int64_t i) {
      const int64_t m = (q + Q * (i + g)) * kBlock + l;
      return m < M ? ad.rows[m] : -1;
    };
    int64_t base = 0;
    int sub = 0;
    uint64_t here = __ballot(ids_at(0) == a);
    int ids_next = ids_at(4);
    auto next = [&](uint32_t& mine) -> int64_t {  // the next block that holds one of them, -1 at the end
      for (;;) {
        if (sub == 4) {
          base += 4;
          sub = 0;
          here = __ballot(ids_next == a);
          ids_next = ids_at(base + 4);
        }
        const int64_t b = q + Q * (base + sub);
        if (b >= blocks) return -1;
        mine = static_cast<uint32_t>(here >> (16 * sub)) & 0xffffu;
        ++sub;
        if (mine) return b;
      }
    };
    auto load = [&](int64_t b, Some<XT, CW> (&xr)[4], float (&vr)[RT][4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t m = min(b * kBlock + 4 * g + i, M - 1);
        xr[i] = load_some<XT, CW>(X + (m * C + at.first) * kBytes<XT>);
#pragma unroll
        for (int t = 0; t < RT; ++t) vr[t][i] = V[m * ad.R + min(r0 + 16 * t + l, ad.R - 1)];
      }
    };
    auto add = [&](uint32_t own, Some<XT, CW> (&xr)[4], float (&vr)[RT][4]) {
      if (own != 0xffffu) {  // rows of others: zeros on both sides
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!(own >> (4 * g + i) & 1u)) {
            xr[i] = Some<XT, CW>{};
#pragma unroll
            for (int t = 0; t < RT; ++t) vr[t][i] = 0.0f;
          }
      }
      s16x4 xp[kPlanes<XT>][CW];
      column_planes<XT, CW>(xr, xp);
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        s16x4 vp[3];
        value_planes(f32x4{vr[t][0], vr[t][1], vr[t][2], vr[t][3]}, vp);
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
          for (int s = 0; s < kPlanes<XT>; ++s)
            if (p + s <= 2) {
#pragma unroll
              for (int j = 0; j < CW; ++j)
                acc[t][j] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(vp[p], xp[s][j], acc[t][j], 0, 0, 0);
            }
      }
    };
    Some<XT, CW> x0[4], x1[4];
    float v0[RT][4], v1[RT][4];
    uint32_t mine0 = 0u, mine1 = 0u;
    int64_t b = next(mine0);
    if (b >= 0) load(b, x0, v0);
    while (b >= 0) {
      b = next(mine1);
      if (b >= 0) load(b, x1, v1);
      add(mine0, x0, v0);
      if (b < 0) break;
      b = next(mine0);
      if (b >= 0) load(b, x0, v0);
      add(mine1, x1, v1);
    }
    const float scale = scaled ? ad.scales[a] : 1.0f;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < CW; ++j) sums[wave][j][lane] = acc[t][j];
      __syncthreads();
      const int r = r0 + 16 * t + 4 * g + wave;
      if (r >= ad.R) continue;
      float* to = out + ((static_cast<int64_t>(part) * ad.A + a) * ad.R + r) * C + at.first;
      float v[CW];
#pragma unroll
      for (int j = 0; j < CW; ++j) {
        float s = reinterpret_cast<const float*>(&sums[0][j][lane])[wave];
#pragma unroll
        for (int w = 1; w < kAdapterWaves; ++w) s += reinterpret_cast<const float*>(&sums[w][j][lane])[wave];
        v[j] = __fmul_rn(s, scale);
      }
      if (at.skip == 0) {
#pragma unroll
        for (int h = 0; h < CW / 4; ++h)
          *reinterpret_cast<v4u_by4*>(to + 4 * h) = v4u{__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]),
                                                        __float_as_uint(v[4 * h + 2]), __float_as_uint(v[4 * h + 3])};
      } else {
#pragma unroll
        for (int j = 0; j < CW; ++j)
          if (j >= at.skip) to[j] = v[j];
      }
    }
    __syncthreads();
  }
}

// dW = scale * the sum of its parts (64x4096 in 8 parts 5.2 us, the products 16.6)
__global__ __launch_bounds__(kAdapterThreads) void grad_join_kernel(const float* __restrict__ parts, int nparts, int64_t n,
                                                             int64_t per_adapter, const float* __restrict__ scales,
                                                             float* __restrict__ dW) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kAdapterThreads + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * kAdapterThreads) {
    float v = parts[i];
    for (int s = 1; s < nparts; ++s) v += parts[s * n + i];
    dW[i] = __fmul_rn(v, scales[i / per_adapter]);
  }
}

// ---- fewer than 8 columns (expand: or more than 2^24) -------------------------------
// A lane of shrink takes eight columns, and a row has to hold that many (a group's rows
// of Y have to fit a buffer resource); else one thread to a value, float32 sums.  Lanes
// of expand and grad take four: they could do with rows of 4 to 7, which go the same way
// as in shrink so that there is one cut (no projection is that narrow).
template <int DT>
__device__ __forceinline__ float value_at(const char* p, int64_t i) {
  if constexpr (DT == kF32) return reinterpret_cast<const float*>(p)[i];
  else return bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[i]);
}

template <int XT, int WT>
__global__ __launch_bounds__(kAdapterThreads) void shrink_short_kernel(const char* __restrict__ X, int64_t M, int64_t C, Adapters ad,
                                                                const char* __restrict__ W, float* __restrict__ T) {
  const int Rp = (ad.R + 15) & ~15;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kAdapterThreads + threadIdx.x; i < M * Rp;
       i += static_cast<int64_t>(gridDim.x) * kAdapterThreads) {
    const int64_t m = i / Rp;
    const int r = static_cast<int>(i - m * Rp), id = ad.rows[m];
    float v = 0.0f;
    if (id >= 0 && id < ad.A && r < ad.R)
      for (int64_t c = 0; c < C; ++c)
        v = __fmaf_rn(value_at<XT>(X, m * C + c), value_at<WT>(W, (static_cast<int64_t>(id) * ad.R + r) * C + c), v);
    T[i] = v;
  }
}

template <int WT>
__global__ __launch_bounds__(kAdapterThreads) void expand_short_kernel(const float* __restrict__ parts, int nparts, int64_t M,
                                                                int64_t C, Adapters ad, const char* __restrict__ W, float* Y,
                                                                int accumulate) {
  const int Rp = (ad.R + 15) & ~15;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kAdapterThreads + threadIdx.x; i < M * C;
       i += static_cast<int64_t>(gridDim.x) * kAdapterThreads) {
    const int64_t m = i / C;
    const int64_t c = i - m * C;
    const int id = ad.rows[m];
    const bool has = id >= 0 && id < ad.A;
    if (!has) {
      if (!accumulate) Y[i] = 0.0f;
      continue;
    }
    const float scale = ad.scales[id];
    float v = 0.0f;
    for (int r = 0; r < ad.R; ++r) {
      float t = parts[m * Rp + r];
      for (int s = 1; s < nparts; ++s) t += parts[(s * M + m) * Rp + r];
      v = __fmaf_rn(__fmul_rn(t, scale), value_at<WT>(W, (static_cast<int64_t>(id) * ad.R + r) * C + c), v);
    }
    Y[i] = accumulate ? __fadd_rn(Y[i], v) : v;
  }
}

// one workgroup to a value of dW: its tokens in turn, the threads' sums in LDS
template <int XT>
__global__ __launch_bounds__(kAdapterThreads) void grad_short_kernel(const float* __restrict__ V, const char* __restrict__ X,
                                                              int64_t M, int64_t C, Adapters ad, float* __restrict__ dW,
                                                              int64_t n) {
  __shared__ float slot[kAdapterWaves];
  for (int64_t i = blockIdx.x; i < n; i += gridDim.x) {
    const int64_t row = i / C;
    const int64_t c = i - row * C;
    const int a = static_cast<int>(row / ad.R), r = static_cast<int>(row - int64_t(a) * ad.R);
    float v[1] = {0.0f};
    for (int64_t m = threadIdx.x; m < M; m += kAdapterThreads)
      if (ad.rows[m] == a) v[0] = __fmaf_rn(V[m * ad.R + r], value_at<XT>(X, m * C + c), v[0]);
    team_sum<kAdapterWaves, 1>(v, slot, wave_id(), threadIdx.x & 63);
    if (threadIdx.x == 0) dW[i] = __fmul_rn(v[0], ad.scales[a]);
    __syncthreads();
  }
}

unsigned flat_grid(int64_t n) {
  return static_cast<unsigned>(std::min<int64_t>((n + kAdapterThreads - 1) / kAdapterThreads, int64_t(1) << 16));
}

// Columns for the short kernels.  (Such few columns are one part of a shrink.)
bool few(int64_t C) { return C < 8; }

template <int XT, int WT, int RB>
hipError_t shrink_as(const void* X, int64_t M, int64_t C, const Adapters& ad, const void* W, float* parts,
                     const ShrinkPlan& p, hipStream_t s) {
  const int64_t groups = (M + RB * kBlock - 1) / (RB * kBlock);
  const dim3 grid(static_cast<unsigned>(std::min(groups, kMaxGrid)), p.parts, p.spread);
  auto kernel = ad.R <= 16   ? shrink_kernel<XT, WT, RB, 1>
                : ad.R <= 32 ? shrink_kernel<XT, WT, RB, 2>
                             : shrink_kernel<XT, WT, RB, 4>;
  kernel<<<grid, kAdapterThreads, 0, s>>>(static_cast<const char*>(X), M, C, ad, static_cast<const char*>(W), parts, groups);
  return hipGetLastError();
}

template <int XT, int WT>
hipError_t shrink_any(const void* X, int64_t M, int64_t C, const Adapters& ad, const void* W, float* parts,
                      hipStream_t s) {
  const ShrinkPlan p = shrink_plan(M, C);
  if (few(C)) {
    shrink_short_kernel<XT, WT><<<flat_grid(M * padded_r(ad.R)), kAdapterThreads, 0, s>>>(
        static_cast<const char*>(X), M, C, ad, static_cast<const char*>(W), parts);
    return hipGetLastError();
  }
  return p.blocks == 4 ? shrink_as<XT, WT, 4>(X, M, C, ad, W, parts, p, s)
                       : shrink_as<XT, WT, 1>(X, M, C, ad, W, parts, p, s);
}

template <int WT, int RB>
hipError_t expand_as(const float* parts, const ShrinkPlan& p, const uint16_t* planes, int64_t M, int64_t C,
                     const Adapters& ad, const void* W, float* Y, bool accumulate, float* T, hipStream_t s) {
  constexpr int CW = kExpandCols;
  const int64_t groups = (M + RB * kBlock - 1) / (RB * kBlock);
  const int64_t tiles = (C + kAdapterWaves * 16 * CW - 1) / (kAdapterWaves * 16 * CW), items = groups * tiles;
  const dim3 grid(static_cast<unsigned>(std::min(items, kMaxGrid)), planes ? 1 : expand_spread(p, items));
  const size_t lds = size_t(3) * RB * kBlock * (padded_r(ad.R) + 4) * 2;
  expand_kernel<WT, RB, CW><<<grid, kAdapterThreads, lds, s>>>(parts, p.parts, planes, M, C, ad,
                                                               static_cast<const char*>(W), Y, accumulate, T, items,
                                                               tiles);
  return hipGetLastError();
}

template <int WT>
hipError_t expand_any(const float* parts, uint16_t* planes, int64_t M, int64_t C0, int64_t C, const Adapters& ad,
                      const void* W, float* Y, bool accumulate, float* T, hipStream_t s) {
  const ShrinkPlan p = shrink_plan(M, C0);
  if (few(C) || C > (int64_t(1) << 24)) {
    expand_short_kernel<WT><<<flat_grid(M * C), kAdapterThreads, 0, s>>>(parts, p.parts, M, C, ad,
                                                                 static_cast<const char*>(W), Y, accumulate);
    return T ? launch_join(parts, M, C0, ad, T, nullptr, s) : hipGetLastError();
  }
  // A launch of its own for the planes (5 us) where a workgroup's parts are at least
  // half of the rows of Y that it reads and writes: 2048x4096, 64 ranks in 8 parts
  // 31 us without it and 25 with; 700x4096, 16 ranks in 4 parts 8.4 either way.
  if (p.blocks == 1 || padded_r(ad.R) * p.parts < 256) {
    planes = nullptr;
  } else {
    const hipError_t e = launch_join(parts, M, C0, ad, T, planes, s);
    if (e != hipSuccess) return e;
    T = nullptr;
  }
  return p.blocks == 4 && expand_blocks(M, C) == 2
             ? expand_as<WT, 2>(parts, p, planes, M, C, ad, W, Y, accumulate, T, s)
             : expand_as<WT, 1>(parts, p, planes, M, C, ad, W, Y, accumulate, T, s);
}

template <int XT>
hipError_t grad_as(const float* V, const void* X, int64_t M, int64_t C, const Adapters& ad, float* dW, float* ws,
                   hipStream_t s) {
  if (few(C)) {
    const int64_t n = int64_t(ad.A) * ad.R * C;
    grad_short_kernel<XT><<<static_cast<unsigned>(std::min(n, kMaxGrid)), kAdapterThreads, 0, s>>>(
        V, static_cast<const char*>(X), M, C, ad, dW, n);
    return hipGetLastError();
  }
  const GradPlan p = grad_plan(M, C, ad.A, ad.R);
  const int64_t items = int64_t(p.tiles) * p.groups * ad.A * p.parts;
  const unsigned grid = static_cast<unsigned>(std::min(items, kMaxGrid));
  const bool one = p.parts == 1;
  auto kernel = ad.R <= 16 ? grad_kernel<XT, 1> : ad.R <= 32 ? grad_kernel<XT, 2> : grad_kernel<XT, 4>;
  kernel<<<grid, kAdapterThreads, 0, s>>>(V, static_cast<const char*>(X), M, C, ad, one ? dW : ws, one, p.parts, items, p.tiles,
                                   p.groups);
  if (!one) {
    const int64_t per = int64_t(ad.R) * C, n = per * ad.A;
    grad_join_kernel<<<flat_grid(n), kAdapterThreads, 0, s>>>(ws, p.parts, n, per, ad.scales, dW);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_shrink(const void* X, int x_dtype, int64_t M, int64_t C, const Adapters& ad, const void* W,
                         float* parts, hipStream_t s) {
  if (x_dtype == kF32)
    return ad.w_dtype == kF32 ? shrink_any<kF32, kF32>(X, M, C, ad, W, parts, s)
                              : shrink_any<kF32, kBf16>(X, M, C, ad, W, parts, s);
  return ad.w_dtype == kF32 ? shrink_any<kBf16, kF32>(X, M, C, ad, W, parts, s)
                            : shrink_any<kBf16, kBf16>(X, M, C, ad, W, parts, s);
}

hipError_t launch_expand(const float* parts, uint16_t* planes, int64_t M, int64_t C0, int64_t C, const Adapters& ad,
                         const void* W, float* Y, bool accumulate, float* T, hipStream_t s) {
  return ad.w_dtype == kF32 ? expand_any<kF32>(parts, planes, M, C0, C, ad, W, Y, accumulate, T, s)
                            : expand_any<kBf16>(parts, planes, M, C0, C, ad, W, Y, accumulate, T, s);
}

hipError_t launch_join(const float* parts, int64_t M, int64_t C0, const Adapters& ad, float* T, uint16_t* planes,
                       hipStream_t s) {
  join_kernel<<<flat_grid(M * (padded_r(ad.R) / 4)), kAdapterThreads, 0, s>>>(parts, shrink_plan(M, C0).parts, M, ad, T,
                                                                              planes);
  return hipGetLastError();
}

hipError_t launch_adapter_grad(const float* V, const void* X, int x_dtype, int64_t M, int64_t C, const Adapters& ad,
                               float* dW, float* ws, hipStream_t s) {
  return x_dtype == kF32 ? grad_as<kF32>(V, X, M, C, ad, dW, ws, s) : grad_as<kBf16>(V, X, M, C, ad, dW, ws, s);
}

}  // namespace bitlinear
