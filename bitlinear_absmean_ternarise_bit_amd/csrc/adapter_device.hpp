// Device code that the adapters' kernels share (adapters.hip, adapted_decode.hip):
// operand planes, loads, the tokens of an adapter, and the first product.
#pragma once

#include "adapter_ops.hpp"
#include "block_device.hpp"

namespace bitlinear {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kAdapterThreads = 256, kAdapterWaves = 4;
constexpr int kBlock = 16;      // tokens of a block
constexpr int kExpandCols = 4;  // columns of a lane in expand
constexpr int kGradCols = 4;    // columns of a lane in grad
constexpr int64_t kMaxGrid = int64_t(1) << 20;  // workgroups; each walks every gridDim.x-th item

template <int DT>
constexpr int kPlanes = DT == kF32 ? 3 : 1;

// upper or lower halves of two words, the first one's in the lower half
__device__ __forceinline__ uint32_t upper(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }
__device__ __forceinline__ uint32_t lower(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }

// Planes of two float32, each rounded half to even: what a plane leaves is exact (15
// bits of the value, then 7), at most 2^-8 and 2^-17 of the value's power of two, and
// the third plane holds all of it.  The first one stays finite where the value is.
__device__ __forceinline__ void split(float a, float b, uint32_t (&p)[3]) {
  constexpr float kTop = 338953138925153547590470800371487866880.0f;  // the largest bfloat16
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    p[i] = i == 0 ? bf16_pair(__builtin_amdgcn_fmed3f(a, -kTop, kTop), __builtin_amdgcn_fmed3f(b, -kTop, kTop))
                  : bf16_pair(a, b);
    if (i == 2) break;
    a = __fsub_rn(a, __uint_as_float(p[i] << 16));
    b = __fsub_rn(b, __uint_as_float(p[i] & 0xffff0000u));
  }
}

// CW consecutive values at p, aligned to their type only.
template <int DT, int CW>
struct Some;  // as they lie in memory: CW / 2 words of bfloat16, CW of float32
template <int CW>
struct Some<kF32, CW> {
  uint32_t w[CW];
};
template <int CW>
struct Some<kBf16, CW> {
  uint32_t w[CW / 2];
};
typedef v2u v2u_by2 __attribute__((aligned(2)));
template <int DT, int CW>
__device__ __forceinline__ Some<DT, CW> load_some(const char* p) {
  Some<DT, CW> r;
  if constexpr (DT == kBf16 && CW == 4) {
    const v2u a = *reinterpret_cast<const v2u_by2*>(p);
    r.w[0] = a.x, r.w[1] = a.y;
  } else if constexpr (DT == kBf16) {
    const v4u a = *reinterpret_cast<const v4u_by2*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = a[i];
  } else {
#pragma unroll
    for (int h = 0; h < CW / 4; ++h) {
      const v4u a = *reinterpret_cast<const v4u_by4*>(p + 16 * h);
#pragma unroll
      for (int i = 0; i < 4; ++i) r.w[4 * h + i] = a[i];
    }
  }
  return r;
}

// A lane's CW columns of a row of C >= CW: chunk c, or the row's last CW columns
// where the chunk is cut by the row's end or behind it.  Every load is then whole,
// without a branch, and column j of the lane is its own where j >= `skip` (CW:
// none): each column of the row has one owner.
struct Columns {
  int64_t first;
  int skip;
};
template <int CW>
__device__ __forceinline__ Columns lane_columns(int64_t C, int64_t c) {
  const int64_t over = CW * (c + 1) - C;
  return {over > 0 ? C - CW : CW * c, static_cast<int>(max(int64_t(0), min(over, int64_t(CW))))};
}

// Eight consecutive values of a row as operand planes (shrink).
template <int DT>
__device__ __forceinline__ void row_planes(const Some<DT, 8>& r, bf16x8 (&p)[kPlanes<DT>]) {
  if constexpr (DT == kBf16) {
    p[0] = __builtin_bit_cast(bf16x8, v4u{r.w[0], r.w[1], r.w[2], r.w[3]});
  } else {
    v4u w[3];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t s[3];
      split(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]), s);
#pragma unroll
      for (int q = 0; q < 3; ++q) w[q][i] = s[q];
    }
#pragma unroll
    for (int q = 0; q < 3; ++q) p[q] = __builtin_bit_cast(bf16x8, w[q]);
  }
}

// Four rows of CW columns as the operand planes of each column: element i of
// plane q of column j is row i's (expand, grad: rows are the contraction).
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
template <int DT, int CW>
__device__ __forceinline__ void column_planes(const Some<DT, CW> (&r)[4], s16x4 (&p)[kPlanes<DT>][CW]) {
  if constexpr (DT == kBf16) {
#pragma unroll
    for (int h = 0; h < CW / 2; ++h) {
      p[0][2 * h] = __builtin_bit_cast(s16x4, u32x2{lower(r[0].w[h], r[1].w[h]), lower(r[2].w[h], r[3].w[h])});
      p[0][2 * h + 1] = __builtin_bit_cast(s16x4, u32x2{upper(r[0].w[h], r[1].w[h]), upper(r[2].w[h], r[3].w[h])});
    }
  } else {
#pragma unroll
    for (int j = 0; j < CW; ++j) {
      uint32_t lo[3], hi[3];
      split(__uint_as_float(r[0].w[j]), __uint_as_float(r[1].w[j]), lo);
      split(__uint_as_float(r[2].w[j]), __uint_as_float(r[3].w[j]), hi);
#pragma unroll
      for (int q = 0; q < 3; ++q) p[q][j] = __builtin_bit_cast(s16x4, u32x2{lo[q], hi[q]});
    }
  }
}

// Four float32 as operand planes.
__device__ __forceinline__ void value_planes(const f32x4& v, s16x4 (&p)[3]) {
  uint32_t lo[3], hi[3];
  split(v[0], v[1], lo);
  split(v[2], v[3], hi);
#pragma unroll
  for (int q = 0; q < 3; ++q) p[q] = __builtin_bit_cast(s16x4, u32x2{lo[q], hi[q]});
}

// The adapter of token m0 + lane, -1 for none; `tokens`: those of the group.
__device__ __forceinline__ int token_adapter(const Adapters& ad, int64_t m0, int64_t M, int tokens, int lane) {
  const int64_t m = m0 + lane;
  const int id = lane < tokens && m < M ? ad.rows[m] : -1;
  return id >= 0 && id < ad.A ? id : -1;
}

// Calls f(a, mine) for the adapters of a group of up to 64 tokens, every
// `spread`-th one from `from`: mine has bit t set where token t is a's.  The
// same for all lanes.
template <typename F>
__device__ __forceinline__ void each_adapter(int id, int spread, int from, F&& f) {
  uint64_t todo = __ballot(id >= 0);
  for (int n = 0; todo; ++n) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    const uint64_t mine = __ballot(id == a);
    todo &= ~mine;
    if (n % spread == from) f(a, mine);
  }
}

// ---- shrink ---------------------------------------------------------------------
// A workgroup takes RB blocks of 16 tokens, one part of the columns and every
// spread-th adapter of those tokens; its four waves share the part's columns in
// steps of 32 (v_mfma_f32_16x16x32_bf16: lane l holds token or rank row l % 16,
// columns 8 (l / 16) .. + 7) and add their sums in LDS.  RT tiles of 16 ranks at
// a time.  With RB = 4 a step's rows of W are read, and split into planes, once
// for 64 tokens; with few tokens RB = 1 makes more workgroups.  What bounds it is
// the waves' own loads, two steps of which fit their registers: 2048x4096 bf16
// against 64 rows of float32 13.4 us, where X passes in 3.4 at the rate of a copy.
// first, step: the groups of tokens that the workgroup goes through; part of
// `nparts` parts; from: its first adapter of `spread`.
template <int XT, int WT, int RB, int RT>
__device__ __forceinline__ void shrink_body(const char* X, int64_t M, int64_t C, const Adapters& ad, const char* W,
                                            float* parts, int64_t groups, int64_t first, int64_t step, int part,
                                            int nparts, int from, int spread) {
  __shared__ f32x4 sums[kAdapterWaves][RB * RT][kWave];
  const int wave = wave_id(), lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const int Rp = (ad.R + 15) & ~15;
  const int64_t steps = (C + 31) / 32, whole = C / 32;
  const int64_t q = static_cast<int64_t>(part) * kAdapterWaves + wave, Q = static_cast<int64_t>(nparts) * kAdapterWaves;
  const int64_t lo = q * steps / Q, hi = (q + 1) * steps / Q;
  for (int64_t group = first; group < groups; group += step) {
    const int64_t m0 = group * (RB * kBlock);
    const char* xrow[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) xrow[b] = X + min(m0 + kBlock * b + l, M - 1) * C * kBytes<XT>;
    float* out = parts + (static_cast<int64_t>(part) * M + m0) * Rp;
    each_adapter(token_adapter(ad, m0, M, RB * kBlock, lane), spread, from, [&](int a, uint64_t mine) {
      for (int r0 = 0; r0 < ad.R; r0 += 16 * RT) {
        f32x4 acc[RB][RT];
        const char* wrow[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
#pragma unroll
          for (int b = 0; b < RB; ++b) acc[b][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
          wrow[t] = W + (static_cast<int64_t>(a) * ad.R + min(r0 + 16 * t + l, ad.R - 1)) * C * kBytes<WT>;
        }
        auto add = [&](const Some<XT, 8> (&xr)[RB], const Some<WT, 8> (&wr)[RT]) {
          bf16x8 w[RT][kPlanes<WT>];
#pragma unroll
          for (int t = 0; t < RT; ++t) row_planes<WT>(wr[t], w[t]);
#pragma unroll
          for (int b = 0; b < RB; ++b) {
            bf16x8 x[kPlanes<XT>];
            row_planes<XT>(xr[b], x);
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
              for (int p = 0; p < kPlanes<XT>; ++p)
#pragma unroll
                for (int s = 0; s < kPlanes<WT>; ++s)
                  if (p + s <= 2) acc[b][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[p], w[t][s], acc[b][t], 0, 0, 0);
          }
        };
        auto load = [&](int64_t col, Some<XT, 8> (&xr)[RB], Some<WT, 8> (&wr)[RT]) {
#pragma unroll
          for (int b = 0; b < RB; ++b) xr[b] = load_some<XT, 8>(xrow[b] + col * kBytes<XT>);
#pragma unroll
          for (int t = 0; t < RT; ++t) wr[t] = load_some<WT, 8>(wrow[t] + col * kBytes<WT>);
        };
        const int64_t end = min(hi, whole);
#pragma unroll 2
        for (int64_t st = lo; st < end; ++st) {
          Some<XT, 8> xr[RB];
          Some<WT, 8> wr[RT];
          load(32 * st + 8 * g, xr, wr);
          add(xr, wr);
        }
        if (whole >= lo && whole < hi) {
          // the step that the row's end cuts: columns that are not the lane's own
          // meet zeros (their weights are this row's too: they can make nothing
          // non-finite that is not so anyway)
          const Columns at = lane_columns<8>(C, 4 * whole + g);
          Some<XT, 8> xr[RB];
          Some<WT, 8> wr[RT];
          load(at.first, xr, wr);
#pragma unroll
          for (int b = 0; b < RB; ++b)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if constexpr (XT == kF32) {
                if (j < at.skip) xr[b].w[j] = 0u;
              } else {
                if (j < at.skip) xr[b].w[j / 2] &= j & 1 ? 0x0000ffffu : 0xffff0000u;
              }
            }
          add(xr, wr);
        }
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
          for (int t = 0; t < RT; ++t) sums[wave][b * RT + t][lane] = acc[b][t];
        __syncthreads();
        for (int i = wave; i < RB * RT; i += kAdapterWaves) {
          f32x4 v = sums[0][i][lane];
#pragma unroll
          for (int w = 1; w < kAdapterWaves; ++w) v += sums[w][i][lane];
          const int b = i / RT, r = r0 + 16 * (i - b * RT) + l;
          if (r < Rp) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int token = kBlock * b + 4 * g + k;
              if (mine >> token & 1u) out[static_cast<int64_t>(token) * Rp + r] = r < ad.R ? v[k] : 0.0f;
            }
          }
        }
        __syncthreads();
      }
    });
  }
}

}  // namespace

}  // namespace bitlinear
