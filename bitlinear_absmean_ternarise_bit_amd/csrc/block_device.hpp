// Device helpers of the operators around BitLinear: rows in chunks of eight
// values, the 8-bit saved format, reductions.
//
// Every kernel works on chunks of 8 consecutive columns of a row, one lane to
// a chunk whatever the type (32 bytes of float32, 16 of bfloat16, 8 codes), so
// that a 64-column group of the saved format is 8 neighbouring lanes and its
// largest magnitude comes from three DPP moves.  A row's start need only be
// aligned to its element: gfx950 takes 16-byte accesses at any address, and
// hipcc emits them for the under-aligned vector types below.  The last chunk
// of a row may hold fewer than 8 values.
#pragma once

#include "block_ops.hpp"
#include "common.hpp"

namespace bitlinear {

typedef unsigned v2u __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef v4u v4u_by4 __attribute__((aligned(4)));
typedef v4u v4u_by2 __attribute__((aligned(2)));

template <int DT>
constexpr int kBytes = DT == kF32 ? 4 : DT == kBf16 ? 2 : 1;

// One chunk as it lies in memory.
template <int DT>
struct Raw;
template <>
struct Raw<kF32> {
  v4u a, b;
};
template <>
struct Raw<kBf16> {
  v4u a;
};
template <>
struct Raw<kSaved8> {
  v2u a;
  float scale;
};

// The wave's number in its workgroup, as a scalar: row addresses and per-row
// loads that follow from it stay out of the vector registers.
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6)); }

// Values of chunk c that lie inside a row of K (0 to 8).
__device__ __forceinline__ int chunk_values(int K, int c) { return max(0, min(8, K - 8 * c)); }

// The last n < 8 values of a row, moved down to the front of the chunk and
// followed by zeros, from the row's last 8 values.
__device__ __forceinline__ void move_down(v4u& a, v4u& b, int n) {  // 32-bit values in a, b
  const int by = 8 - n;
  if (by & 4) a = b, b = v4u{0u, 0u, 0u, 0u};
  if (by & 2) a = v4u{a.z, a.w, b.x, b.y}, b = v4u{b.z, b.w, 0u, 0u};
  if (by & 1) a = v4u{a.y, a.z, a.w, b.x}, b = v4u{b.y, b.z, b.w, 0u};
}
__device__ __forceinline__ void move_down(v4u& a, int n) {  // 16-bit values
  const int by = 8 - n;
  if (by & 4) a = v4u{a.z, a.w, 0u, 0u};
  if (by & 2) a = v4u{a.y, a.z, a.w, 0u};
  if (by & 1)
    a = v4u{(a.x >> 16) | (a.y << 16), (a.y >> 16) | (a.z << 16), (a.z >> 16) | (a.w << 16), a.w >> 16};
}

// A row as a buffer resource of `bytes` bytes: what lies behind its end reads as
// zeros and is not written, and an empty one (a row or an array that is not
// there) takes a whole loop's stores without a branch (see fetch_chunk).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_resource(const void* row, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(row), 0, bytes, 0x00020000);
}
constexpr uint32_t kNowhere = 0x80000000u;  // an offset past every resource

// Chunk first + c of a row of a multiple of 8 values, zeros behind it.  `first`
// is the same for a wave's lanes: it moves the resource, and chunks at several
// of them share a lane's offset.
template <int DT>
__device__ __forceinline__ Raw<DT> fetch_whole(const char* row, const float* scales, int K, int cpr, int first, int c) {
  Raw<DT> r;
  const int bytes = (DT == kSaved8 ? cpr * 8 : K * kBytes<DT>) - first * 8 * kBytes<DT>;
  const __amdgpu_buffer_rsrc_t from = row_resource(row + first * 8 * kBytes<DT>, max(bytes, 0));
  if constexpr (DT == kSaved8) {
    r.a = __builtin_amdgcn_raw_buffer_load_b64(from, 8 * c, 0, 0);
    const __amdgpu_buffer_rsrc_t sc = row_resource(scales + (first >> 3), max(cpr - first, 0) / 2);
    r.scale = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(sc, c >> 3 << 2, 0, 0));
  } else if constexpr (DT == kBf16) {
    r.a = __builtin_amdgcn_raw_buffer_load_b128(from, 16 * c, 0, 0);
  } else {
    r.a = __builtin_amdgcn_raw_buffer_load_b128(from, 32 * c, 0, 0);
    r.b = __builtin_amdgcn_raw_buffer_load_b128(from, 32 * c + 16, 0, 0);
  }
  return r;
}

// Chunk c of the row of K >= 8 values at `row` as it lies in memory, for any c.
// `scales`: the row's scales (kSaved8, whose rows are padded with zero codes).
// Nothing is conditional, so a loop that loads its next row ahead waits for
// those loads alone: around a branch with memory operations the compiler waits
// for all that is outstanding, the last row's stores among them.
// WHOLE: K is a multiple of 8; chunks behind the row are zeros.  Else the row's
// end is read as its last 8 values (value by value the loads would wait for one
// another, 4 us a row), and so is a chunk behind it: settle_chunk() before use.
template <int DT, bool WHOLE>
__device__ __forceinline__ Raw<DT> fetch_chunk(const char* row, const float* scales, int K, int cpr, int c) {
  Raw<DT> r;
  if constexpr (WHOLE) {
    r = fetch_whole<DT>(row, scales, K, cpr, 0, c);
  } else if constexpr (DT == kSaved8) {
    const uint32_t at = static_cast<uint32_t>(min(c, cpr - 1));
    r.a = *reinterpret_cast<const v2u*>(row + 8u * at);
    r.scale = *reinterpret_cast<const float*>(reinterpret_cast<const char*>(scales) + 4u * (at >> 3));
  } else if constexpr (DT == kBf16) {
    r.a = *reinterpret_cast<const v4u_by2*>(row + 2u * static_cast<uint32_t>(min(8 * c, K - 8)));
  } else {
    const char* p = row + 4u * static_cast<uint32_t>(min(8 * c, K - 8));
    r.a = *reinterpret_cast<const v4u_by4*>(p);
    r.b = *reinterpret_cast<const v4u_by4*>(p + 16);
  }
  return r;
}

// Waits for a chunk's loads.  Called before a loop that loads ahead: with loads
// outstanding on entry, each turn would wait for everything (the loop's head is
// reached from outside with no stores behind the loads).
__device__ __forceinline__ void arrive(Raw<kF32>& r) { asm volatile("" : "+v"(r.a), "+v"(r.b)); }
__device__ __forceinline__ void arrive(Raw<kBf16>& r) { asm volatile("" : "+v"(r.a)); }
__device__ __forceinline__ void arrive(Raw<kSaved8>& r) { asm volatile("" : "+v"(r.a), "+v"(r.scale)); }

// Puts a fetched chunk's n values in place, zeros behind them.
template <int DT>
__device__ __forceinline__ void settle_chunk(Raw<DT>& r, int n) {
  if (n == 8) return;
  if constexpr (DT == kSaved8) {
    if (n == 0) r.a = v2u{0u, 0u}, r.scale = 0.0f;
  } else if constexpr (DT == kBf16) {
    if (n > 0) move_down(r.a, n);
    else r.a = v4u{0u, 0u, 0u, 0u};
  } else {
    if (n > 0) move_down(r.a, r.b, n);
    else r.a = r.b = v4u{0u, 0u, 0u, 0u};
  }
}

// Chunk c (n values) of the row of K values at `row`, in place.  SHORT: rows of
// fewer than 8 values, which go value by value.
template <int DT, bool SHORT = false>
__device__ __forceinline__ Raw<DT> load_chunk(const char* row, const float* scales, int K, int c, int n) {
  Raw<DT> r;
  if constexpr (DT == kSaved8 || !SHORT) {
    if (n > 0) r = fetch_chunk<DT, false>(row, scales, K, 1 << 30, c);
    settle_chunk<DT>(r, n);
  } else {
    r.a = v4u{0u, 0u, 0u, 0u};
    if constexpr (DT == kF32) r.b = v4u{0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) {
        if constexpr (DT == kBf16)
          r.a[i >> 1] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(row)[i]) << (16 * (i & 1));
        else
          (i < 4 ? r.a : r.b)[i & 3] = reinterpret_cast<const uint32_t*>(row)[i];
      }
  }
  return r;
}

template <int DT>
__device__ __forceinline__ void chunk_f32(const Raw<DT>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (DT == kF32) {
      v[i] = __uint_as_float(i < 4 ? r.a[i & 3] : r.b[i & 3]);
    } else if constexpr (DT == kBf16) {
      v[i] = __uint_as_float((i & 1) ? r.a[i >> 1] & 0xffff0000u : r.a[i >> 1] << 16);
    } else {
      v[i] = r.scale * static_cast<float>(static_cast<int8_t>(r.a[i >> 2] >> (8 * (i & 3))));
    }
  }
}

// Two float32 as packed bfloat16, each rounded half to even.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const f32x2 v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

template <int DT>
__device__ __forceinline__ void store_chunk(char* row, int c, int n, const float (&v)[8]) {
  static_assert(DT != kSaved8, "saved rows are written by save_chunk");
  if constexpr (DT == kBf16) {
    uint16_t* p = reinterpret_cast<uint16_t*>(row) + 8 * c;
    const v4u w = {bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
    if (n == 8) {
      *reinterpret_cast<v4u_by2*>(p) = w;
    } else if (n > 0) {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (i < n) p[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
    }
  } else {
    uint32_t* p = reinterpret_cast<uint32_t*>(row) + 8 * c;
    if (n == 8) {
      *reinterpret_cast<v4u_by4*>(p) = v4u{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                           __float_as_uint(v[3])};
      *reinterpret_cast<v4u_by4*>(p + 4) = v4u{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                                               __float_as_uint(v[7])};
    } else if (n > 0) {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (i < n) p[i] = __float_as_uint(v[i]);
    }
  }
}

// Chunk c (n values) of a row.  WHOLE: chunks are whole or behind the row; else
// a chunk that the row's end cuts goes value by value, the only branch.
template <int DT, bool WHOLE>
__device__ __forceinline__ void put_chunk(__amdgpu_buffer_rsrc_t row, int c, int n, const float (&v)[8]) {
  const uint32_t at = WHOLE || n == 8 ? 8u * kBytes<DT> * c : kNowhere;
  if constexpr (DT == kBf16) {
    const v4u w = {bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
    __builtin_amdgcn_raw_buffer_store_b128(w, row, at, 0, 0);
    if (!WHOLE && n > 0 && n < 8) {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (i < n)
          __builtin_amdgcn_raw_buffer_store_b16(static_cast<short>(w[i >> 1] >> (16 * (i & 1))), row, 16u * c + 2u * i,
                                                0, 0);
    }
  } else {
    const v4u lo = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    const v4u hi = {__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
    __builtin_amdgcn_raw_buffer_store_b128(lo, row, at, 0, 0);
    __builtin_amdgcn_raw_buffer_store_b128(hi, row, at + 16u, 0, 0);
    if (!WHOLE && n > 0 && n < 8) {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (i < n) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[i]), row, 32u * c + 4u * i, 0, 0);
    }
  }
}

template <int CTRL>
__device__ __forceinline__ int dpp_move(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xf, 0xf, false);
}

// The 8-bit form of a chunk (v is 0 past the row's end): its codes and its
// group's scale.  All 8 lanes of a group take part.  |x| is compared as an
// integer, so a NaN is the largest.  x * s is rounded to an integer by one FMA
// with 1.5 * 2^23: the sum has unit spacing and rounds the exact product half to
// even, and its low byte is the code.  No step depends on the order of
// anything: the codes are the same whichever kernel saves.
__device__ __forceinline__ void codes_of(const float (&v)[8], v2u& w, float& scale) {
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  m = max(m, static_cast<unsigned>(dpp_move<0xb1>(static_cast<int>(m))));   // quad_perm 1,0,3,2
  m = max(m, static_cast<unsigned>(dpp_move<0x4e>(static_cast<int>(m))));   // quad_perm 2,3,0,1
  m = max(m, static_cast<unsigned>(dpp_move<0x141>(static_cast<int>(m))));  // row_half_mirror
  const float amax = __uint_as_float(m);
  const bool finite = m < 0x7f800000u;
  const bool live = finite && amax >= 0x1p-100f;
  const float s = live ? __fdiv_rn(127.0f, amax) : 0.0f;
  scale = live ? __fmul_rn(amax, 1.0f / 127.0f) : finite ? 0.0f : __uint_as_float(0x7fc00000u);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = __float_as_uint(__fmaf_rn(v[4 * h + i], s, 12582912.0f));
    // low bytes of q[0], q[1] and q[2], q[3]; selector 12 gives a zero byte
    w[h] = __builtin_amdgcn_perm(q[1], q[0], 0x0c0c0400u) | __builtin_amdgcn_perm(q[3], q[2], 0x04000c0cu);
  }
  if (!finite) w = v2u{0u, 0u};
}

// Saves chunk c of a row: its codes, and by the first lane of each group the
// group's scale.
__device__ __forceinline__ void save_chunk(const float (&v)[8], int8_t* codes, float* scales, int c) {
  v2u w;
  float scale;
  codes_of(v, w, scale);
  *reinterpret_cast<v2u*>(codes + 8 * c) = w;
  if ((c & 7) == 0) scales[c >> 3] = scale;
}
// The same into a row's resources; chunks behind the row fall outside them.
__device__ __forceinline__ void save_chunk(const float (&v)[8], __amdgpu_buffer_rsrc_t codes,
                                           __amdgpu_buffer_rsrc_t scales, int c) {
  v2u w;
  float scale;
  codes_of(v, w, scale);
  __builtin_amdgcn_raw_buffer_store_b64(w, codes, 8u * c, 0, 0);
  __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(scale), scales, (c & 7) == 0 ? c >> 1 : kNowhere, 0, 0);
}

// Sum over a wave, in every lane: within each row of 16 lanes by DPP moves,
// then the four rows' sums, always in the same order.
__device__ __forceinline__ float wave_sum_f32(float v) {
  v += __int_as_float(dpp_move<0xb1>(__float_as_int(v)));
  v += __int_as_float(dpp_move<0x4e>(__float_as_int(v)));
  v += __int_as_float(dpp_move<0x141>(__float_as_int(v)));
  v += __int_as_float(dpp_move<0x140>(__float_as_int(v)));
  const int b = __float_as_int(v);
  return (__int_as_float(__builtin_amdgcn_readlane(b, 0)) + __int_as_float(__builtin_amdgcn_readlane(b, 16))) +
         (__int_as_float(__builtin_amdgcn_readlane(b, 32)) + __int_as_float(__builtin_amdgcn_readlane(b, 48)));
}

// Sums of NV values over a team of W waves of the workgroup, in every lane.
// slot: this reduction's LDS area, W x NV floats of the team's own; two
// consecutive reductions use different slots (a wave that is still reading one
// has not passed the barrier of the next).  Every wave of the workgroup calls.
// Lane i reads wave i % W's sum, and DPP moves add them in every lane.
template <int W, int NV>
__device__ __forceinline__ void team_sum(float (&v)[NV], float* slot, int wave_in_team, int lane) {
  static_assert(W == 1 || W == 2 || W == 4 || W == 8 || W == 16, "waves of a team");
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = wave_sum_f32(v[i]);
  if constexpr (W > 1) {
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) slot[wave_in_team * NV + i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float t = slot[(lane & (W - 1)) * NV + i];
      t += __int_as_float(dpp_move<0xb1>(__float_as_int(t)));
      if constexpr (W >= 4) t += __int_as_float(dpp_move<0x4e>(__float_as_int(t)));
      if constexpr (W >= 8) t += __int_as_float(dpp_move<0x141>(__float_as_int(t)));
      if constexpr (W >= 16) t += __int_as_float(dpp_move<0x140>(__float_as_int(t)));
      v[i] = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(t)));
    }
  }
}

}  // namespace bitlinear
