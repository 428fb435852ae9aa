// bf16 matrix-core GEMM of the backward passes (backward.hip, gated_backward.hip),
// and what its callers share.
#pragma once

#include <type_traits>

#include "block_device.hpp"
#include "kernels.hpp"

namespace bitlinear {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

namespace {

// dYp[m, n] = dY[m, n] for n < N, 0 for N <= n < Np (bf16 bit patterns; Np a
// multiple of 64): a thread to 8 columns, read at any address (2048x4097: value
// by value 20 us, this 7.8).
__global__ __launch_bounds__(256) void pad_rows_bf16_kernel(const uint16_t* __restrict__ src, int64_t M, int64_t N,
                                                            uint16_t* __restrict__ dst, int64_t Np) {
  const int64_t per_row = Np >> 3, total = M * per_row;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t m = i / per_row;
    const int c = static_cast<int>(i - m * per_row), n = chunk_values(static_cast<int>(N), c);
    const char* row = reinterpret_cast<const char*>(src + m * N);
    const Raw<kBf16> r = N >= 8 ? load_chunk<kBf16, false>(row, nullptr, static_cast<int>(N), c, n)
                                : load_chunk<kBf16, true>(row, nullptr, static_cast<int>(N), c, n);
    *reinterpret_cast<v4u*>(dst + 8 * i) = r.a;
  }
}

// Masked store of a finished tile: C[p, q] = acc where bit q of row p of the
// range mask is set, else 0.  The lane holds rows lrow + 32 i + 8 (e / 4) +
// e % 4 and columns lcol + 32 j of the tile.  The tile's mask words go into
// LDS first (every wave is past the last stage's LDS reads): vector-memory
// operations complete in order, so mask loads interleaved with the output
// stores would each wait for the stores before them.  The outputs are written
// nontemporally: they are not read again here, and streaming them evicts less
// of the operand panels that other tiles on this XCD still read.
template <int BM, int BN, int THREADS, int MI, int NI>
__device__ __forceinline__ void store_masked(const f32x16 (&acc)[MI][NI], char* smem, int tid, int lrow, int lcol,
                                             int lr, int64_t p0, int64_t q0, int64_t P, int64_t Q,
                                             float* __restrict__ C, int64_t ldc, const uint32_t* __restrict__ mask,
                                             int64_t kw) {
  constexpr int WPR32 = BN / 32;  // mask words per tile row
  uint32_t* mb = reinterpret_cast<uint32_t*>(smem);
  const int64_t w0 = q0 >> 5;
  for (int idx = tid; idx < BM * WPR32; idx += THREADS) {
    const int row = idx / WPR32, wi = idx % WPR32;
    const int64_t p = p0 + row, w = w0 + wi;
    mb[idx] = (p < P && w < kw) ? mask[p * kw + w] : 0u;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int row = lrow + i * 32 + 8 * (e >> 2) + (e & 3);
      const int64_t p = p0 + row;
      if (p >= P) continue;
      // bit lr of words (row, lcol / 32 + j): columns lcol + 32 j
      const uint32_t* wrow = mb + row * WPR32 + (lcol >> 5);
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const int64_t q = q0 + lcol + j * 32;
        if (q >= Q) continue;
        __builtin_nontemporal_store((wrow[j] >> lr) & 1u ? acc[i][j][e] : 0.0f, C + p * ldc + q);
      }
    }
}

// bf16 MFMA GEMM, C[p, q] = sum_r A[p, r] B[q, r] over r < Rp (a multiple of 64).
// A: bf16 [P, Rp] with row stride lda >= Rp; rows 16-byte aligned.  B: bf16 [Q, Rp]
// (BMODE 0) or the 2-bit ternary codes of a [Q, Rp] matrix in the packed
// format (BMODE 1), expanded to bf16 c - 1.  BMODE 2: packed, and A's rows hold
// lda < Rp columns (a multiple of 8): what lies past a row's end is read as
// zeros, since the next row's infinities and NaN must not meet the padding
// codes' zero weights.  (In the same kernel the comparison cost whole rows 1 to
// 2%: 17x2048 over 5632 68.2 us and 69.5.)
// EPI 2: the sum of two products of the same shapes, gamma (A B^T) + gamma2
// (A2 B2^T): the stages of the second follow those of the first without a
// break, and the first one's accumulators are scaled and put by in between (64
// more registers a lane with 256 x 128 tiles).  Of each product the stages
// first .. first + count - 1 are taken.
// EPI 0: C * gamma;  EPI 1: C where bit q of row p of the range mask is set
// (mask: rows of kw 32-bit words, bit q % 32 of word q / 32), else 0.
//
// Tile BM x BN, WM x WN waves each owning (BM/WM) x (BN/WN) (64 or 128 rows)
// of 32 x 32 MFMA tiles; 64 r per LDS stage, two stages.  Global loads run two
// stages ahead into two register sets, and the next stage is written to LDS
// halfway through the contraction of the current one, so one barrier per
// stage suffices and the matrix cores keep working while loads are in flight.
// Operand rows of a stage are 128 bytes with 16-byte slot c of row r stored at
// slot c ^ ((r >> 1) & 7): the 16 lanes one LDS cycle serves (16 consecutive
// rows, same slot) hit distinct bank groups of the 64-bank LDS.
struct SecondProduct {
  const uint16_t* A;
  const void* B;
  const float* gamma;
  int first, count;
};

template <int BM, int BN, int WM, int WN, int BMODE, int EPI>
__device__ __forceinline__ void bf16_gemm_nt_body(
    const uint16_t* __restrict__ A, int64_t P, int64_t lda, const void* __restrict__ B, int64_t Q, int64_t Rp,
    float* __restrict__ C, int64_t ldc, const float* __restrict__ gamma, const uint32_t* __restrict__ mask,
    int64_t kw, int bytes_a, int bytes_b, int tiles_p, int tiles_q, const SecondProduct& second) {
  constexpr int BK = 64;
  constexpr int ROWB = BK * 2;
  constexpr int THREADS = 64 * WM * WN;
  constexpr int A_BYTES = BM * ROWB;
  constexpr int STAGE = A_BYTES + BN * ROWB;
  constexpr int WROWS = BM / WM;  // rows of a wave's tile
  constexpr int MI = WROWS / 32, NI = BN / WN / 32;
  constexpr int A_LOADS = BM * 8 / THREADS;
  constexpr int B_LOADS = BMODE == 0 ? BN * 8 / THREADS : BN * 4 / THREADS;  // 16-byte slots, or packed words
  static_assert((WROWS == 64 || WROWS == 128) && A_LOADS >= 1 && B_LOADS >= 1 && NI >= 1, "tile shape");
  static_assert(BMODE == 0 || (B_LOADS <= 4 && BN * 4 == B_LOADS * THREADS), "packed B: whole words per thread");
  __shared__ __align__(1024) char smem[2 * STAGE];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = tid >> 6;
  const int wm = wave / WN, wn = wave % WN;

  // Workgroup -> tile: each XCD (workgroups are dealt round-robin to the 8
  // XCDs) gets a contiguous run of tiles, walked in groups of 8 tile rows so
  // resident tiles share operand panels in the XCD's L2.
  const int num_tiles = tiles_p * tiles_q;
  int t = blockIdx.x;
  if (num_tiles % 8 == 0) t = (t & 7) * (num_tiles >> 3) + (t >> 3);
  constexpr int GROUP = 8;
  const int group = t / (GROUP * tiles_q);
  const int first_p = group * GROUP;
  const int gsize = min(tiles_p - first_p, GROUP);
  const int in_group = t - group * GROUP * tiles_q;
  const int64_t p0 = static_cast<int64_t>(first_p + in_group % gsize) * BM;
  const int64_t q0 = static_cast<int64_t>(in_group / gsize) * BN;

  const int half = EPI == 2 ? second.count : static_cast<int>(Rp / BK);  // stages of a product
  const int niter = EPI == 2 ? 2 * half : half;
  const uint32_t rowbytes = static_cast<uint32_t>(Rp) * 2u;
  const uint32_t rowbytes_a = static_cast<uint32_t>(lda) * 2u;

  const __amdgpu_buffer_rsrc_t rsrc_a =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(A), 0, bytes_a, 0x00020000);
  const __amdgpu_buffer_rsrc_t rsrc_b =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(B), 0, bytes_b, 0x00020000);
  constexpr uint32_t kOff = 0x80000000u;  // past every resource: reads zeros

  // operand slot s = tid + THREADS i: row s / 8, logical slot s % 8
  uint32_t a_off[A_LOADS], a_dst[A_LOADS];
#pragma unroll
  for (int i = 0; i < A_LOADS; ++i) {
    const int s = tid + THREADS * i, r = s >> 3, c = s & 7;
    a_off[i] = (p0 + r < P) ? static_cast<uint32_t>(p0 + r) * rowbytes_a + 16u * c : kOff;
    a_dst[i] = r * ROWB + 16 * (c ^ ((r >> 1) & 7));
  }
  const int a_end = static_cast<int>(rowbytes_a) - 16 * (tid & 7);  // (BMODE 2) offsets within a row end here
  uint32_t b_off[B_LOADS], b_dst[B_LOADS];
  if constexpr (BMODE == 0) {
#pragma unroll
    for (int i = 0; i < B_LOADS; ++i) {
      const int s = tid + THREADS * i, r = s >> 3, c = s & 7;
      b_off[i] = (q0 + r < Q) ? static_cast<uint32_t>(q0 + r) * rowbytes + 16u * c : kOff;
      b_dst[i] = A_BYTES + r * ROWB + 16 * (c ^ ((r >> 1) & 7));
    }
  }
  // packed B: word s % 4 of row s / 4's unit (16 codes, two 16-byte slots of
  // bf16) for s = tid + THREADS i, so the expansion is spread over every wave
  const uint32_t units = static_cast<uint32_t>(Rp >> 6);
  const int pb_w = tid & 3;

  v4u ra[2][A_LOADS], rb[2][BMODE == 0 ? B_LOADS : 1];  // packed B: word i in element i
  auto gload_from = [&](__amdgpu_buffer_rsrc_t rsrc_a, __amdgpu_buffer_rsrc_t rsrc_b, int it, auto set_tag) {
    constexpr int S = decltype(set_tag)::value;
    // (a thread's slots are the same 8 columns of different rows; sums of two offsets
    // past the resource stay past it)
    const uint32_t at = 128u * it, to = static_cast<int>(at) >= a_end ? kOff : at;
#pragma unroll
    for (int i = 0; i < A_LOADS; ++i) {
      const uint32_t off = BMODE == 2 ? __builtin_elementwise_add_sat(a_off[i], to) : a_off[i] == kOff ? kOff : a_off[i] + at;
      ra[S][i] = __builtin_amdgcn_raw_buffer_load_b128(rsrc_a, off, 0, 0);
    }
    if constexpr (BMODE == 0) {
#pragma unroll
      for (int i = 0; i < B_LOADS; ++i)
        rb[S][i] =
            __builtin_amdgcn_raw_buffer_load_b128(rsrc_b, b_off[i] == kOff ? kOff : b_off[i] + 128u * it, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < B_LOADS; ++i) {
        const int r = (tid + THREADS * i) >> 2;
        const uint32_t off = q0 + r < Q ? unit_offset(static_cast<uint32_t>(q0 + r), static_cast<uint32_t>(it),
                                                      static_cast<uint32_t>(Q), units) + 4u * pb_w
                                        : kOff;
        rb[S][0][i] = __builtin_amdgcn_raw_buffer_load_b32(rsrc_b, off, 0, 0);
      }
    }
  };
  auto gload = [&](int it, auto set_tag) {
    if constexpr (EPI == 2) {
      const bool two = it >= half;
      gload_from(__builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(two ? second.A : A), 0, bytes_a, 0x00020000),
                 __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(two ? second.B : B), 0, bytes_b, 0x00020000),
                 second.first + (two ? it - half : it), set_tag);
    } else {
      gload_from(rsrc_a, rsrc_b, it, set_tag);
    }
  };
  auto swrite = [&](char* st, auto set_tag) {
    constexpr int S = decltype(set_tag)::value;
#pragma unroll
    for (int i = 0; i < A_LOADS; ++i) *reinterpret_cast<v4u*>(st + a_dst[i]) = ra[S][i];
    if constexpr (BMODE == 0) {
#pragma unroll
      for (int i = 0; i < B_LOADS; ++i) *reinterpret_cast<v4u*>(st + b_dst[i]) = rb[S][i];
    } else {
      // 16 codes -> 16 bf16 values c - 1 through two byte tables (v_perm):
      // high bytes {0xBF, 0x00, 0x3F} and low bytes {0x80, 0x00, 0x80} for c = 0, 1, 2
      constexpr uint32_t kHi = 0x003F00BFu, kLo = 0x00800080u;
#pragma unroll
      for (int i = 0; i < B_LOADS; ++i) {
        const int r = (tid + THREADS * i) >> 2;
        char* sb = st + A_BYTES + r * ROWB;
        const uint32_t w = rb[S][0][i];
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {  // slot c = 2 pb_w + cc: k = 8c .. 8c + 7, fields i = 2 cc, 2 cc + 1
          const int c = 2 * pb_w + cc;
          v4u out;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x = (w >> (2 * (2 * cc + h))) & 0x03030303u;
            const uint32_t hi = __builtin_amdgcn_perm(0u, kHi, x);
            const uint32_t lo = __builtin_amdgcn_perm(0u, kLo, x);
            out[2 * h] = __builtin_amdgcn_perm(hi, lo, 0x05010400u);
            out[2 * h + 1] = __builtin_amdgcn_perm(hi, lo, 0x07030602u);
          }
          *reinterpret_cast<v4u*>(sb + 16 * (c ^ ((r >> 1) & 7))) = out;
        }
      }
    }
  };

  f32x16 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  const int lr = lane & 31, lh = lane >> 5;
  // LDS byte offsets of this lane's operands for k step ks of a stage (slot
  // 2 ks + lh of its row); tile mi / ni adds 32 rows = 4096 bytes
  int a_rd[4], b_rd[4];
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    const int sw = 16 * ((2 * ks + lh) ^ ((lr >> 1) & 7));
    a_rd[ks] = (wm * WROWS + lr) * ROWB + sw;
    b_rd[ks] = A_BYTES + (wn * (BN / WN) + lr) * ROWB + sw;
  }
  auto contract_half = [&](const char* st, int hs) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const int ks = 2 * hs + kk;
      bf16x8 a[MI], b[NI];
#pragma unroll
      for (int i = 0; i < MI; ++i) a[i] = *reinterpret_cast<const bf16x8*>(st + a_rd[ks] + i * 32 * ROWB);
#pragma unroll
      for (int j = 0; j < NI; ++j) b[j] = *reinterpret_cast<const bf16x8*>(st + b_rd[ks] + j * 32 * ROWB);
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
    }
  };

  using S0 = std::integral_constant<int, 0>;
  using S1 = std::integral_constant<int, 1>;
  // prologue: stage 0 -> LDS 0; stage 1 in register set 1; stage 2 loading into set 0
  gload(0, S0());
  gload(min(1, niter - 1), S1());
  swrite(smem, S0());
  gload(min(2, niter - 1), S0());
  __syncthreads();

  // Iteration it contracts LDS stage it % 2; halfway it writes stage it + 1
  // (register set (it + 1) % 2, loaded two iterations earlier) into the other
  // LDS stage and reloads that register set with stage it + 3 (past the last
  // stage: the last stage again, written to the idle LDS stage, harmless).
  f32x16 first[EPI == 2 ? MI : 1][NI];  // (EPI 2) the first product
  auto iteration = [&](int it, auto set_tag) {
    if constexpr (EPI == 2) {
      if (it == half) {
        const float g = gamma[0];
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              first[i][j][e] = __fmul_rn(acc[i][j][e], g);
              acc[i][j][e] = 0.0f;
            }
      }
    }
    const char* cur = smem + (it & 1) * STAGE;
    char* nxt = smem + ((it + 1) & 1) * STAGE;
    contract_half(cur, 0);
    swrite(nxt, set_tag);
    gload(min(it + 3, niter - 1), set_tag);
    contract_half(cur, 1);
    __syncthreads();
  };
  int it = 0;
  for (; it + 1 < niter; it += 2) {
    iteration(it, S1());
    iteration(it + 1, S0());
  }
  if (it < niter) iteration(it, S1());

  // epilogue: lane holds rows 8 (e / 4) + 4 lh + e % 4, column lr of each
  // 32 x 32 tile.  The lane's first row and column are opaque to the
  // compiler, so it does not compute the output addresses before the main
  // loop and keep them live (spilled) across it.  The outputs are written
  // nontemporally (see store_masked).
  int lrow = wm * WROWS + 4 * lh;
  int lcol = wn * (BN / WN) + lr;
  asm volatile("" : "+v"(lrow), "+v"(lcol));
  if constexpr (EPI == 0 || EPI == 2) {
    const float g = EPI == 2 ? second.gamma[0] : gamma[0];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int64_t p = p0 + lrow + i * 32 + 8 * (e >> 2) + (e & 3);
        if (p >= P) continue;
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          const int64_t q = q0 + lcol + j * 32;
          float v = __fmul_rn(acc[i][j][e], g);
          if constexpr (EPI == 2) v = __fadd_rn(first[i][j][e], v);
          if (q < Q) __builtin_nontemporal_store(v, C + p * ldc + q);
        }
      }
  } else {
    store_masked<BM, BN, THREADS, MI, NI>(acc, smem, tid, lrow, lcol, lr, p0, q0, P, Q, C, ldc, mask, kw);
  }
}

}  // namespace

}  // namespace bitlinear
