// Gated hidden layer H = act(X W_gate^T) * (X W_up^T) over ternary weights
// (include/bitlinear_gated.h): the INT8-MFMA GEMM with both projections in one
// tile (prefill_gemm.hpp, EPI 3), and a decode kernel for up to 16 tokens.
// 2048x4096x11008: 187 us, 1.97 POPS; 8192x8192x28672: 2.76 ms, 2.79 POPS, where the
// library's int8 product of 8192^3 reaches 2.64: the matrix cores and their clock.
#include <algorithm>

#include "gated_ops.hpp"
#include "prefill_gemm.hpp"
#include "quant_act.hpp"

namespace bitlinear {

namespace {

template <int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 1) void gated_gemm_kernel(
    const int8_t* __restrict__ Xq, const float* __restrict__ gamma_a, const int32_t* __restrict__ rowsum, int64_t M,
    int64_t Kp, const uint32_t* __restrict__ packed_gate, int64_t N, int64_t ldy, const float* __restrict__ gamma_gate,
    int tiles_m, int tiles_n, int bytes_a, int bytes_b, GatedOut go) {
  prefill_gemm_body<BM, BN, WM, WN, 3>(Xq, gamma_a, rowsum, M, Kp, packed_gate, N, ldy, gamma_gate, nullptr, nullptr,
                                       tiles_m, tiles_n, bytes_a, bytes_b, go, AdapterOut{});
}

constexpr int64_t kCUs = 256;

void* moved(void* p, int dtype, int64_t n) {
  return p ? static_cast<char*>(p) + n * (dtype == kF32 ? 4 : 2) : nullptr;
}

// Columns [n0, n0 + N) of the hidden layer.
template <int BM, int BN, int WM, int WN>
hipError_t launch_tile(const int8_t* Xq, const float* ga, const int32_t* rs, int64_t M, int64_t Kp,
                       const GatedWeights& w, int64_t n0, int64_t N, int64_t ldy, const GatedOutputs& o,
                       hipStream_t stream) {
  // buffer offsets are 32-bit: the tokens go in chunks of < 2^31 code bytes
  const int64_t chunk = ((int64_t(1) << 31) - 1) / Kp / BM * BM;
  const int bytes_b = static_cast<int>(N * (Kp / 4));
  const int64_t words = n0 * (Kp / 16);  // n0 is a multiple of 16: whole blocks of the packed order
  for (int64_t r0 = 0; r0 < M; r0 += chunk) {
    const int64_t Mc = std::min(M - r0, chunk);
    const int tiles_m = static_cast<int>((Mc + BM - 1) / BM);
    const int tiles_n = static_cast<int>((N + BN / 2 - 1) / (BN / 2));
    // persistent workgroups, one to a CU
    const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(int64_t(tiles_m) * tiles_n, kCUs));
    const int64_t at = r0 * ldy + n0;
    const GatedOut go = {w.up + words, w.gamma_up, moved(o.H, o.h_dtype, at), moved(o.G, o.gu_dtype, at),
                         moved(o.U, o.gu_dtype, at), w.act, o.h_dtype, o.gu_dtype};
    gated_gemm_kernel<BM, BN, WM, WN><<<blocks, 64 * WM * WN, 0, stream>>>(
        Xq + r0 * Kp, ga + r0, rs + r0, Mc, Kp, w.gate + words, N, ldy, w.gamma_gate, tiles_m, tiles_n,
        static_cast<int>(Mc * Kp), bytes_b, go);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// ---- decode: up to 16 tokens --------------------------------------------------
//
// A workgroup of eight waves takes blocks of 16 hidden columns.  Waves 0 to 3
// stream the block's gate rows, each a quarter of K, waves 4 to 7 its up rows,
// as one contiguous KiB a load instruction (the packed format's row order), and
// contract them with the tokens' codes in LDS by v_mfma_i32_16x16x64_i8 (lane l:
// token l % 16 against weight row l % 16, the same 16 k, as in the decode
// forward).  The exact INT32 partial sums meet in LDS, and one wave, another one
// for each block, adds them, forms act(g) * u and writes it.
//
// 1x2048x5632 6.6 us, 8 tokens 9.0: 5.8 MB of weights take 1.2 at the rate of a copy,
// an empty kernel 1.3; the rest is one memory latency after another (the tokens,
// the weights, the sums through LDS), which is why all loads start before any wait.
//
// The tokens are quantised once by each workgroup, while its first weights are
// on their way, and a workgroup walks every gridDim.x-th block with the next
// batch of loads in flight.
constexpr int kGatedThreads = 512, kGatedWaves = 8, kQuarters = 4;
constexpr int kBatch = 4;        // loads a lane and batch
constexpr int kRowChunks = 4;    // 16-byte chunks a lane of a token row that is loaded ahead
constexpr int64_t kGatedGrid = 512;
constexpr size_t kGatedSums = 2 * kGatedWaves * kWave * sizeof(v4i);  // two blocks' partial sums

// One token whose row a wave holds in registers: every wave quantises just the
// quarter that it contracts and waits for nobody.
__host__ __device__ inline bool own_quarter(int DT, bool vec, int64_t M, int64_t K) {
  return DT != 2 && vec && M == 1 && K / (DT == 0 ? 4 : 8) <= kRowChunks * kWave;
}

// DT: 0 = float32 tokens, 1 = bfloat16 tokens, 2 = codes with ga_in and rs_in
template <int DT, bool VEC>
__global__ __launch_bounds__(kGatedThreads) void gated_decode_kernel(const void* __restrict__ X, int M, int64_t K,
                                                                     int64_t Kp, GatedWeights w, int64_t N,
                                                                     GatedOutputs out,
                                                                     const float* __restrict__ ga_in,
                                                                     const int32_t* __restrict__ rs_in, int blocks) {
  extern __shared__ __align__(16) int8_t sxq[];
  __shared__ float s_ga[kDecodeMaxM];
  __shared__ int s_rs[kDecodeMaxM];
  constexpr int esize = DT == 0 ? 4 : DT == 1 ? 2 : 1;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int lane = threadIdx.x & (kWave - 1), j = lane & 15, g = lane >> 4;
  const int matrix = wave / kQuarters, quarter = wave % kQuarters;
  const int64_t stride = Kp + 16;  // +16: token rows start on different banks
  const uint32_t units = static_cast<uint32_t>(Kp >> 6), N32 = static_cast<uint32_t>(N);
  const int chunks = static_cast<int>((units + 3) >> 2);  // load instructions of a block of rows
  const int c_lo = quarter * chunks / kQuarters, c_hi = (quarter + 1) * chunks / kQuarters;
  const int per_block = ((chunks + kQuarters - 1) / kQuarters + kBatch - 1) / kBatch;  // batches, the same for all waves
  const int my_blocks = (blocks - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
  const int batches = my_blocks * per_block;

  // Loads are unconditional: what must not be read (rows past N, units past a
  // row's end, chunks of another quarter, batches past the last) is at an offset
  // past the resource and comes back as zeros.
  const __amdgpu_buffer_rsrc_t wsrc = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint32_t*>(matrix ? w.up : w.gate), 0, static_cast<int>(N * (Kp / 4)), 0x00020000);
  auto load_batch = [&](int b, uint4 (&r)[kBatch]) {
    const int i = b / per_block, cb = b - i * per_block;
    const uint32_t n0 = 16u * (blockIdx.x + static_cast<uint32_t>(i) * gridDim.x);
    const uint32_t R = N32 > n0 ? min(16u, N32 - n0) : 0u;  // rows of the block
    const bool row_ok = b < batches && static_cast<uint32_t>(j) < R;
    const uint32_t base = n0 * units * 16u;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int cs = c_lo + cb * kBatch + u;
      const uint32_t un = static_cast<uint32_t>(cs) * 4u + g;
      const uint32_t W = min(4u, units - min(units, 4u * cs));  // units of the chunk
      const bool ok = row_ok && cs < c_hi && un < units;
      const uint32_t off = ok ? base + (cs * R * 4u + j * W + g) * 16u : 0xfffffff0u;
      const v4u v = __builtin_amdgcn_raw_buffer_load_b128(wsrc, off, 0, 2);  // 2: streaming, every byte is used once
      r[u] = make_uint4(v[0], v[1], v[2], v[3]);
    }
  };

  const bool alone = own_quarter(DT, VEC, M, K);
  int8_t* codes = sxq + (alone ? matrix * stride : 0);
  v4i* sums = reinterpret_cast<v4i*>(sxq + (alone ? 2 : M) * stride);
  const char* xb = static_cast<const char*>(X);
  const int64_t xnc = K / (DT == 0 ? 4 : 8);
  const bool early = DT != 2 && VEC && xnc <= kRowChunks * kWave;
  uint4 xv[kRowChunks], buf0[kBatch], buf1[kBatch];
  if constexpr (DT != 2 && VEC) {
    if (early) load_row_chunks<DT, kRowChunks>(xb + (wave < M ? wave : 0) * K * esize, xnc, lane, xv);
  }
  load_batch(0, buf0);
  const float gm_gate = w.gamma_gate[0], gm_up = w.gamma_up[0];
  __builtin_amdgcn_sched_barrier(0);

  int own_sum = 0;  // (alone) code sum of the wave's quarter
  if constexpr (DT == 2) {
    const uint4* src = static_cast<const uint4*>(X);
    const int per_row = static_cast<int>(Kp >> 4), total = M * per_row;
    for (int i0 = threadIdx.x; i0 < total; i0 += 4 * kGatedThreads) {
      uint4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = src[min(i0 + u * kGatedThreads, total - 1)];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * kGatedThreads, m = i / per_row;
        if (i < total) *reinterpret_cast<uint4*>(codes + m * stride + 16 * (i - m * per_row)) = v[u];
      }
    }
    if (threadIdx.x < M) {
      s_ga[threadIdx.x] = ga_in[threadIdx.x];
      s_rs[threadIdx.x] = rs_in[threadIdx.x];
    }
  } else {
    int m = wave;
    float ga = 0.0f;
    int rs = 0;
    if constexpr (VEC) {
      if (alone) {
        constexpr int P = ActTraits<DT>::kPerChunk;
        float mx = 0.0f;
#pragma unroll
        for (int u = 0; u < kRowChunks; ++u) {
          float f[P];
          chunk_to_f32<DT>(xv[u], f);
          float mu = 0.0f;
#pragma unroll
          for (int i = 0; i < P; ++i) mu = fmaxf(mu, fabsf(f[i]));
          mx = lane + u * kWave < xnc ? fmaxf(mx, mu) : mx;
        }
        mx = quant_wave_max(mx);
        const float sc = __fdiv_rn(127.0f, __fadd_rn(mx, kEps));
        const int64_t k_lo = int64_t(256) * c_lo, k_hi = min(int64_t(256) * c_hi, Kp);
        int sum = 0;
#pragma unroll
        for (int u = 0; u < kRowChunks; ++u) {
          const int64_t c = lane + u * kWave;
          if (c < xnc && c * P >= k_lo && c * P < k_hi) sum += quantize_chunk<DT>(xv[u], sc, codes + c * P);
        }
        for (int64_t k = max(K, k_lo) + lane; k < k_hi; k += kWave) codes[k] = 0;
        own_sum = quant_wave_sum(sum);
        if (wave == 0 && lane == 0) {
          s_ga[0] = mx;
          s_rs[0] = 0;  // the waves subtract their own
        }
        m = M;
      } else if (early) {
        if (wave < M) {
          quantize_loaded_row<DT, kRowChunks>(xv, xnc, K, Kp, lane, codes + wave * stride, ga, rs);
          if (lane == 0) s_ga[wave] = ga, s_rs[wave] = rs;
        }
        m += kGatedWaves;
      }
    }
    for (; m < M; m += kGatedWaves) {
      quantize_row_wave<DT, VEC>(xb + m * K * esize, K, Kp, lane, codes + m * stride, ga, rs);
      if (lane == 0) s_ga[m] = ga, s_rs[m] = rs;
    }
  }
  if (alone)
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // a wave reads only the codes that it wrote
  else
    __syncthreads();

  // lanes of tokens past M read token 0's codes: they feed sums that are not stored
  const int8_t* arow = codes + (j < M ? j : 0) * stride;
  const v4i zero = {0, 0, 0, 0};
  v4i c = zero;
  auto contract = [&](int b, const uint4 (&r)[kBatch]) {
    const int cb = b % per_block;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int cs = c_lo + cb * kBatch + u;
      const uint32_t un = static_cast<uint32_t>(cs) * 4u + g;
      // slots that were loaded as zeros may meet any codes in bounds
      const uint32_t at = un < units ? 64u * un : 0u;
      const uint32_t wd[4] = {r[u].x, r[u].y, r[u].z, r[u].w};
#pragma unroll
      for (int t = 0; t < 4; ++t)
        c = __builtin_amdgcn_mfma_i32_16x16x64_i8(*reinterpret_cast<const v4i*>(arow + at + 16u * t), unpack_word(wd[t]),
                                                  c, 0, 0, 0);
    }
  };
  // After a block's last batch.  The sums of two blocks in turn have areas of
  // their own, so one barrier a block suffices: a wave that writes an area again
  // has passed the barrier of the block in between, and so has its reader.
  auto finish = [&](int b) {
    const int i = b / per_block;
    if (b - i * per_block != per_block - 1) return;
    v4i* area = sums + (i & 1) * kGatedWaves * kWave;
    if (alone && g == 0) c[0] -= own_sum;  // lanes 0 to 15 hold token 0
    area[threadIdx.x] = c;
    c = zero;
    __syncthreads();
    if ((i & (kGatedWaves - 1)) != wave) return;
    v4i vg = area[lane], vu = area[kQuarters * kWave + lane];
#pragma unroll
    for (int q = 1; q < kQuarters; ++q) {
      vg += area[q * kWave + lane];
      vu += area[(kQuarters + q) * kWave + lane];
    }
    const uint32_t n = 16u * (blockIdx.x + static_cast<uint32_t>(i) * gridDim.x) + j;
    if (n >= N32) return;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int m = 4 * g + r;
      if (m >= M) continue;
      const float ga = s_ga[m];
      const int rs = s_rs[m];
      const float gate = __fmul_rn(static_cast<float>(vg[r] - rs), __fdiv_rn(__fmul_rn(gm_gate, ga), 127.0f));
      const float up = __fmul_rn(static_cast<float>(vu[r] - rs), __fdiv_rn(__fmul_rn(gm_up, ga), 127.0f));
      const int64_t at = static_cast<int64_t>(m) * N + n;
      store_one(out.H, out.h_dtype, at, gated_value(w.act, gate, up));
      if (out.G) {
        store_one(out.G, out.gu_dtype, at, gate);
        store_one(out.U, out.gu_dtype, at, up);
      }
    }
  };

  load_batch(1, buf1);
  __builtin_amdgcn_sched_barrier(0);
  int b = 0;
  for (; b + 1 < batches; b += 2) {
    contract(b, buf0);
    load_batch(b + 2, buf0);
    __builtin_amdgcn_sched_barrier(0);
    finish(b);
    contract(b + 1, buf1);
    load_batch(b + 3, buf1);
    __builtin_amdgcn_sched_barrier(0);
    finish(b + 1);
  }
  if (b < batches) {
    contract(b, buf0);
    finish(b);
  }
}

template <int DT, bool VEC>
hipError_t launch_decode_as(const void* X, const float* ga, const int32_t* rs, int64_t M, int64_t D, int64_t F,
                            const GatedWeights& w, const GatedOutputs& o, hipStream_t stream) {
  const int64_t Kp = padded_k(D), blocks = (F + 15) / 16;
  const size_t lds = static_cast<size_t>((own_quarter(DT, VEC, M, D) ? 2 : M) * (Kp + 16)) + kGatedSums;
  gated_decode_kernel<DT, VEC><<<static_cast<unsigned>(std::min(blocks, kGatedGrid)), kGatedThreads, lds, stream>>>(
      X, static_cast<int>(M), D, Kp, w, F, o, ga, rs, static_cast<int>(blocks));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gated_gemm(const int8_t* Xq, const float* ga, const int32_t* rs, int64_t M, int64_t D, int64_t F,
                             const GatedWeights& w, const GatedOutputs& o, hipStream_t stream) {
  const int64_t Kp = padded_k(D);
  // Tiles of 256 tokens x 128 columns (of both projections), 128 x 128 or 128 x 64.
  // A round of the largest takes 1.75 times as long as one of the middle ones
  // (4096 columns of X: 46 us and 27; K and the rest do not matter), and one of
  // the smallest is no faster than the middle (25): those serve where even they
  // are one round (17x2048x5632 12.7 us, middle 14.2).  Else the fewest rounds so
  // weighed: 333x8192x28672 153 us with the middle tile, 172 with the largest;
  // 300x4096x11008 54 and 50; 2048x4096x11008 183 and 165.  Whole rounds of the
  // largest and then one round of middle tiles for the last columns are a third
  // way (1024x4096x11008: 89, 94 and 102).
  auto tiles = [&](int64_t bm, int64_t bn) { return ((M + bm - 1) / bm) * ((F + bn - 1) / bn); };
  auto rounds = [&](int64_t n) { return (n + kCUs - 1) / kCUs; };
  if (tiles(128, 64) <= kCUs) return launch_tile<128, 128, 2, 2>(Xq, ga, rs, M, Kp, w, 0, F, F, o, stream);
  const int64_t large = 7 * rounds(tiles(256, 128)), middle = 4 * rounds(tiles(128, 128));
  const int64_t whole = tiles(256, 128) / kCUs, per_column = (M + 255) / 256;  // per column of tiles
  const int64_t n = whole * kCUs / per_column * 128;  // columns of whole rounds of the largest
  if (n > 0 && n < F && (M + 127) / 128 * ((F - n + 127) / 128) <= kCUs && 7 * whole + 4 < std::min(large, middle)) {
    const hipError_t e = launch_tile<256, 256, 4, 2>(Xq, ga, rs, M, Kp, w, 0, n, F, o, stream);
    return e != hipSuccess ? e : launch_tile<128, 256, 2, 4>(Xq, ga, rs, M, Kp, w, n, F - n, F, o, stream);
  }
  if (middle < large) return launch_tile<128, 256, 2, 4>(Xq, ga, rs, M, Kp, w, 0, F, F, o, stream);
  return launch_tile<256, 256, 4, 2>(Xq, ga, rs, M, Kp, w, 0, F, F, o, stream);
}

hipError_t launch_gated_decode(const void* X, int x_dtype, const int8_t* Xq, const float* ga, const int32_t* rs,
                               int64_t M, int64_t D, int64_t F, const GatedWeights& w, const GatedOutputs& o,
                               hipStream_t stream) {
  if (!X) return launch_decode_as<2, true>(Xq, ga, rs, M, D, F, w, o, stream);
  const int esize = x_dtype == kF32 ? 4 : 2;
  const bool vec = reinterpret_cast<uintptr_t>(X) % 16 == 0 && (D * esize) % 16 == 0;
  if (x_dtype == kF32)
    return vec ? launch_decode_as<0, true>(X, nullptr, nullptr, M, D, F, w, o, stream)
               : launch_decode_as<0, false>(X, nullptr, nullptr, M, D, F, w, o, stream);
  return vec ? launch_decode_as<1, true>(X, nullptr, nullptr, M, D, F, w, o, stream)
             : launch_decode_as<1, false>(X, nullptr, nullptr, M, D, F, w, o, stream);
}

}  // namespace bitlinear
