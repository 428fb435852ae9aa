// Layer norm's backward pass (include/bitlinear_block.h).  With
// xhat = (x - mean) rstd and g = dy w:
//   dx = rstd (g - sum_k g / K - xhat sum_k (g xhat) / K)
//   dw = sum_m dy xhat,  db = sum_m dy
// in float32, from x as it was or from its 8-bit copy.  Bound by the bytes of
// x, dy and dx: ln_backward_kernel reads each row once and keeps it in
// registers between the row's sums and its dx, with the columns' dw and db in
// registers across all of a workgroup's rows.  Rows over kLnBwdMaxChunks chunks
// take ln_backward_long_kernel, which keeps dw in LDS; where it does not apply
// the first kernel gives dx alone, and a column kernel reads x and dy again for
// dw and db; over kLnLongMaxChunks, and for rows of fewer than 8 values, dx
// comes from a kernel that reads each row twice.
#include "block_device.hpp"

namespace bitlinear {

namespace {

// dx, dw and db in one pass.  A team of W waves holds a row, NC chunks of 8
// columns to a lane; a workgroup is T = blockDim.x / (64 W) teams.  Team t of
// workgroup b takes rows (i G + b) T + t, i = 0, 1, ...  (G workgroups).  A row
// is converted to xhat and g in registers, and the next one's loads are issued
// before the sums are formed, so that they are in flight through the reduction,
// its barrier and the stores.  A team past the last row works on zeros.  At the
// end the teams' dw and db are added through LDS and the workgroup writes one
// partial row of each (the gradients themselves where it is the only one), so
// no sum depends on the order in which anything runs.
//
// dx is two FMAs,  dx = rstd g - rstd c1 - xhat (rstd c2),  c1, c2 the sums over
// K, and a value is converted once: 125 (float32) to 150 (8-bit x) vector
// instructions for a wave's 512 columns.  1024 SIMDs at 2.4 GHz and 4 clocks an
// instruction issue 600 G of them a second, two to three times what the rates
// here need.  8192x8192, dy float32, dx bfloat16: from the 8-bit copy 92 us (5.15
// TB/s); all float32 147 us (5.5 TB/s).  Smaller arrays pay 4 to 6.5 us for the
// teams' sums, the partial rows and their kernel: 2048x2048 from 8 bits 12.3
// us, dx alone 7.3; 2048x4096 16.6 and 11.0.
//
// PARAMS false: dx alone, for rows whose dw and db do not fit beside them.
// WHOLE: K is a multiple of 8.
template <int XT, int DT, int OT, int W, int NC, int THREADS, bool PARAMS, bool WHOLE>
__global__ __launch_bounds__(THREADS) void ln_backward_kernel(
    const char* __restrict__ dY, const char* __restrict__ X, const float* __restrict__ x_scales,
    const float* __restrict__ mean_in, const float* __restrict__ rstd_in, int64_t M, int K, int cpr,
    const float* __restrict__ weight, char* __restrict__ dX, float* __restrict__ dw_out, float* __restrict__ db_out,
    int64_t out_stride) {
  constexpr bool kWeightInLds = NC > 1;  // else in registers
  constexpr int kMaxT = THREADS / (64 * W);
  constexpr int kTeamFloats = 64 * W * NC * 8;                     // one row
  constexpr int kLds = kTeamFloats * (kMaxT > 2 ? kMaxT / 2 : 1);  // the weight; later half the teams' sums
  __shared__ float slots[2][kMaxT * W * 2];
  __shared__ __align__(16) float lds[kLds];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  const int team = wave / W, wt = wave % W, T = blockDim.x / (64 * W);
  const int64_t G = cpr >> 3, Kp = int64_t(cpr) * 8;
  const float inv_k = 1.0f / static_cast<float>(K);
  // lane's place in a team's area, chunk j: 8 floats in two halves, so that a
  // wave's 16-byte accesses are consecutive
  auto place = [&](int t, int j, int half) { return t * kTeamFloats + ((j * 2 + half) * 64 * W + wt * 64 + lane) * 4; };
  int c[NC], n[NC];
  float dw[PARAMS ? NC : 1][8], db[PARAMS ? NC : 1][8], held_w[8];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    c[j] = wt * 64 + lane + j * 64 * W;
    n[j] = c[j] < cpr ? chunk_values(K, c[j]) : 0;
    float w[8];
    if (weight) {
      Raw<kF32> rw = fetch_chunk<kF32, WHOLE>(reinterpret_cast<const char*>(weight), nullptr, K, cpr, c[j]);
      if constexpr (!WHOLE) settle_chunk<kF32>(rw, n[j]);
      chunk_f32<kF32>(rw, w);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = 1.0f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (PARAMS) dw[j][e] = db[j][e] = 0.0f;
      if constexpr (kWeightInLds) lds[place(0, j, e >> 2) + (e & 3)] = w[e];
      else held_w[e] = w[e];
    }
  }
  auto weight_of = [&](int j, int e) {
    if constexpr (kWeightInLds) return lds[place(0, j, e >> 2) + (e & 3)];
    else return held_w[e];
  };
  Raw<XT> rx[NC];
  Raw<DT> rd[NC];
  float next_mean, next_rstd;
  auto load_row = [&](int64_t m) {
    // behind the last row: any row, whose loads (WHOLE) or values are zeros
    const int behind = m < M ? 0 : cpr;
    m = m < M ? m : 0;
    next_mean = mean_in[m];
    next_rstd = rstd_in[m];
    const char* row = X + (XT == kSaved8 ? m * Kp : m * K * kBytes<XT>);
    const char* drow = dY + m * K * kBytes<DT>;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      rx[j] = fetch_chunk<XT, WHOLE>(row, x_scales + m * G, K, cpr, c[j] + behind);
      rd[j] = fetch_chunk<DT, WHOLE>(drow, nullptr, K, cpr, c[j] + behind);
    }
  };
  const int64_t stride = static_cast<int64_t>(gridDim.x) * T;
  // workgroups are dealt round-robin to the 8 XCDs: consecutive rows to an XCD
  // (2% to 4% at 2048x11008 and 8192x8192)
  const uint32_t b = gridDim.x % 8 == 0 ? (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3) : blockIdx.x;
  int64_t m = static_cast<int64_t>(b) * T + team;
  const int64_t iters = (M + stride - 1) / stride;
  load_row(m);
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    arrive(rx[j]);
    arrive(rd[j]);
  }
  for (int64_t it = 0; it < iters; ++it, m += stride) {
    const bool ok = m < M;
    // a team past the last row has x = dy = 0; with xhat 0 too, whatever the
    // first row's statistics are
    const float mu = ok ? next_mean : 0.0f, rs = ok ? next_rstd : 0.0f;
    float xh[NC][8], g[NC][8], s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      if constexpr (!WHOLE) {
        const int nj = ok ? n[j] : 0;
        settle_chunk<XT>(rx[j], nj);
        settle_chunk<DT>(rd[j], nj);
      }
      chunk_f32<XT>(rx[j], xh[j]);
      chunk_f32<DT>(rd[j], g[j]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // behind the row x is 0, and mean rstd may be infinite and meet dy = 0
        const float mean = (WHOLE ? n[j] > 0 : e < n[j]) ? mu : 0.0f;
        xh[j][e] = (xh[j][e] - mean) * rs;
      }
    }
    load_row(m + stride);
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (PARAMS) {
          db[j][e] += g[j][e];
          dw[j][e] = __fmaf_rn(g[j][e], xh[j][e], dw[j][e]);
        }
        g[j][e] *= weight_of(j, e);
        s[0] += g[j][e];
        s[1] = __fmaf_rn(g[j][e], xh[j][e], s[1]);
      }
    team_sum<W>(s, slots[it & 1] + team * W * 2, wt, lane);
    const __amdgpu_buffer_rsrc_t to = row_resource(dX + (ok ? m * K * kBytes<OT> : 0), dX && ok ? K * kBytes<OT> : 0);
    const float k1 = rs * (s[0] * inv_k), k2 = rs * (s[1] * inv_k);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
#pragma unroll
      for (int e = 0; e < 8; ++e) g[j][e] = __fmaf_rn(-k2, xh[j][e], __fmaf_rn(rs, g[j][e], -k1));
      put_chunk<OT, WHOLE>(to, c[j], n[j], g[j]);
    }
  }
  if (!PARAMS || (!dw_out && !db_out)) return;
  // add the upper half of the teams to the lower half until one is left
  auto combine = [&](auto& v) {
    for (int left = T; left > 1;) {
      const int half = (left + 1) / 2;
      __syncthreads();
      if (team >= half && team < left) {
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) lds[place(team - half, j, e >> 2) + (e & 3)] = v[j][e];
      }
      __syncthreads();
      if (team < left - half) {
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[j][e] += lds[place(team, j, e >> 2) + (e & 3)];
      }
      left = half;
    }
  };
  auto finish = [&](auto& v, float* out) {
    if (!out) return;
    combine(v);
    if (team == 0) {
#pragma unroll
      for (int j = 0; j < NC; ++j)
        store_chunk<kF32>(reinterpret_cast<char*>(out + blockIdx.x * out_stride), c[j], n[j], v[j]);
    }
  };
  if constexpr (PARAMS) {
    finish(dw, dw_out);
    finish(db, db_out);
  }
}

// Long rows of a multiple of 8 values, all three gradients from one pass over x
// and dy: 8 waves, 7 chunks to a lane, a workgroup to each CU.  What does not
// fit into registers beside dy and x: dw and two of a lane's 7 chunks of db lie
// in LDS (144 KB; a lane adds to its own columns alone, 16 bytes at a time), the
// weight is read again from the cache, a chunk ahead, and x stays as it is in
// memory until its xhat is needed, twice.  The next row's chunk is loaded where
// this row's has been stored.  2048x28672: float32 163 us, 8-bit x (dy float32,
// dx bfloat16) 108; with all of db in registers, which spill, 193 and 120; the
// two passes that it replaces 228 and 147.  8192x28672 from 8 bits 337 us, 4.9
// TB/s.
// The same kernel for rows of up to 16384 is 5% to 30% slower than the one above.
template <int XT, int DT, int OT>
__global__ __launch_bounds__(512) void ln_backward_long_kernel(
    const char* __restrict__ dY, const char* __restrict__ X, const float* __restrict__ x_scales,
    const float* __restrict__ mean_in, const float* __restrict__ rstd_in, int64_t M, int K, int cpr,
    const float* __restrict__ weight, char* __restrict__ dX, float* __restrict__ dw_out, float* __restrict__ db_out,
    int64_t out_stride) {
  constexpr int NC = kLnLongChunks, kStep = 512, kInLds = 2;
  __shared__ float slots[2][16];
  __shared__ __align__(16) float sums_lds[(NC + kInLds) * kStep * 8];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  const int64_t G = cpr >> 3, Kp = int64_t(cpr) * 8;
  const float inv_k = 1.0f / static_cast<float>(K);
  auto place = [&](int j, int half) { return ((j * 2 + half) * kStep + tid) * 4; };
  float held_db[NC - kInLds][8];
  auto dw = [&](int j, int e) -> float& { return sums_lds[place(j, e >> 2) + (e & 3)]; };
  auto db = [&](int j, int e) -> float& {
    return j < kInLds ? dw(NC + j, e) : held_db[j < kInLds ? 0 : j - kInLds][e];
  };
#pragma unroll
  for (int j = 0; j < NC; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) db(j, e) = dw(j, e) = 0.0f;
  Raw<XT> rx[NC];
  Raw<DT> rd[NC];
  auto load = [&](int64_t m, int j) {
    // behind the last row: a row without values
    const int k = m < M ? K : 0, cp = m < M ? cpr : 0;
    m = m < M ? m : 0;
    rd[j] = fetch_whole<DT>(dY + m * K * kBytes<DT>, nullptr, k, cp, j * kStep, tid);
    rx[j] = fetch_whole<XT>(X + (XT == kSaved8 ? m * Kp : m * K * kBytes<XT>), x_scales + m * G, k, cp, j * kStep,
                            tid);
  };
  auto weight_chunk = [&](int j, float (&w)[8]) {
    if (weight) {
      chunk_f32<kF32>(fetch_whole<kF32>(reinterpret_cast<const char*>(weight), nullptr, K, cpr, j * kStep, tid), w);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = 1.0f;
    }
  };
  const int64_t stride = gridDim.x;
  // consecutive rows to an XCD, as above
  const uint32_t b = gridDim.x % 8 == 0 ? (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3) : blockIdx.x;
  int64_t m = b;
#pragma unroll
  for (int j = 0; j < NC; ++j) load(m, j);
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    arrive(rd[j]);
    arrive(rx[j]);
  }
  for (int turn = 0; m < M; m += stride, turn ^= 1) {
    const float mu = mean_in[m], rs = rstd_in[m];
    float g[NC][8], s[2] = {0.0f, 0.0f}, w[2][8];
    weight_chunk(0, w[0]);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      if (j + 1 < NC) weight_chunk(j + 1, w[(j + 1) & 1]);
      float xh[8];
      chunk_f32<DT>(rd[j], g[j]);
      chunk_f32<XT>(rx[j], xh);
      const float mean = j * kStep + tid < K >> 3 ? mu : 0.0f;  // behind the row x is 0
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xh[e] = (xh[e] - mean) * rs;
        db(j, e) += g[j][e];
        dw(j, e) = __fmaf_rn(g[j][e], xh[e], dw(j, e));
        g[j][e] *= w[j & 1][e];
        s[0] += g[j][e];
        s[1] = __fmaf_rn(g[j][e], xh[e], s[1]);
      }
    }
    team_sum<8>(s, slots[turn], wave, lane);
    const float k1 = rs * (s[0] * inv_k), k2 = rs * (s[1] * inv_k);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      float xh[8];
      chunk_f32<XT>(rx[j], xh);
      const float mean = j * kStep + tid < K >> 3 ? mu : 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        g[j][e] = __fmaf_rn(-k2, (xh[e] - mean) * rs, __fmaf_rn(rs, g[j][e], -k1));
      const int at = j * kStep * 8 * kBytes<OT>, bytes = dX ? max(K * kBytes<OT> - at, 0) : 0;
      put_chunk<OT, true>(row_resource(dX + (bytes ? m * K * kBytes<OT> + at : 0), bytes), tid, 8, g[j]);
      load(m + stride, j);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    float v[8], u[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = dw(j, e), u[e] = db(j, e);
    const int c = j * kStep + tid, n = c < K >> 3 ? 8 : 0;
    if (dw_out) store_chunk<kF32>(reinterpret_cast<char*>(dw_out + blockIdx.x * out_stride), c, n, v);
    if (db_out) store_chunk<kF32>(reinterpret_cast<char*>(db_out + blockIdx.x * out_stride), c, n, u);
  }
}

// dx of long rows, and of rows of fewer than 8 values (SHORT): one workgroup per
// row, rows gridDim.x apart; the row is read for the two sums and again for the
// output.  2048x32768 from 8 bits 159 us (2048x28672 in the kernels above 84),
// 2048x53248 273, 2.8 TB/s of x, dy and dx once.
template <int XT, int DT, int OT, bool SHORT>
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
      chunk_f32<XT>(load_chunk<XT, SHORT>(row, x_scales + m * G, K, c, n), xh);
      chunk_f32<DT>(load_chunk<DT, SHORT>(drow, nullptr, K, c, n), g);
      if (weight) {
        float w[8];
        chunk_f32<kF32>(load_chunk<kF32, SHORT>(reinterpret_cast<const char*>(weight), nullptr, K, c, n), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] *= w[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) xh[e] = e < n ? (xh[e] - mean) * rstd : 0.0f;
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
template <int XT, int DT, bool SHORT>
__global__ __launch_bounds__(256) void ln_param_cols_kernel(
    const char* __restrict__ dY, const char* __restrict__ X, const float* __restrict__ x_scales,
    const float* __restrict__ mean_in, const float* __restrict__ rstd_in, int64_t M, int K, int cpr,
    float* __restrict__ dw_out, float* __restrict__ db_out, int64_t out_stride) {
  __shared__ float sums[8][32 * 8];
  const int tid = threadIdx.x, cl = tid & 31, r = tid >> 5;
  const int c = blockIdx.x * 32 + cl;
  const int64_t G = cpr >> 3, Kp = int64_t(cpr) * 8;
  const int n = c < cpr ? chunk_values(K, c) : 0;
  float dw[8] = {}, db[8] = {};
  for (int64_t m = blockIdx.y * 8 + r; m < M; m += int64_t(gridDim.y) * 8) {
    float xh[8], d[8];
    const char* row = X + (XT == kSaved8 ? m * Kp : m * K * kBytes<XT>);
    chunk_f32<XT>(load_chunk<XT, SHORT>(row, x_scales + m * G, K, c, n), xh);
    chunk_f32<DT>(load_chunk<DT, SHORT>(dY + m * K * kBytes<DT>, nullptr, K, c, n), d);
    const float mean = mean_in[m], rstd = rstd_in[m];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      db[e] += d[e];
      dw[e] = __fmaf_rn(d[e], (xh[e] - mean) * rstd, dw[e]);
    }
  }
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    float* out = a ? db_out : dw_out;
    if (!out) continue;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[r][cl * 8 + e] = a ? db[e] : dw[e];
    __syncthreads();
    const int k = blockIdx.x * 256 + tid;
    if (k < K) {
      float t = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) t += sums[i][tid];
      out[blockIdx.y * out_stride + k] = t;
    }
  }
}

// dw[k] = sum over the partial rows of partial[row][0][k], db likewise from
// [1]: 64 columns to a workgroup, a wave to every 16th row (at most 256 rows, so
// 16 loads, all in flight), then the 16 waves' sums in order.
__global__ __launch_bounds__(1024) void ln_param_sum_kernel(const float* __restrict__ partial, int rows, int K,
                                                            float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float sums[16][64];
  float* out = blockIdx.y ? db : dw;
  if (!out) return;
  const int kl = threadIdx.x & 63, r = threadIdx.x >> 6;
  const int k = blockIdx.x * 64 + kl;
  const float* p = partial + static_cast<int64_t>(blockIdx.y) * K + min(k, K - 1);
  float t = 0.0f;
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = r + 16 * i < rows ? p[static_cast<int64_t>(r + 16 * i) * 2 * K] : 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) t += v[i];
  sums[r][kl] = t;
  __syncthreads();
  if (r == 0 && k < K) {
    t = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += sums[i][kl];
    out[k] = t;
  }
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

// Where a kernel's sums go: the partial rows, or the gradients themselves.
float* dweight_to(const Args& a, const LnBwdPlan& p) {
  return !a.dweight ? nullptr : ln_bwd_alone(p, a.K) ? a.dweight : a.partial;
}
float* dbias_to(const Args& a, const LnBwdPlan& p) {
  return !a.dbias ? nullptr : ln_bwd_alone(p, a.K) ? a.dbias : a.partial + a.K;
}

template <int XT, int DT, int OT, int W, int NC, int THREADS = 1024, bool PARAMS = true>
void launch_one(const Args& a, const LnBwdPlan& p, hipStream_t stream) {
  const int64_t K = a.K;
  auto kernel = K % 8 == 0 ? ln_backward_kernel<XT, DT, OT, W, NC, THREADS, PARAMS, true>
                           : ln_backward_kernel<XT, DT, OT, W, NC, THREADS, PARAMS, false>;
  kernel<<<p.groups, 64 * W * p.teams, 0, stream>>>(
      static_cast<const char*>(a.dY), static_cast<const char*>(a.X.p), a.X.scales, a.mean, a.rstd, a.M,
      static_cast<int>(K), static_cast<int>(padded_k(K) / 8), a.weight, static_cast<char*>(a.dX),
      dweight_to(a, p), dbias_to(a, p), 2 * K);
}

template <int XT, int DT, int OT>
hipError_t launch(const Args& a, hipStream_t stream) {
  const int cpr = static_cast<int>(padded_k(a.K) / 8), K = static_cast<int>(a.K);
  const LnBwdPlan p = ln_bwd_plan(a.M, a.K, a.dweight || a.dbias);
  const char* dY = static_cast<const char*>(a.dY);
  const char* X = static_cast<const char*>(a.X.p);
  if (p.chunks == kLnLongChunks) {
    ln_backward_long_kernel<XT, DT, OT><<<p.groups, 512, 0, stream>>>(
        dY, X, a.X.scales, a.mean, a.rstd, a.M, K, cpr, a.weight, static_cast<char*>(a.dX), dweight_to(a, p),
        dbias_to(a, p), 2 * a.K);
  } else if (p.waves == 0) {
    if (a.dX && K >= 8 && cpr <= kLnLongMaxChunks) {
      const LnBwdPlan dx = {8, kLnLongChunks, 1, static_cast<int>(a.M < 256 ? a.M : 256)};
      launch_one<XT, DT, OT, 8, kLnLongChunks, 512, false>(a, dx, stream);
    } else if (a.dX) {
      const unsigned blocks = static_cast<unsigned>(a.M < (1 << 20) ? a.M : (1 << 20));
      auto kernel = K < 8 ? ln_dx_rows_kernel<XT, DT, OT, true> : ln_dx_rows_kernel<XT, DT, OT, false>;
      kernel<<<blocks, 256, 0, stream>>>(dY, X, a.X.scales, a.mean, a.rstd, a.M, K, cpr, a.weight,
                                         static_cast<char*>(a.dX));
    }
    if (a.dweight || a.dbias) {
      auto kernel = K < 8 ? ln_param_cols_kernel<XT, DT, true> : ln_param_cols_kernel<XT, DT, false>;
      kernel<<<dim3((cpr + 31) / 32, p.groups), 256, 0, stream>>>(dY, X, a.X.scales, a.mean, a.rstd, a.M, K, cpr,
                                                                  dweight_to(a, p), dbias_to(a, p), 2 * a.K);
    }
  } else if (p.chunks == 1) {
    if (p.waves == 1) launch_one<XT, DT, OT, 1, 1>(a, p, stream);
    else if (p.waves == 2) launch_one<XT, DT, OT, 2, 1>(a, p, stream);
    else if (p.waves == 4) launch_one<XT, DT, OT, 4, 1>(a, p, stream);
    else if (p.waves == 8) launch_one<XT, DT, OT, 8, 1>(a, p, stream);
    else launch_one<XT, DT, OT, 16, 1>(a, p, stream);
  } else {
    if (p.chunks == 3) launch_one<XT, DT, OT, 8, 3, 512>(a, p, stream);
    else launch_one<XT, DT, OT, 8, 4, 512>(a, p, stream);
  }
  if ((a.dweight || a.dbias) && !ln_bwd_alone(p, a.K))
    ln_param_sum_kernel<<<dim3((K + 63) / 64, 2), 1024, 0, stream>>>(a.partial, p.groups, K, a.dweight, a.dbias);
  return hipGetLastError();
}

template <int DT, int OT>
hipError_t launch_from(const Args& a, hipStream_t s) {
  if (a.X.dtype == kF32) return launch<kF32, DT, OT>(a, s);
  if (a.X.dtype == kBf16) return launch<kBf16, DT, OT>(a, s);
  return launch<kSaved8, DT, OT>(a, s);
}

}  // namespace

hipError_t launch_layer_norm_backward(const void* dY, int dy_dtype, BlockIn X, const float* mean, const float* rstd,
                                      int64_t M, int64_t K, const float* weight, void* dX, int dx_dtype,
                                      float* dweight, float* dbias, void* workspace, hipStream_t stream) {
  const Args a = {dY, X, mean, rstd, M, K, weight, dX, dweight, dbias, static_cast<float*>(workspace)};
  if (!dX) dx_dtype = kF32;  // not written
  if (dy_dtype == kF32)
    return dx_dtype == kF32 ? launch_from<kF32, kF32>(a, stream) : launch_from<kF32, kBf16>(a, stream);
  return dx_dtype == kF32 ? launch_from<kBf16, kF32>(a, stream) : launch_from<kBf16, kBf16>(a, stream);
}

}  // namespace bitlinear
