// A decode batch through a projection and its adapters (include/bitlinear_adapters.h)
// in two launches.  What a small call costs is launches (about 4 us each on the
// host) and kernels that wait for one memory access after another, so:
//   1. what reads X alone: the adapters' first product, and the tokens' codes;
//   2. the decode forward's split form (decode_kernel.hpp) on those codes, one
//      block of 16 weight rows to a workgroup, which also forms the adapters'
//      second product for its 16 columns while its first weights are on their way.
// Tokens whose codes do not fit one workgroup's LDS go in up to four pieces, each
// through all weight rows.  On the GPU 1x2048x2048 takes 4.8 and 7.3 us, 16x4096x4096
// with an adapter of 16 ranks for every token 5.8 and 11.4.
#include "adapter_ops.hpp"
#include "block_device.hpp"
#include "decode_kernel.hpp"

namespace bitlinear {

namespace {

struct PartOfGrid {
  uint32_t index, count;
  __device__ uint32_t block() const { return index; }
  __device__ uint32_t blocks() const { return count; }
};

// The second product for 16 columns and up to 16 tokens: a thread to an output.
// LDS: T of the tokens, scaled ([16][R] float32), then the 16 x 16 results.
template <int WT>
struct AddAdapters {
  static constexpr bool kOn = true;
  Adapters ad;
  const char* up;
  const float* parts;  // from the piece's first token
  int nparts, stride;  // floats from part to part
  float* T;            // NULL, or the piece's rows of T (written by the first block)
  int m0, block;

  __device__ __forceinline__ int adapter(int i) const {
    const int id = ad.rows[m0 + i];
    return id >= 0 && id < ad.A ? id : -1;
  }
  __device__ __forceinline__ float weight(int a, int r, uint32_t n, uint32_t N) const {
    const int64_t at = (static_cast<int64_t>(a) * ad.R + r) * N + n;
    if constexpr (WT == kF32) return reinterpret_cast<const float*>(up)[at];
    else return bf16_to_f32(reinterpret_cast<const uint16_t*>(up)[at]);
  }
  __device__ __forceinline__ void prepare(int M, uint32_t n0, uint32_t N, int8_t* lds) const {
    float* t = reinterpret_cast<float*>(lds);
    float* d = t + 16 * ad.R;
    const int Rp = (ad.R + 15) & ~15;
    const int i = threadIdx.x >> 4;
    const uint32_t n = n0 + (threadIdx.x & 15u);
    const int a = i < M && n < N ? adapter(i) : -1;
    // the first 16 ranks' weights are asked for before T's parts are added
    float w[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) w[r] = a >= 0 && r < ad.R ? weight(a, r, n, N) : 0.0f;
    for (int x = threadIdx.x; x < M * ad.R; x += kDecodeThreads) {
      const int token = x / ad.R, r = x - token * ad.R, id = adapter(token);
      float v = 0.0f;
      if (id >= 0) {
        const float* from = parts + token * Rp + r;
        v = from[0];
#pragma unroll 4
        for (int s = 1; s < nparts; ++s) v += from[s * stride];
      }
      if (T != nullptr && block == 0) T[x] = v;
      t[x] = id >= 0 ? __fmul_rn(v, ad.scales[id]) : 0.0f;
    }
    __syncthreads();
    float sum = -0.0f;  // without an adapter: leaves every output as it is, its sign of zero too
    if (a >= 0) {
      const float* mine = t + i * ad.R;
      sum = __fmul_rn(mine[0], w[0]);
#pragma unroll
      for (int r = 1; r < 16; ++r)
        if (r < ad.R) sum = __fmaf_rn(mine[r], w[r], sum);
#pragma unroll 8
      for (int r = 16; r < ad.R; ++r) sum = __fmaf_rn(mine[r], weight(a, r, n, N), sum);
    }
    d[threadIdx.x] = sum;
  }
  // token i (0 to 15), row j of the block
  __device__ __forceinline__ float add(int i, int j, float y, const int8_t* lds) const {
    return __fadd_rn(y, reinterpret_cast<const float*>(lds)[16 * ad.R + 16 * i + j]);
  }
};

template <int SPLIT, int WT>
__global__ __launch_bounds__(kDecodeThreads) void adapted_decode_kernel(const int8_t* Xq, const float* ga,
                                                                        const int32_t* rs, int M, int64_t K, int64_t Kp,
                                                                        const uint32_t* packed, int64_t N,
                                                                        const float* gamma, float* Y, int piece,
                                                                        int row_blocks, Adapters ad, const char* up,
                                                                        const float* parts, int nparts, float* T) {
  const uint32_t which = blockIdx.x / static_cast<uint32_t>(row_blocks), b = blockIdx.x - which * row_blocks;
  const int m0 = static_cast<int>(which) * piece, m = min(piece, M - m0), Rp = (ad.R + 15) & ~15;
  const AddAdapters<WT> extra = {ad, up, parts + m0 * Rp, nparts, M * Rp, T ? T + m0 * ad.R : nullptr,
                                 m0, static_cast<int>(b)};
  decode_body<2, 2, true, kEpiY, SPLIT>(Xq + m0 * Kp, m, K, Kp, Kp / 64, packed, N, gamma, Y + m0 * N, nullptr,
                                        row_blocks, 1, 0, ga + m0, rs + m0,
                                        PartOfGrid{b, static_cast<uint32_t>(row_blocks)}, extra);
}

template <int WT>
hipError_t launch_second(int64_t M, int64_t K, const uint32_t* packed, int64_t N, const float* gamma, float* Y,
                         const Adapters& ad, const void* up, const float* parts, int nparts, float* T, int64_t piece,
                         const int8_t* Xq, const float* ga, const int32_t* rs, hipStream_t stream) {
  const int64_t Kp = padded_k(K), row_blocks = (N + 15) / 16, pieces = (M + piece - 1) / piece;
  // loads a batch as in the decode forward
  auto kernel = ((Kp / 64 + 3) / 4 + 3) / 4 <= 8 ? adapted_decode_kernel<2, WT> : adapted_decode_kernel<4, WT>;
  const size_t lds = static_cast<size_t>(piece * (Kp + 16)) + kDecodeThreads * sizeof(v4i) +
                     static_cast<size_t>(16 * ad.R + 256) * 4;
  kernel<<<static_cast<unsigned>(pieces * row_blocks), kDecodeThreads, lds, stream>>>(
      Xq, ga, rs, static_cast<int>(M), K, Kp, packed, N, gamma, Y, static_cast<int>(piece),
      static_cast<int>(row_blocks), ad, static_cast<const char*>(up), parts, nparts, T);
  return hipGetLastError();
}

}  // namespace

int64_t adapted_decode_piece(int64_t M, int64_t K, int64_t N) {
  const int64_t blocks16 = (N + 15) / 16, rows = int64_t(kWaves) * kRowsPerWave * pick_groups(1, N);
  const int64_t blocks = (N + rows - 1) / rows;
  // the split form's own condition, and what its launches need
  if (M > kDecodeMaxM || K < 8 || blocks >= kSplitBelow || blocks16 <= blocks || M * N >= (int64_t(1) << 29)) return 0;
  for (int64_t pieces = 1; pieces <= 4; ++pieces) {
    const int64_t piece = (M + pieces - 1) / pieces;
    if (piece * (padded_k(K) + 16) <= kDecodeMaxCodes) return piece;
  }
  return 0;
}

hipError_t launch_adapted_decode(const void* X, int x_dtype, int64_t M, int64_t K, const uint32_t* packed, int64_t N,
                                 const float* gamma, float* Y, const Adapters& ad, const void* down, const void* up,
                                 float* parts, float* T, int64_t piece, int8_t* Xq, float* ga, int32_t* rs,
                                 hipStream_t stream) {
  const ShrinkPlan p = shrink_plan(M, K);
  const hipError_t e = launch_adapted_first(X, x_dtype, M, K, ad, down, parts, Xq, ga, rs, stream);
  if (e != hipSuccess) return e;
  return ad.w_dtype == kF32
             ? launch_second<kF32>(M, K, packed, N, gamma, Y, ad, up, parts, p.parts, T, piece, Xq, ga, rs, stream)
             : launch_second<kBf16>(M, K, packed, N, gamma, Y, ad, up, parts, p.parts, T, piece, Xq, ga, rs, stream);
}

}  // namespace bitlinear
