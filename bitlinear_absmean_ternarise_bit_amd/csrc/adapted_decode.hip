// A decode batch through a projection and its adapters (include/bitlinear_adapters.h):
// the ternary product and the adapters' first product, which both read X alone,
// in one launch.  What a small call costs is launches (about 4 us each on the
// host, where the two kernels run 3 to 4 us), so this saves one of three.
//
// The first workgroups take the first product, the others the decode forward's
// split form (one block of 16 weight rows each, decode_kernel.hpp).  Tokens whose
// codes do not fit one workgroup's LDS go in up to four pieces, each through all
// weight rows (16 x 4096 x 4096: 5.9 us instead of 23.6 for the quantiser and the
// GEMM, which reads the weights once but has 32 workgroups).
#include "adapter_device.hpp"
#include "decode_kernel.hpp"

namespace bitlinear {

namespace {

struct PartOfGrid {
  uint32_t index, count;
  __device__ uint32_t block() const { return index; }
  __device__ uint32_t blocks() const { return count; }
};

struct ShrinkArgs {
  const char* W;
  float* parts;
  int nparts, spread;
};

// piece: tokens of a piece; row_blocks: blocks of 16 weight rows
template <int DT, bool VEC, int SPLIT, int WT>
__global__ __launch_bounds__(kDecodeThreads) void adapted_decode_kernel(const char* X, int M, int64_t K, int64_t Kp,
                                                                        int64_t units, const uint32_t* packed, int64_t N,
                                                                        const float* gamma, float* Y, int piece,
                                                                        int row_blocks, Adapters ad, ShrinkArgs sh) {
  static_assert(kDecodeThreads == kAdapterThreads, "one launch for both");
  const int first = sh.nparts * sh.spread;
  if (static_cast<int>(blockIdx.x) < first) {
    const int b = static_cast<int>(blockIdx.x);
    shrink_body<DT, WT, 1, 1>(X, M, K, ad, sh.W, sh.parts, 1, 0, 1, b % sh.nparts, sh.nparts, b / sh.nparts, sh.spread);
    return;
  }
  const uint32_t b = blockIdx.x - static_cast<uint32_t>(first), which = b / static_cast<uint32_t>(row_blocks);
  const int m0 = static_cast<int>(which) * piece;
  decode_body<2, DT, VEC, kEpiY, SPLIT>(X + m0 * K * kBytes<DT>, min(piece, M - m0), K, Kp, units, packed, N, gamma,
                                        Y + m0 * N, nullptr, row_blocks, 1, 0, nullptr, nullptr,
                                        PartOfGrid{b - which * static_cast<uint32_t>(row_blocks), static_cast<uint32_t>(row_blocks)});
}

template <int DT, int WT>
hipError_t launch_as(const void* X, int64_t M, int64_t K, const uint32_t* packed, int64_t N, const float* gamma,
                     float* Y, const Adapters& ad, const ShrinkArgs& sh, int64_t piece, hipStream_t stream) {
  const int64_t Kp = padded_k(K), units = Kp / 64, row_blocks = (N + 15) / 16, pieces = (M + piece - 1) / piece;
  const bool vec = reinterpret_cast<uintptr_t>(X) % 16 == 0 && (K * kBytes<DT>) % 16 == 0;
  const bool two = ((units + 3) / 4 + 3) / 4 <= 8;  // loads a batch, as in the decode forward
  auto kernel = vec ? (two ? adapted_decode_kernel<DT, true, 2, WT> : adapted_decode_kernel<DT, true, 4, WT>)
                    : (two ? adapted_decode_kernel<DT, false, 2, WT> : adapted_decode_kernel<DT, false, 4, WT>);
  const size_t lds = static_cast<size_t>(piece * (Kp + 16)) + kDecodeThreads * sizeof(v4i);
  kernel<<<static_cast<unsigned>(sh.nparts * sh.spread + pieces * row_blocks), kDecodeThreads, lds, stream>>>(
      static_cast<const char*>(X), static_cast<int>(M), K, Kp, units, packed, N, gamma, Y, static_cast<int>(piece),
      static_cast<int>(row_blocks), ad, sh);
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
                                 const float* gamma, float* Y, const Adapters& ad, const void* down, float* parts,
                                 int64_t piece, hipStream_t stream) {
  const ShrinkPlan p = shrink_plan(M, K);
  const ShrinkArgs sh = {static_cast<const char*>(down), parts, p.parts, p.spread};
  if (x_dtype == kF32)
    return ad.w_dtype == kF32 ? launch_as<kF32, kF32>(X, M, K, packed, N, gamma, Y, ad, sh, piece, stream)
                              : launch_as<kF32, kBf16>(X, M, K, packed, N, gamma, Y, ad, sh, piece, stream);
  return ad.w_dtype == kF32 ? launch_as<kBf16, kF32>(X, M, K, packed, N, gamma, Y, ad, sh, piece, stream)
                            : launch_as<kBf16, kBf16>(X, M, K, packed, N, gamma, Y, ad, sh, piece, stream);
}

}  // namespace bitlinear
