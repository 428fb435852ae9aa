// C ABI of the operators around BitLinear (include/bitlinear_block.h):
// argument checks on the host, then the launches.
#include <math.h>
#include <stdint.h>

#include "../../include/bitlinear_block.h"
#include "block_ops.hpp"

using namespace bitlinear;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_mk(int64_t M, int64_t K) {
  if (M < 1 || K < 1 || K > (int64_t(1) << 20) || M > (int64_t(1) << 31)) return BITLINEAR_ERR_SHAPE;
  return static_cast<uint64_t>(M) * static_cast<uint64_t>(K) >= (uint64_t(1) << 40) ? BITLINEAR_ERR_SHAPE
                                                                                    : BITLINEAR_OK;
}

bool plain_dtype(int dt) { return dt == BITLINEAR_F32 || dt == BITLINEAR_BF16; }

// A memory range of an argument; NULL ranges overlap nothing.
struct Range {
  const void* p;
  uint64_t bytes;
};

bool overlap(const Range& a, const Range& b) {
  if (!a.p || !b.p) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y ? y - x < a.bytes : x - y < b.bytes;
}

// Whether an output overlaps an input or another output.
template <int NO, int NI>
bool any_overlap(const Range (&out)[NO], const Range (&in)[NI]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < NI; ++j)
      if (overlap(out[i], in[j])) return true;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return true;
  }
  return false;
}

// Sizes of arrays within the limits of check_mk (no overflow in 64 bits).
Range array(const void* p, int dt, int64_t M, int64_t K) {
  const uint64_t m = static_cast<uint64_t>(M);
  if (dt == BITLINEAR_SAVED8) return {p, m * static_cast<uint64_t>(padded_k(K))};
  return {p, m * static_cast<uint64_t>(K) * (dt == BITLINEAR_F32 ? 4 : 2)};
}
Range floats(const float* p, int64_t n) { return {p, static_cast<uint64_t>(n) * 4}; }
Range scale_range(const float* p, int64_t M, int64_t K) { return floats(p, M * saved_groups(K)); }

bool aligned_to(const void* p, int dt) {
  return aligned(p, dt == BITLINEAR_F32 ? 4 : dt == BITLINEAR_BF16 ? 2 : 16);
}

// An input that may be whole or saved: dtype, scales, alignment.
int check_in(const void* p, const float* scales, int dt) {
  if (!plain_dtype(dt) && dt != BITLINEAR_SAVED8) return BITLINEAR_ERR_DTYPE;
  if (dt == BITLINEAR_SAVED8 && !scales) return BITLINEAR_ERR_NULL;
  if (!aligned_to(p, dt) || (dt == BITLINEAR_SAVED8 && !aligned(scales, 4))) return BITLINEAR_ERR_ALIGN;
  return BITLINEAR_OK;
}

// An optional pair of saved outputs.
int check_saved_out(const int8_t* codes, const float* scales, int in_dtype) {
  if (!codes != !scales) return BITLINEAR_ERR_NULL;
  if (!codes) return BITLINEAR_OK;
  if (in_dtype == BITLINEAR_SAVED8) return BITLINEAR_ERR_ARG;
  return aligned(codes, 16) && aligned(scales, 4) ? BITLINEAR_OK : BITLINEAR_ERR_ALIGN;
}

int hip_status(hipError_t e) { return e == hipSuccess ? BITLINEAR_OK : BITLINEAR_ERR_HIP; }

BlockIn block_in(const void* p, const float* scales, int dt) {
  return {p, dt == BITLINEAR_SAVED8 ? scales : nullptr, dt};
}

}  // namespace

extern "C" {

int64_t bitlinear_saved_groups(int64_t K) { return size_args_ok(K) ? saved_groups(K) : 0; }

int bitlinear_save_activations(const void* X, int x_dtype, int64_t M, int64_t K, int8_t* codes, float* scales,
                               void* stream) {
  if (!X || !codes || !scales) return BITLINEAR_ERR_NULL;
  int st = check_mk(M, K);
  if (st) return st;
  if (!plain_dtype(x_dtype)) return BITLINEAR_ERR_DTYPE;
  if (!aligned_to(X, x_dtype)) return BITLINEAR_ERR_ALIGN;
  st = check_saved_out(codes, scales, x_dtype);
  if (st) return st;
  const Range out[] = {array(codes, BITLINEAR_SAVED8, M, K), scale_range(scales, M, K)};
  const Range in[] = {array(X, x_dtype, M, K)};
  if (any_overlap(out, in)) return BITLINEAR_ERR_ARG;
  return hip_status(launch_save(X, x_dtype, M, K, codes, scales, static_cast<hipStream_t>(stream)));
}

int bitlinear_restore_activations(const int8_t* codes, const float* scales, int64_t M, int64_t K, void* X,
                                  int x_dtype, void* stream) {
  if (!X || !codes || !scales) return BITLINEAR_ERR_NULL;
  int st = check_mk(M, K);
  if (st) return st;
  if (!plain_dtype(x_dtype)) return BITLINEAR_ERR_DTYPE;
  st = check_in(codes, scales, BITLINEAR_SAVED8);
  if (st) return st;
  if (!aligned_to(X, x_dtype)) return BITLINEAR_ERR_ALIGN;
  const Range out[] = {array(X, x_dtype, M, K)};
  const Range in[] = {array(codes, BITLINEAR_SAVED8, M, K), scale_range(scales, M, K)};
  if (any_overlap(out, in)) return BITLINEAR_ERR_ARG;
  return hip_status(launch_restore(block_in(codes, scales, BITLINEAR_SAVED8), M, K, X, x_dtype,
                                   static_cast<hipStream_t>(stream)));
}

int bitlinear_layer_norm(const void* X, const float* x_scales, int x_dtype, int64_t M, int64_t K,
                         const float* weight, const float* bias, float eps, void* Y, int y_dtype, float* mean,
                         float* rstd, int8_t* saved, float* saved_scales, void* stream) {
  if (!X || !Y || !mean != !rstd) return BITLINEAR_ERR_NULL;
  int st = check_mk(M, K);
  if (st) return st;
  st = check_in(X, x_scales, x_dtype);
  if (st) return st;
  if (!plain_dtype(y_dtype)) return BITLINEAR_ERR_DTYPE;
  if (!aligned_to(Y, y_dtype) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(mean, 4) || !aligned(rstd, 4))
    return BITLINEAR_ERR_ALIGN;
  st = check_saved_out(saved, saved_scales, x_dtype);
  if (st) return st;
  if (!(eps >= 0.0f) || isinf(eps)) return BITLINEAR_ERR_ARG;
  const BlockIn x = block_in(X, x_scales, x_dtype);
  const Range out[] = {array(Y, y_dtype, M, K), floats(mean, M), floats(rstd, M),
                       array(saved, BITLINEAR_SAVED8, M, K), scale_range(saved_scales, M, K)};
  const Range in[] = {array(X, x_dtype, M, K), scale_range(x.scales, M, K), floats(weight, K), floats(bias, K)};
  if (any_overlap(out, in)) return BITLINEAR_ERR_ARG;
  return hip_status(launch_layer_norm(x, M, K, weight, bias, eps, Y, y_dtype, mean, rstd, saved, saved_scales,
                                      static_cast<hipStream_t>(stream)));
}

size_t bitlinear_layer_norm_backward_workspace_bytes(int64_t M, int64_t K) { return ln_bwd_workspace_bytes(M, K); }

int bitlinear_layer_norm_backward(const void* dY, int dy_dtype, const void* X, const float* x_scales, int x_dtype,
                                  const float* mean, const float* rstd, int64_t M, int64_t K, const float* weight,
                                  void* dX, int dx_dtype, float* dweight, float* dbias, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  if (!dY || !X || !mean || !rstd || (!dX && !dweight && !dbias)) return BITLINEAR_ERR_NULL;
  int st = check_mk(M, K);
  if (st) return st;
  if (!plain_dtype(dy_dtype)) return BITLINEAR_ERR_DTYPE;
  st = check_in(X, x_scales, x_dtype);
  if (st) return st;
  if (dX && !plain_dtype(dx_dtype)) return BITLINEAR_ERR_DTYPE;
  if (!aligned_to(dY, dy_dtype) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(weight, 4) ||
      (dX && !aligned_to(dX, dx_dtype)) || !aligned(dweight, 4) || !aligned(dbias, 4))
    return BITLINEAR_ERR_ALIGN;
  const size_t need = dweight || dbias ? ln_bwd_workspace_bytes(M, K) : 0;
  if (need) {
    if (!workspace || workspace_bytes < need) return BITLINEAR_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return BITLINEAR_ERR_ALIGN;
  }
  const BlockIn x = block_in(X, x_scales, x_dtype);
  const Range out[] = {array(dX, dx_dtype, M, K), floats(dweight, K), floats(dbias, K),
                       {need ? workspace : nullptr, need}};
  const Range in[] = {array(dY, dy_dtype, M, K), array(X, x_dtype, M, K), scale_range(x.scales, M, K),
                      floats(mean, M), floats(rstd, M), floats(weight, K)};
  if (any_overlap(out, in)) return BITLINEAR_ERR_ARG;
  return hip_status(launch_layer_norm_backward(dY, dy_dtype, x, mean, rstd, M, K, weight, dX, dx_dtype, dweight,
                                               dbias, workspace, static_cast<hipStream_t>(stream)));
}

int bitlinear_relu2(const void* H, const float* h_scales, int h_dtype, int64_t M, int64_t K, void* A, int a_dtype,
                    int8_t* saved, float* saved_scales, void* stream) {
  if (!H || !A) return BITLINEAR_ERR_NULL;
  int st = check_mk(M, K);
  if (st) return st;
  st = check_in(H, h_scales, h_dtype);
  if (st) return st;
  if (!plain_dtype(a_dtype)) return BITLINEAR_ERR_DTYPE;
  if (!aligned_to(A, a_dtype)) return BITLINEAR_ERR_ALIGN;
  st = check_saved_out(saved, saved_scales, h_dtype);
  if (st) return st;
  const BlockIn h = block_in(H, h_scales, h_dtype);
  const Range out[] = {array(A, a_dtype, M, K), array(saved, BITLINEAR_SAVED8, M, K), scale_range(saved_scales, M, K)};
  const Range in[] = {array(H, h_dtype, M, K), scale_range(h.scales, M, K)};
  if (any_overlap(out, in)) return BITLINEAR_ERR_ARG;
  return hip_status(launch_relu2(h, M, K, A, a_dtype, saved, saved_scales, static_cast<hipStream_t>(stream)));
}

int bitlinear_relu2_backward(const void* dA, int da_dtype, const void* H, const float* h_scales, int h_dtype,
                             int64_t M, int64_t K, void* dH, int dh_dtype, void* stream) {
  if (!dA || !H || !dH) return BITLINEAR_ERR_NULL;
  int st = check_mk(M, K);
  if (st) return st;
  if (!plain_dtype(da_dtype) || !plain_dtype(dh_dtype)) return BITLINEAR_ERR_DTYPE;
  st = check_in(H, h_scales, h_dtype);
  if (st) return st;
  if (!aligned_to(dA, da_dtype) || !aligned_to(dH, dh_dtype)) return BITLINEAR_ERR_ALIGN;
  const BlockIn h = block_in(H, h_scales, h_dtype);
  const Range out[] = {array(dH, dh_dtype, M, K)};
  const Range in[] = {array(dA, da_dtype, M, K), array(H, h_dtype, M, K), scale_range(h.scales, M, K)};
  if (any_overlap(out, in)) return BITLINEAR_ERR_ARG;
  return hip_status(launch_relu2_backward(dA, da_dtype, h, M, K, dH, dh_dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
