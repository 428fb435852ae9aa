// C ABI of the low-rank adapters and of dropout (include/bitlinear_adapters.h):
// argument checks on the host, then the launches.
#include <stdint.h>

#include "../../include/bitlinear_adapters.h"
#include "abi_common.hpp"
#include "adapter_ops.hpp"
#include "prefill_parts.hpp"

using namespace bitlinear;

namespace {

// Sizes, types and alignment that every adapter call shares.
int check_adapters(int64_t M, int64_t K, int64_t N, int64_t A, int64_t R, const void* down, const void* up, int w_dtype,
                   const float* scales, const int32_t* rows) {
  const int st = check_mnk(M, N, K);
  if (st) return st;
  if (A < 1 || A > kAdapterMaxA || R < 1 || R > kAdapterMaxR) return BITLINEAR_ERR_SHAPE;
  const int64_t C = K > N ? K : N, lim = int64_t(1) << 40;
  if (A * R * C >= lim || M * R >= lim) return BITLINEAR_ERR_SHAPE;
  if (!plain_dtype(w_dtype)) return BITLINEAR_ERR_DTYPE;
  if (!aligned_to(down, w_dtype) || !aligned_to(up, w_dtype) || !aligned(scales, 4) || !aligned(rows, 4))
    return BITLINEAR_ERR_ALIGN;
  return BITLINEAR_OK;
}

Range weights(const void* p, int w_dtype, int64_t A, int64_t R, int64_t C) { return array(p, w_dtype, A * R, C); }
Range ids(const int32_t* rows, int64_t M) { return {rows, 4 * static_cast<uint64_t>(M)}; }

// The planes behind a first product's parts.
uint16_t* planes_of(void* ws, int64_t M, int64_t C, int64_t R) {
  return reinterpret_cast<uint16_t*>(static_cast<char*>(ws) + parts_ws_bytes(M, C, R));
}

int add_adapters(const void* X, int x_dtype, int64_t M, int64_t K, int64_t N, const Adapters& ad, const void* down,
                 const void* up, float* Y, float* T, void* ws, hipStream_t s) {
  float* parts = static_cast<float*>(ws);
  const hipError_t e = launch_shrink(X, x_dtype, M, K, ad, down, parts, s);
  if (e != hipSuccess) return BITLINEAR_ERR_HIP;
  uint16_t* planes = planes_of(ws, M, K, ad.R);
  return hip_status(launch_expand(parts, planes, M, K, N, ad, up, Y, true, T, s));
}

}  // namespace

extern "C" {

size_t bitlinear_adapters_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t R) {
  return size_args_ok(N) ? adapters_ws_bytes(M, K, R) : 0;
}

int bitlinear_adapters_forward(const void* X, int x_dtype, int64_t M, int64_t K, int64_t N, const int32_t* rows,
                               int64_t A, int64_t R, const void* down, const void* up, int w_dtype,
                               const float* scales, float* Y, float* T, void* workspace, size_t workspace_bytes,
                               void* stream) {
  if (!X || !rows || !down || !up || !scales || !Y) return BITLINEAR_ERR_NULL;
  int st = check_adapters(M, K, N, A, R, down, up, w_dtype, scales, rows);
  if (st) return st;
  st = check_x(X, x_dtype);
  if (st) return st;
  if (!aligned(Y, 4) || !aligned(T, 4)) return BITLINEAR_ERR_ALIGN;
  const size_t need = adapters_ws_bytes(M, K, R);
  if (!workspace || workspace_bytes < need) return BITLINEAR_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return BITLINEAR_ERR_ALIGN;
  const Range out[] = {floats(Y, M * N), floats(T, M * R), {workspace, need}};
  const Range in[] = {array(X, x_dtype, M, K), ids(rows, M), weights(down, w_dtype, A, R, K),
                      weights(up, w_dtype, A, R, N), floats(scales, A)};
  if (any_overlap(out, in)) return BITLINEAR_ERR_ARG;
  const Adapters ad = {rows, scales, static_cast<int>(A), static_cast<int>(R), w_dtype};
  return add_adapters(X, x_dtype, M, K, N, ad, down, up, Y, T, workspace, static_cast<hipStream_t>(stream));
}

size_t bitlinear_adapted_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t R) {
  if (!size_args_ok(N)) return 0;
  const size_t all = size_add(adapters_ws_bytes(M, K, R), prefill_ws_bytes(M, K)), sums = prefill_parts_bytes(M, N, K);
  return sums ? size_add(all, sums) : all;
}

int bitlinear_adapted_forward(const void* X, int x_dtype, int64_t M, int64_t K, const uint32_t* packed, int64_t N,
                              const float* gamma, const int32_t* rows, int64_t A, int64_t R, const void* down,
                              const void* up, int w_dtype, const float* scales, float* Y, float* T, int path,
                              void* workspace, size_t workspace_bytes, void* stream) {
  if (!X || !packed || !gamma || !rows || !down || !up || !scales || !Y) return BITLINEAR_ERR_NULL;
  int st = check_adapters(M, K, N, A, R, down, up, w_dtype, scales, rows);
  if (st) return st;
  bool decode = false;
  st = check_forward_args(X, x_dtype, M, K, packed, N, gamma, Y, nullptr, path, &decode);
  if (st) return st;
  if (!aligned(T, 4)) return BITLINEAR_ERR_ALIGN;
  const size_t low = adapters_ws_bytes(M, K, R), codes = prefill_ws_bytes(M, K), sums = prefill_parts_bytes(M, N, K);
  const size_t need = low + codes + sums;
  if (!workspace || workspace_bytes < need) return BITLINEAR_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return BITLINEAR_ERR_ALIGN;
  const Range out[] = {floats(Y, M * N), floats(T, M * R), {workspace, need}};
  const Range in[] = {array(X, x_dtype, M, K),
                      {packed, static_cast<uint64_t>(N) * static_cast<uint64_t>(padded_k(K)) / 4},
                      floats(gamma, 1),
                      ids(rows, M),
                      weights(down, w_dtype, A, R, K),
                      weights(up, w_dtype, A, R, N),
                      floats(scales, A)};
  if (any_overlap(out, in)) return BITLINEAR_ERR_ARG;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const Adapters ad = {rows, scales, static_cast<int>(A), static_cast<int>(R), w_dtype};
  const int64_t piece = path == BITLINEAR_PATH_PREFILL ? 0 : adapted_decode_piece(M, K, N);
  hipError_t e;
  const PrefillWs c = prefill_ws(static_cast<char*>(workspace) + low, M, K);
  if (piece)
    return hip_status(launch_adapted_decode(X, x_dtype, M, K, packed, N, gamma, Y, ad, down, up,
                                            static_cast<float*>(workspace), T, piece, c.xq, c.ga, c.rs, s));
  if (!decode && K >= 8) {
    float* parts = static_cast<float*>(workspace);
    uint16_t* planes = planes_of(workspace, M, K, R);
    e = launch_adapted_first(X, x_dtype, M, K, ad, down, parts, c.xq, c.ga, c.rs, s);
    // the second product in the GEMM's epilogue, unless parts of K save more than its
    // own pass over Y costs (16 ranks: 256x4096x4096 33 us and 36, 1024x8192x1024 58
    // and 45)
    if (adapted_gemm_takes(M, N, R) && prefill_parts(M, N, K).saved <= 4000 + M * N / 300) {
      if (e == hipSuccess) e = launch_join(parts, M, K, ad, T, planes, s);
      if (e == hipSuccess) e = launch_adapted_gemm(c.xq, c.ga, c.rs, M, K, packed, N, gamma, Y, planes, ad, up, s);
    } else {
      if (e == hipSuccess && sums)
        e = launch_prefill_parts(c.xq, c.ga, c.rs, M, K, packed, N, gamma, Y,
                                 reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + low + codes), s);
      else if (e == hipSuccess)
        e = launch_prefill_gemm(c.xq, c.ga, c.rs, M, K, packed, N, gamma, Y, nullptr, s);
      if (e == hipSuccess) e = launch_expand(parts, planes, M, K, N, ad, up, Y, true, T, s);
    }
    return hip_status(e);
  }
  if (decode) {
    e = launch_decode(X, x_dtype, M, K, packed, N, gamma, Y, nullptr, 1, s);
  } else {
    e = launch_act_quant(X, x_dtype, M, K, c.xq, c.ga, c.rs, s);
    if (e == hipSuccess) e = launch_prefill_gemm(c.xq, c.ga, c.rs, M, K, packed, N, gamma, Y, nullptr, s);
  }
  if (e != hipSuccess) return BITLINEAR_ERR_HIP;
  return add_adapters(X, x_dtype, M, K, N, ad, down, up, Y, T, workspace, s);
}

size_t bitlinear_adapters_backward_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t A, int64_t R) {
  return adapters_backward_ws_bytes(M, K, N, A, R);
}

int bitlinear_adapters_backward(const void* dY, int dy_dtype, const void* X, int x_dtype, const float* T, int64_t M,
                                int64_t K, int64_t N, const int32_t* rows, int64_t A, int64_t R, const void* down,
                                const void* up, int w_dtype, const float* scales, float* dX, int accumulate,
                                float* ddown, float* dup, void* workspace, size_t workspace_bytes, void* stream) {
  if (!dY || !rows || !down || !up || !scales || (!dX && !ddown && !dup) || (ddown && !X) || (dup && !T))
    return BITLINEAR_ERR_NULL;
  int st = check_adapters(M, K, N, A, R, down, up, w_dtype, scales, rows);
  if (st) return st;
  st = check_x(dY, dy_dtype);
  if (st) return st;
  if (ddown) st = check_x(X, x_dtype);
  if (st) return st;
  if (!aligned(T, 4) || !aligned(dX, 4) || !aligned(ddown, 4) || !aligned(dup, 4)) return BITLINEAR_ERR_ALIGN;
  const size_t need = adapters_backward_ws_bytes(M, K, N, A, R);
  if (!workspace || workspace_bytes < need) return BITLINEAR_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return BITLINEAR_ERR_ALIGN;
  const Range out[] = {floats(dX, M * K), floats(ddown, A * R * K), floats(dup, A * R * N), {workspace, need}};
  const Range in[] = {array(dY, dy_dtype, M, N),        array(ddown ? X : nullptr, x_dtype, M, K),
                      floats(dup ? T : nullptr, M * R), ids(rows, M),
                      weights(down, w_dtype, A, R, K),  weights(up, w_dtype, A, R, N),
                      floats(scales, A)};
  if (any_overlap(out, in)) return BITLINEAR_ERR_ARG;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const Adapters ad = {rows, scales, static_cast<int>(A), static_cast<int>(R), w_dtype};
  char* ws = static_cast<char*>(workspace);
  float* parts = reinterpret_cast<float*>(ws);
  ws += shrink_ws_bytes(M, N, R);
  float* V = reinterpret_cast<float*>(ws);  // without the scale: the gradient's kernel applies it once
  ws += align256(static_cast<size_t>(M) * static_cast<size_t>(R) * 4);
  float* grads = reinterpret_cast<float*>(ws);
  hipError_t e = hipSuccess;
  if (dX || ddown) {
    e = launch_shrink(dY, dy_dtype, M, N, ad, up, parts, s);
    if (e == hipSuccess && dX)
      e = launch_expand(parts, planes_of(workspace, M, N, R), M, N, K, ad, down, dX, accumulate != 0,
                        ddown ? V : nullptr, s);
    else if (e == hipSuccess)
      e = launch_join(parts, M, N, ad, V, nullptr, s);
  }
  if (e == hipSuccess && ddown) e = launch_adapter_grad(V, X, x_dtype, M, K, ad, ddown, grads, s);
  if (e == hipSuccess && dup) e = launch_adapter_grad(T, dY, dy_dtype, M, N, ad, dup, grads, s);
  return hip_status(e);
}

int bitlinear_dropout(const void* X, int x_dtype, const void* residual, int r_dtype, int64_t n, double p,
                      uint64_t seed, uint64_t offset, void* Y, int y_dtype, void* stream) {
  if (!X || !Y) return BITLINEAR_ERR_NULL;
  if (n < 1 || n >= (int64_t(1) << 40)) return BITLINEAR_ERR_SHAPE;
  if (!plain_dtype(x_dtype) || !plain_dtype(y_dtype) || (residual && !plain_dtype(r_dtype))) return BITLINEAR_ERR_DTYPE;
  if (!aligned_to(X, x_dtype) || !aligned_to(Y, y_dtype) || (residual && !aligned_to(residual, r_dtype)))
    return BITLINEAR_ERR_ALIGN;
  if (!(p >= 0.0) || !(p < 1.0)) return BITLINEAR_ERR_ARG;
  // in place, value by value, or apart
  const Range out = array(Y, y_dtype, 1, n);
  if (!(X == Y && x_dtype == y_dtype) && overlap(out, array(X, x_dtype, 1, n))) return BITLINEAR_ERR_ARG;
  if (residual && !(residual == Y && r_dtype == y_dtype) && overlap(out, array(residual, r_dtype, 1, n)))
    return BITLINEAR_ERR_ARG;
  return hip_status(launch_dropout(X, x_dtype, residual, r_dtype, n, p, seed, offset, Y, y_dtype,
                                   static_cast<hipStream_t>(stream)));
}

}  // extern "C"
