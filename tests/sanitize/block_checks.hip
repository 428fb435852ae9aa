// Driver for a host-only build of csrc/block_api.hip under AddressSanitizer and
// UndefinedBehaviorSanitizer: the launchers are stubs that count their calls
// and keep what they were given, nothing touches a GPU.  Every entry point is
// called with bad arguments (nothing may be launched), with arguments at the
// limits of the size arithmetic, with good arguments and with a failing launch.
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "../../bitlinear_absmean_ternarise_bit_amd/csrc/block_ops.hpp"
#include "../../include/bitlinear_block.h"

namespace {
int g_calls = 0, g_run = 0, g_failed = 0;
bool g_fail = false;
char g_name[32];
int64_t g_M = 0, g_K = 0;
bitlinear::BlockIn g_in;

hipError_t record(const char* name, int64_t M, int64_t K, bitlinear::BlockIn in) {
  ++g_calls;
  snprintf(g_name, sizeof(g_name), "%s", name);
  g_M = M;
  g_K = K;
  g_in = in;
  return g_fail ? hipErrorLaunchFailure : hipSuccess;
}

#define CHECK(x)                                            \
  do {                                                      \
    ++g_run;                                                \
    if (!(x)) {                                             \
      ++g_failed;                                           \
      printf("line %d: %s does not hold\n", __LINE__, #x);  \
    }                                                       \
  } while (0)
}  // namespace

namespace bitlinear {
hipError_t launch_save(const void* X, int dt, int64_t M, int64_t K, int8_t*, float*, hipStream_t) {
  return record("save", M, K, {X, nullptr, dt});
}
hipError_t launch_restore(BlockIn in, int64_t M, int64_t K, void*, int, hipStream_t) { return record("restore", M, K, in); }
hipError_t launch_relu2(BlockIn in, int64_t M, int64_t K, void*, int, int8_t*, float*, hipStream_t) {
  return record("relu2", M, K, in);
}
hipError_t launch_relu2_backward(const void*, int, BlockIn in, int64_t M, int64_t K, void*, int, hipStream_t) {
  return record("relu2_backward", M, K, in);
}
hipError_t launch_layer_norm(BlockIn in, int64_t M, int64_t K, const float*, const float*, float, void*, int, float*,
                             float*, int8_t*, float*, hipStream_t) {
  return record("layer_norm", M, K, in);
}
hipError_t launch_layer_norm_backward(const void*, int, BlockIn in, const float*, const float*, int64_t M, int64_t K,
                                      const float*, void*, int, float*, float*, void*, hipStream_t) {
  return record("layer_norm_backward", M, K, in);
}
}  // namespace bitlinear

namespace {
// Fake addresses, never dereferenced: 2^44 bytes apart, farther than any array is long.
char* at(int i) { return reinterpret_cast<char*>(uintptr_t(i + 1) << 44); }
template <typename T>
T* as(int i) {
  return reinterpret_cast<T*>(at(i));
}

int save(const void* X, int dt, int64_t M, int64_t K, void* codes = at(1), void* scales = at(2)) {
  return bitlinear_save_activations(X, dt, M, K, static_cast<int8_t*>(codes), static_cast<float*>(scales), nullptr);
}
int restore(const void* codes, const void* scales, int64_t M, int64_t K, void* X, int dt) {
  return bitlinear_restore_activations(static_cast<const int8_t*>(codes), static_cast<const float*>(scales), M, K, X,
                                       dt, nullptr);
}
int norm(int dt, const float* xs, int64_t M, int64_t K, float eps = 1e-5f, void* Y = at(3), float* mean = as<float>(4),
         float* rstd = as<float>(5), int8_t* saved = nullptr, float* ss = nullptr) {
  return bitlinear_layer_norm(at(0), xs, dt, M, K, as<float>(1), as<float>(2), eps, Y, 1, mean, rstd, saved, ss, nullptr);
}
int norm_bwd(int dt, const float* xs, int64_t M, int64_t K, void* dX, float* dw, float* db, void* ws, size_t wsb) {
  return bitlinear_layer_norm_backward(at(0), 0, at(1), xs, dt, as<float>(2), as<float>(3), M, K, nullptr, dX, 1, dw,
                                       db, ws, wsb, nullptr);
}
int relu(int dt, const float* hs, int64_t M, int64_t K, void* A = at(3), int8_t* saved = nullptr, float* ss = nullptr) {
  return bitlinear_relu2(at(0), hs, dt, M, K, A, 0, saved, ss, nullptr);
}
int relu_bwd(int dt, const float* hs, int64_t M, int64_t K, void* dH = at(3)) {
  return bitlinear_relu2_backward(at(1), 1, at(0), hs, dt, M, K, dH, 1, nullptr);
}
}  // namespace

int main() {
  const int64_t I64MAX = INT64_MAX, I64MIN = INT64_MIN, M31 = int64_t(1) << 31, K20 = int64_t(1) << 20;
  const int64_t bad[][2] = {{0, 8},          {8, 0},          {-1, 8},           {8, -1},     {M31 + 1, 1},
                            {8, K20 + 1},    {K20, K20},      {I64MAX, I64MAX},  {I64MAX, 1}, {1, I64MAX},
                            {I64MIN, I64MIN}, {M31, 512},     {int64_t(1) << 21, int64_t(1) << 19}};
  for (auto& s : bad) {
    CHECK(save(at(0), 0, s[0], s[1]) == BITLINEAR_ERR_SHAPE);
    CHECK(restore(at(0), at(1), s[0], s[1], at(2), 0) == BITLINEAR_ERR_SHAPE);
    CHECK(norm(0, nullptr, s[0], s[1]) == BITLINEAR_ERR_SHAPE);
    CHECK(norm_bwd(0, nullptr, s[0], s[1], at(4), as<float>(5), as<float>(6), at(7), SIZE_MAX) == BITLINEAR_ERR_SHAPE);
    CHECK(relu(0, nullptr, s[0], s[1]) == BITLINEAR_ERR_SHAPE);
    CHECK(relu_bwd(0, nullptr, s[0], s[1]) == BITLINEAR_ERR_SHAPE);
  }
  for (int dt : {-1, 3, INT32_MAX, INT32_MIN}) {
    CHECK(save(at(0), dt, 2, 8) == BITLINEAR_ERR_DTYPE);
    CHECK(restore(at(0), at(1), 2, 8, at(2), dt) == BITLINEAR_ERR_DTYPE);
    CHECK(norm(dt, nullptr, 2, 8) == BITLINEAR_ERR_DTYPE);
    CHECK(norm_bwd(dt, nullptr, 2, 8, at(4), nullptr, nullptr, nullptr, 0) == BITLINEAR_ERR_DTYPE);
    CHECK(relu(dt, nullptr, 2, 8) == BITLINEAR_ERR_DTYPE);
    CHECK(relu_bwd(dt, nullptr, 2, 8) == BITLINEAR_ERR_DTYPE);
  }
  CHECK(save(at(0), BITLINEAR_SAVED8, 2, 8) == BITLINEAR_ERR_DTYPE);
  for (float eps : {-1.0f, -1e-30f, NAN, INFINITY, -INFINITY}) CHECK(norm(0, nullptr, 2, 8, eps) == BITLINEAR_ERR_ARG);
  CHECK(norm(2, nullptr, 2, 8) == BITLINEAR_ERR_NULL);
  CHECK(norm(2, as<float>(9), 2, 8, 1e-5f, at(3), as<float>(4), as<float>(5), as<int8_t>(6), as<float>(7)) ==
        BITLINEAR_ERR_ARG);
  CHECK(norm(0, nullptr, 2, 8, 1e-5f, at(3), nullptr) == BITLINEAR_ERR_NULL);
  CHECK(norm(0, nullptr, 2, 8, 1e-5f, at(3), as<float>(4), as<float>(5), as<int8_t>(6), nullptr) == BITLINEAR_ERR_NULL);
  CHECK(relu(2, as<float>(9), 2, 8, at(3), as<int8_t>(6), as<float>(7)) == BITLINEAR_ERR_ARG);
  CHECK(norm_bwd(0, nullptr, 2, 8, nullptr, nullptr, nullptr, nullptr, 0) == BITLINEAR_ERR_NULL);
  // overlaps: the first and the last byte of an array, and none one byte past it
  CHECK(save(at(0), 1, 5, 100, at(0) + 992) == BITLINEAR_ERR_ARG);  // X: 1000 bytes
  CHECK(norm(1, nullptr, 5, 100, 1e-5f, at(0) + 998) == BITLINEAR_ERR_ARG);
  CHECK(norm(1, nullptr, 5, 100, 1e-5f, at(0) - 2) == BITLINEAR_ERR_ARG);
  CHECK(relu_bwd(2, as<float>(9), 5, 100, at(9) + 5 * 2 * 4 - 2) == BITLINEAR_ERR_ARG);  // the last scale
  CHECK(g_calls == 0);

  const size_t need = bitlinear_layer_norm_backward_workspace_bytes(5000, 100);
  CHECK(need > 0 && need % 256 == 0);
  CHECK(norm_bwd(0, nullptr, 5000, 100, nullptr, as<float>(5), nullptr, nullptr, need) == BITLINEAR_ERR_WORKSPACE);
  CHECK(norm_bwd(0, nullptr, 5000, 100, nullptr, nullptr, as<float>(5), at(7), need - 1) == BITLINEAR_ERR_WORKSPACE);
  CHECK(norm_bwd(0, nullptr, 5000, 100, nullptr, as<float>(5), nullptr, at(7) + 128, need) == BITLINEAR_ERR_ALIGN);
  CHECK(norm_bwd(0, nullptr, 5000, 100, at(7) + need - 4, as<float>(5), nullptr, at(7), need) == BITLINEAR_ERR_ARG);
  CHECK(g_calls == 0);

  // good calls, the largest sizes among them
  const int64_t good[][2] = {{1, 1}, {5, 100}, {M31, 511}, {K20 - 1, K20}, {M31, 1}, {1, K20}};
  int n = 0;
  for (auto& s : good) {
    const int64_t M = s[0], K = s[1];
    const size_t ws = bitlinear_layer_norm_backward_workspace_bytes(M, K);
    CHECK(ws <= size_t(256) * 8 * K + 255);
    CHECK(save(at(0), 0, M, K) == BITLINEAR_OK && g_calls == ++n && !strcmp(g_name, "save") && g_M == M && g_K == K);
    CHECK(restore(at(0), at(1), M, K, at(2), 1) == BITLINEAR_OK && g_calls == ++n && g_in.dtype == 2 &&
          g_in.scales == as<float>(1));
    CHECK(norm(1, as<float>(1), M, K) == BITLINEAR_OK && g_calls == ++n && !g_in.scales);  // scales not taken
    CHECK(norm(0, nullptr, M, K, 0.0f, at(3), nullptr, nullptr, as<int8_t>(6), as<float>(7)) == BITLINEAR_OK &&
          g_calls == ++n);
    CHECK(norm_bwd(2, as<float>(8), M, K, at(4), as<float>(5), as<float>(6), at(7), ws) == BITLINEAR_OK &&
          g_calls == ++n && g_in.scales == as<float>(8));
    CHECK(norm_bwd(1, nullptr, M, K, at(4), nullptr, nullptr, nullptr, 0) == BITLINEAR_OK && g_calls == ++n);
    CHECK(relu(0, nullptr, M, K, at(3), as<int8_t>(6), as<float>(7)) == BITLINEAR_OK && g_calls == ++n);
    CHECK(relu_bwd(2, as<float>(8), M, K) == BITLINEAR_OK && g_calls == ++n && !strcmp(g_name, "relu2_backward"));
  }
  CHECK(norm(1, nullptr, 5, 100, 1e-5f, at(0) + 1000) == BITLINEAR_OK && g_calls == ++n);  // right behind X
  g_fail = true;
  CHECK(save(at(0), 0, 2, 8) == BITLINEAR_ERR_HIP);
  CHECK(restore(at(0), at(1), 2, 8, at(2), 0) == BITLINEAR_ERR_HIP);
  CHECK(norm(0, nullptr, 2, 8) == BITLINEAR_ERR_HIP);
  CHECK(norm_bwd(0, nullptr, 2, 8, at(4), nullptr, nullptr, nullptr, 0) == BITLINEAR_ERR_HIP);
  CHECK(relu(0, nullptr, 2, 8) == BITLINEAR_ERR_HIP);
  CHECK(relu_bwd(0, nullptr, 2, 8) == BITLINEAR_ERR_HIP);

  // every plan: a row fits its team, a workgroup fits 16 waves, every row has a team, sizes agree
  for (int64_t K = 1; K <= 40000; K = K < 200 ? K + 1 : K + 61)
    for (int64_t M : {int64_t(1), int64_t(2), int64_t(3), int64_t(16), int64_t(33), int64_t(255), int64_t(257),
                      int64_t(5000), M31})
      for (bool params : {false, true}) {
        const bitlinear::LnBwdPlan p = bitlinear::ln_bwd_plan(M, K, params);
        bool ok = p.groups >= 1 && p.groups <= 256;
        if (p.waves > 0)
          ok = ok && int64_t(64) * p.waves * p.chunks * 8 >= K && p.waves * p.teams <= (p.chunks == 1 ? 16 : 8) &&
               p.teams >= 1 && (p.groups == 256 || int64_t(p.groups) * p.teams * (params ? 2 : 1) >= M);
        CHECK(ok);
        const size_t w = bitlinear_layer_norm_backward_workspace_bytes(M, K);
        if (params) CHECK(ln_bwd_alone(p, K) ? w == 0 : w >= size_t(p.groups) * 8 * K);
      }
  printf("%d checks, %d failed\n", g_run, g_failed);
  return g_failed != 0;
}
