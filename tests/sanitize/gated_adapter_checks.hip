// Driver for a host-only build of csrc/gated_api.hip and csrc/adapter_api.hip under
// AddressSanitizer and UndefinedBehaviorSanitizer: the launchers are stubs
// (launch_stub.hip has those that other calls share), nothing touches a GPU.
// Every entry point is called with bad arguments (nothing may be launched), with
// arguments at the limits of the size arithmetic, with good arguments and with a
// failing launch.
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "../../bitlinear_absmean_ternarise_bit_amd/csrc/adapter_ops.hpp"
#include "../../bitlinear_absmean_ternarise_bit_amd/csrc/gated_ops.hpp"
#include "../../bitlinear_absmean_ternarise_bit_amd/csrc/prefill_parts.hpp"
#include "../../include/bitlinear_adapters.h"
#include "../../include/bitlinear_gated.h"
#include "stub.h"

namespace {
int g_run = 0, g_failed = 0;
int64_t g_piece = 0;
bool g_fail = false;
char g_calls[256];  // this driver's own launchers, in order

hipError_t record(const char* name) {
  strncat(g_calls, name, sizeof(g_calls) - strlen(g_calls) - 2);
  strcat(g_calls, " ");
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
hipError_t launch_gated_decode(const void*, int, const int8_t*, const float*, const int32_t*, int64_t, int64_t, int64_t,
                               const GatedWeights&, const GatedOutputs&, hipStream_t) {
  return record("gated_decode");
}
hipError_t launch_gated_gemm(const int8_t*, const float*, const int32_t*, int64_t, int64_t, int64_t, const GatedWeights&,
                             const GatedOutputs&, hipStream_t) {
  return record("gated_gemm");
}
hipError_t launch_prefill_parts(const int8_t*, const float*, const int32_t*, int64_t, int64_t, const uint32_t*, int64_t,
                                const float*, float*, int32_t*, hipStream_t) {
  return record("parts");
}
hipError_t launch_gated_backward(const void*, int, const void*, const void*, int, int64_t, int64_t, int, void*, void*,
                                 int, hipStream_t) {
  return record("gated_backward");
}
hipError_t launch_gated_input_backward(const uint16_t*, const uint16_t*, int64_t, int64_t, int64_t, const uint32_t*,
                                       const float*, const uint32_t*, const float*, float*, float*, void* copies, hipStream_t) {
  return record(copies ? "dx_copies" : "dx");
}
int64_t adapted_decode_piece(int64_t, int64_t, int64_t) { return g_piece; }
hipError_t launch_adapted_decode(const void*, int, int64_t, int64_t, const uint32_t*, int64_t, const float*, float*,
                                 const Adapters&, const void*, const void*, float*, float*, int64_t, int8_t*, float*,
                                 int32_t*, hipStream_t) {
  return record("adapted_decode");
}
hipError_t launch_adapted_first(const void*, int, int64_t, int64_t, const Adapters&, const void*, float*, int8_t*,
                                float*, int32_t*, hipStream_t) {
  return record("first");
}
hipError_t launch_adapted_gemm(const int8_t*, const float*, const int32_t*, int64_t, int64_t, const uint32_t*, int64_t,
                               const float*, float*, const uint16_t*, const Adapters&, const void*, hipStream_t) {
  return record("adapted_gemm");
}
hipError_t launch_shrink(const void*, int, int64_t, int64_t, const Adapters&, const void*, float*, hipStream_t) {
  return record("shrink");
}
hipError_t launch_expand(const float*, uint16_t*, int64_t, int64_t, int64_t, const Adapters&, const void*, float*, bool,
                         float*, hipStream_t) {
  return record("expand");
}
hipError_t launch_join(const float*, int64_t, int64_t, const Adapters&, float*, uint16_t*, hipStream_t) {
  return record("join");
}
hipError_t launch_adapter_grad(const float*, const void*, int, int64_t, int64_t, const Adapters&, float*, float*,
                               hipStream_t) {
  return record("grad");
}
hipError_t launch_dropout(const void*, int, const void*, int, int64_t, double, uint64_t, uint64_t, void*, int,
                          hipStream_t) {
  return record("dropout");
}
}  // namespace bitlinear

namespace {
// Fake addresses, never dereferenced: 2^44 bytes apart, farther than any array is long.
char* at(int i) { return reinterpret_cast<char*>(uintptr_t(i + 1) << 44); }
template <typename T>
T* as(int i) {
  return reinterpret_cast<T*>(at(i));
}

struct Gated {
  const void* X = at(0);
  int xt = 0, act = 0, ht = 0, gut = 0, path = BITLINEAR_PATH_AUTO;
  void *H = at(5), *G = nullptr, *U = nullptr, *ws = at(8);
  size_t wsb = SIZE_MAX;
  int run(int64_t M, int64_t D, int64_t F) const {
    return bitlinear_gated_forward(X, xt, M, D, F, as<uint32_t>(1), as<float>(2), as<uint32_t>(3), as<float>(4), act, H,
                                   ht, G, U, gut, path, ws, wsb, nullptr);
  }
  int codes(int64_t M, int64_t D, int64_t F) const {
    return bitlinear_gated_forward_quantized(as<int8_t>(0), as<float>(9), as<int32_t>(10), M, D, F, as<uint32_t>(1),
                                             as<float>(2), as<uint32_t>(3), as<float>(4), act, H, ht, G, U, gut,
                                             nullptr);
  }
  int block(int64_t M, int64_t D, int64_t F, int64_t O, float* hidden = nullptr) const {
    return bitlinear_gated_ffn_forward(X, xt, M, D, F, O, as<uint32_t>(1), as<float>(2), as<uint32_t>(3), as<float>(4),
                                       act, as<uint32_t>(6), as<float>(7), static_cast<float*>(H), hidden, path, ws,
                                       wsb, nullptr);
  }
  int back(int64_t M, int64_t F, int dt = 1) const {
    return bitlinear_gated_backward(at(0), xt, at(1), at(2), gut, M, F, act, H, at(6), dt, nullptr);
  }
};

int dx(int64_t M, int64_t F, int64_t D, int skew, void* ws, size_t wsb, float* out = as<float>(5)) {
  return bitlinear_gated_input_backward(as<uint16_t>(0) + skew, as<uint16_t>(6), M, F, D, as<uint32_t>(1), as<float>(2),
                                        as<uint32_t>(3), as<float>(4), out, ws, wsb, nullptr);
}

struct Low {
  const void *X = at(0), *down = at(2), *up = at(3);
  int xt = 0, wt = 0, path = BITLINEAR_PATH_AUTO;
  const int32_t* rows = as<int32_t>(1);
  const float* scales = as<float>(4);
  float *Y = as<float>(5), *T = as<float>(6);
  void* ws = at(7);
  size_t wsb = SIZE_MAX;
  int run(int64_t M, int64_t K, int64_t N, int64_t A, int64_t R) const {
    return bitlinear_adapters_forward(X, xt, M, K, N, rows, A, R, down, up, wt, scales, Y, T, ws, wsb, nullptr);
  }
  int whole(int64_t M, int64_t K, int64_t N, int64_t A, int64_t R) const {
    return bitlinear_adapted_forward(X, xt, M, K, as<uint32_t>(8), N, as<float>(9), rows, A, R, down, up, wt, scales, Y,
                                     T, path, ws, wsb, nullptr);
  }
  int back(int64_t M, int64_t K, int64_t N, int64_t A, int64_t R, float* dX, float* dd, float* du, int acc = 0) const {
    return bitlinear_adapters_backward(at(13), xt, X, xt, T, M, K, N, rows, A, R, down, up, wt, scales, dX, acc, dd, du,
                                       ws, wsb, nullptr);
  }
};

int drop(const void* X, int xt, const void* r, int rt, int64_t n, double p, void* Y, int yt) {
  return bitlinear_dropout(X, xt, r, rt, n, p, 1, 2, Y, yt, nullptr);
}

bool none() { return stub_count() == 0 && !g_calls[0]; }
// What the last calls launched: the shared stub's count, and this driver's names.
bool launched(int shared, const char* own) {
  const bool ok = stub_count() == shared && !strcmp(g_calls, own);
  if (!ok) printf("launched %d and '%s'\n", stub_count(), g_calls);
  stub_reset(-1);
  g_calls[0] = 0;
  return ok;
}
}  // namespace

int main() {
  const int64_t I64MAX = INT64_MAX, I64MIN = INT64_MIN, M31 = int64_t(1) << 31, K20 = int64_t(1) << 20;
  stub_reset(-1);
  const Gated g;
  const Low l;
  float *dX = as<float>(10), *dd = as<float>(11), *du = as<float>(12);

  // sizes: each dimension out of range, and their products
  const int64_t bad[][3] = {{0, 8, 8},           {8, 0, 8},           {8, 8, 0},         {-1, 8, 8},  {8, -1, 8},
                            {8, 8, -1},          {M31 + 1, 1, 1},     {8, K20 + 1, 8},   {1, 8, M31 + 1},
                            {1, K20, 1 << 13},   {I64MAX, 8, 8},      {8, I64MAX, 8},    {8, 8, I64MAX},
                            {I64MIN, I64MIN, 1}, {I64MAX, I64MAX, I64MAX}, {M31, 512, 1}, {M31, 1, 512}};
  for (auto& s : bad) {
    CHECK(g.run(s[0], s[1], s[2]) == BITLINEAR_ERR_SHAPE);
    CHECK(g.codes(s[0], s[1], s[2]) == BITLINEAR_ERR_SHAPE);
    CHECK(g.block(s[0], s[1], s[2], 8) == BITLINEAR_ERR_SHAPE);
    CHECK(dx(s[0], s[1], s[2], 0, at(8), SIZE_MAX) == BITLINEAR_ERR_SHAPE);
    CHECK(l.run(s[0], s[1], s[2], 4, 8) == BITLINEAR_ERR_SHAPE);
    CHECK(l.whole(s[0], s[1], s[2], 4, 8) == BITLINEAR_ERR_SHAPE);
    CHECK(l.back(s[0], s[1], s[2], 4, 8, dX, dd, du) == BITLINEAR_ERR_SHAPE);
  }
  CHECK(g.block(8, 8, 8, 0) == BITLINEAR_ERR_SHAPE && g.block(8, 8, K20 + 1, 8) == BITLINEAR_ERR_SHAPE);
  const int64_t bad2[][2] = {{0, 8}, {8, 0}, {M31 + 1, 1}, {8, K20 + 1}, {I64MAX, I64MAX}, {M31, 512}, {I64MIN, 1}};
  for (auto& s : bad2) CHECK(g.back(s[0], s[1]) == BITLINEAR_ERR_SHAPE);
  const int64_t badAR[][2] = {{0, 8}, {4, 0}, {-1, 8}, {4, -1}, {65536, 8}, {4, 257}, {I64MAX, 256}, {4, I64MAX}, {I64MIN, I64MIN}};
  for (auto& s : badAR) {
    CHECK(l.run(8, 8, 8, s[0], s[1]) == BITLINEAR_ERR_SHAPE);
    CHECK(l.whole(8, 8, 8, s[0], s[1]) == BITLINEAR_ERR_SHAPE);
    CHECK(l.back(8, 8, 8, s[0], s[1], dX, dd, du) == BITLINEAR_ERR_SHAPE);
  }
  CHECK(l.run(8, K20, 8, 65535, 17) == BITLINEAR_ERR_SHAPE && l.run(8, 8, K20, 65535, 17) == BITLINEAR_ERR_SHAPE);
  CHECK(l.run(M31, 8, 8, 4, 256) == BITLINEAR_OK && launched(0, "shrink expand "));  // 2^39 values of T
  CHECK(dx(1 << 20, 1024, 8, 0, at(8), SIZE_MAX) == BITLINEAR_ERR_SHAPE);  // M * padded F = 2^30
  for (int64_t n : {int64_t(0), int64_t(-1), int64_t(1) << 40, I64MAX, I64MIN})
    CHECK(drop(at(0), 0, nullptr, 0, n, 0.5, at(1), 0) == BITLINEAR_ERR_SHAPE);
  for (double p : {-0.1, -1e-300, 1.0, 1.5, double(INFINITY), -double(INFINITY), double(NAN)})
    CHECK(drop(at(0), 0, nullptr, 0, 64, p, at(1), 0) == BITLINEAR_ERR_ARG);

  // types, activations, paths
  for (int dt : {-1, 2, 3, INT32_MAX, INT32_MIN}) {
    Gated b;
    b.xt = dt;
    CHECK(b.run(2, 8, 8) == BITLINEAR_ERR_DTYPE && b.block(2, 8, 8, 8) == BITLINEAR_ERR_DTYPE);
    CHECK(b.back(2, 8) == BITLINEAR_ERR_DTYPE && g.back(2, 8, dt) == BITLINEAR_ERR_DTYPE);
    b = Gated();
    b.ht = dt;
    CHECK(b.run(2, 8, 8) == BITLINEAR_ERR_DTYPE && b.codes(2, 8, 8) == BITLINEAR_ERR_DTYPE);
    b = Gated();
    b.gut = dt;
    CHECK(b.back(2, 8) == BITLINEAR_ERR_DTYPE);
    b.G = at(6), b.U = at(7);
    CHECK(b.run(2, 8, 8) == BITLINEAR_ERR_DTYPE && b.codes(2, 8, 8) == BITLINEAR_ERR_DTYPE);
    b = Gated();
    b.act = dt;
    CHECK(b.run(2, 8, 8) == BITLINEAR_ERR_ARG && b.codes(2, 8, 8) == BITLINEAR_ERR_ARG);
    CHECK(b.block(2, 8, 8, 8) == BITLINEAR_ERR_ARG && b.back(2, 8) == BITLINEAR_ERR_ARG);
    Low c;
    c.xt = dt;
    CHECK(c.run(2, 8, 8, 4, 8) == BITLINEAR_ERR_DTYPE && c.whole(2, 8, 8, 4, 8) == BITLINEAR_ERR_DTYPE);
    CHECK(c.back(2, 8, 8, 4, 8, dX, dd, du) == BITLINEAR_ERR_DTYPE);
    c = Low();
    c.wt = dt;
    CHECK(c.run(2, 8, 8, 4, 8) == BITLINEAR_ERR_DTYPE && c.whole(2, 8, 8, 4, 8) == BITLINEAR_ERR_DTYPE);
    CHECK(c.back(2, 8, 8, 4, 8, dX, dd, du) == BITLINEAR_ERR_DTYPE);
    CHECK(drop(at(0), dt, nullptr, 0, 64, 0.5, at(1), 0) == BITLINEAR_ERR_DTYPE);
    CHECK(drop(at(0), 0, at(2), dt, 64, 0.5, at(1), 0) == BITLINEAR_ERR_DTYPE);
    CHECK(drop(at(0), 0, nullptr, 0, 64, 0.5, at(1), dt) == BITLINEAR_ERR_DTYPE);
  }
  for (int path : {-1, 3, INT32_MAX, INT32_MIN}) {
    Gated b;
    b.path = path;
    CHECK(b.run(2, 8, 8) == BITLINEAR_ERR_ARG && b.block(2, 8, 8, 8) == BITLINEAR_ERR_ARG);
    Low c;
    c.path = path;
    CHECK(c.whole(2, 8, 8, 4, 8) == BITLINEAR_ERR_ARG);
  }
  {
    Gated b;
    b.path = BITLINEAR_PATH_DECODE;
    CHECK(b.run(17, 8, 8) == BITLINEAR_ERR_SHAPE && b.block(17, 8, 8, 8) == BITLINEAR_ERR_SHAPE);
    CHECK(b.run(1, 200000, 8) == BITLINEAR_ERR_SHAPE && b.block(1, 8, 200000, 8) == BITLINEAR_ERR_SHAPE);
    Low c;
    c.path = BITLINEAR_PATH_DECODE;
    CHECK(c.whole(17, 8, 8, 4, 8) == BITLINEAR_ERR_SHAPE);
  }

  // one pointer at a time missing, and half of a pair
  {
    Gated b;
    b.X = nullptr;
    CHECK(b.run(2, 8, 8) == BITLINEAR_ERR_NULL && b.block(2, 8, 8, 8) == BITLINEAR_ERR_NULL);
    b = Gated();
    b.H = nullptr;
    CHECK(b.run(2, 8, 8) == BITLINEAR_ERR_NULL && b.codes(2, 8, 8) == BITLINEAR_ERR_NULL);
    CHECK(b.block(2, 8, 8, 8) == BITLINEAR_ERR_NULL && b.back(2, 8) == BITLINEAR_ERR_NULL);
    b = Gated();
    b.G = at(6);
    CHECK(b.run(2, 8, 8) == BITLINEAR_ERR_NULL && b.codes(2, 8, 8) == BITLINEAR_ERR_NULL);
    b = Gated();
    b.U = at(6);
    CHECK(b.run(2, 8, 8) == BITLINEAR_ERR_NULL && b.codes(2, 8, 8) == BITLINEAR_ERR_NULL);
    CHECK(dx(2, 8, 8, 0, at(8), SIZE_MAX, nullptr) == BITLINEAR_ERR_NULL);
    for (int i = 0; i < 6; ++i) {
      Low c;
      if (i == 0) c.X = nullptr;
      if (i == 1) c.rows = nullptr;
      if (i == 2) c.down = nullptr;
      if (i == 3) c.up = nullptr;
      if (i == 4) c.scales = nullptr;
      if (i == 5) c.Y = nullptr;
      CHECK(c.run(2, 8, 8, 4, 8) == BITLINEAR_ERR_NULL && c.whole(2, 8, 8, 4, 8) == BITLINEAR_ERR_NULL);
      if (i < 5) CHECK(c.back(2, 8, 8, 4, 8, dX, dd, du) == BITLINEAR_ERR_NULL);
    }
    Low c;
    c.T = nullptr;
    CHECK(c.back(2, 8, 8, 4, 8, nullptr, nullptr, du) == BITLINEAR_ERR_NULL);
    CHECK(l.back(2, 8, 8, 4, 8, nullptr, nullptr, nullptr) == BITLINEAR_ERR_NULL);
    CHECK(drop(nullptr, 0, nullptr, 0, 64, 0.5, at(1), 0) == BITLINEAR_ERR_NULL);
    CHECK(drop(at(0), 0, nullptr, 0, 64, 0.5, nullptr, 0) == BITLINEAR_ERR_NULL);
  }
  CHECK(none());

  // alignment: element sizes, 16 bytes for the hidden layer, 256 for workspaces
  {
    Gated b;
    b.X = at(0) + 2;
    CHECK(b.run(2, 8, 8) == BITLINEAR_ERR_ALIGN && b.block(2, 8, 8, 8) == BITLINEAR_ERR_ALIGN);
    CHECK(g.block(2, 8, 8, 8, as<float>(9) + 1) == BITLINEAR_ERR_ALIGN);
    b = Gated();
    b.ws = at(8) + 128;
    CHECK(b.run(20, 8, 8) == BITLINEAR_ERR_ALIGN && b.block(2, 8, 8, 8) == BITLINEAR_ERR_ALIGN);
    CHECK(dx(2, 9, 8, 0, at(8) + 128, SIZE_MAX) == BITLINEAR_ERR_ALIGN);
    Low c;
    c.ws = at(7) + 128;
    CHECK(c.run(2, 8, 8, 4, 8) == BITLINEAR_ERR_ALIGN && c.whole(2, 8, 8, 4, 8) == BITLINEAR_ERR_ALIGN);
    CHECK(c.back(2, 8, 8, 4, 8, dX, dd, du) == BITLINEAR_ERR_ALIGN);
    c = Low();
    c.down = at(2) + 2;
    CHECK(c.run(2, 8, 8, 4, 8) == BITLINEAR_ERR_ALIGN && c.back(2, 8, 8, 4, 8, dX, dd, du) == BITLINEAR_ERR_ALIGN);
    c.wt = 1;
    CHECK(c.run(2, 8, 8, 4, 8) == BITLINEAR_OK && launched(0, "shrink expand "));
    CHECK(drop(at(0) + 1, 1, nullptr, 0, 64, 0.5, at(1), 0) == BITLINEAR_ERR_ALIGN);
    CHECK(drop(at(0), 0, at(2) + 2, 0, 64, 0.5, at(1), 0) == BITLINEAR_ERR_ALIGN);
    CHECK(drop(at(0), 0, nullptr, 0, 64, 0.5, at(1) + 3, 1) == BITLINEAR_ERR_ALIGN);
  }

  // overlaps: the first and the last byte of an array, and none one byte past it
  {
    Gated b;  // X: 5 * 100 * 4 bytes
    b.H = at(0) + 1996;
    CHECK(b.run(5, 100, 8) == BITLINEAR_ERR_ARG && b.block(5, 100, 8, 8) == BITLINEAR_ERR_ARG);
    b.H = at(0) - 5 * 8 * 4 + 4;
    CHECK(b.run(5, 100, 8) == BITLINEAR_ERR_ARG);
    b.H = at(0) + 2000;
    CHECK(b.run(5, 100, 8) == BITLINEAR_OK && launched(0, "gated_decode "));
    b = Gated();
    b.G = at(5) + 5 * 8 * 4 - 4, b.U = at(6);
    CHECK(b.run(5, 100, 8) == BITLINEAR_ERR_ARG && b.codes(5, 100, 8) == BITLINEAR_ERR_ARG);
    CHECK(g.block(5, 100, 8, 8, as<float>(6)) == BITLINEAR_ERR_ARG);  // hidden over the down codes
    b = Gated();
    b.H = at(2);
    CHECK(b.back(5, 8) == BITLINEAR_ERR_ARG);
    Low c;
    c.Y = reinterpret_cast<float*>(at(3) + 4 * 8 * 9 * 4 - 4);  // the last value of `up`
    CHECK(c.run(5, 100, 9, 4, 8) == BITLINEAR_ERR_ARG && c.whole(5, 100, 9, 4, 8) == BITLINEAR_ERR_ARG);
    CHECK(l.back(5, 100, 9, 4, 8, dX, dX + 499, du) == BITLINEAR_ERR_ARG);
    CHECK(l.back(5, 100, 9, 4, 8, as<float>(13), dd, du) == BITLINEAR_ERR_ARG);  // dX over dY
    CHECK(drop(at(0), 0, nullptr, 0, 64, 0.5, at(0) + 4, 0) == BITLINEAR_ERR_ARG);
    CHECK(drop(at(0), 0, nullptr, 0, 64, 0.5, at(0), 1) == BITLINEAR_ERR_ARG);  // another type
    CHECK(drop(at(0), 0, at(1) + 8, 0, 64, 0.5, at(1), 0) == BITLINEAR_ERR_ARG);
    CHECK(none());
    CHECK(drop(at(0), 0, at(0), 0, 64, 0.5, at(0), 0) == BITLINEAR_OK && launched(0, "dropout "));
    CHECK(drop(at(0), 0, at(1), 1, 64, 0.0, at(1), 1) == BITLINEAR_OK && launched(0, "dropout "));
    CHECK(drop(at(0), 0, nullptr, -1, (int64_t(1) << 40) - 1, 0.999999999999, at(1), 1) == BITLINEAR_OK &&
          launched(0, "dropout "));
  }

  // workspaces: one byte short, then enough
  auto exact = [](auto b, size_t need, auto call) {
    b.wsb = need - 1;
    CHECK(need > 0 && need % 256 == 0 && call(b) == BITLINEAR_ERR_WORKSPACE);
    b.wsb = need;
    CHECK(call(b) == BITLINEAR_OK);
    b.ws = nullptr;
    CHECK(call(b) == BITLINEAR_ERR_WORKSPACE);
  };
  exact(g, bitlinear_forward_workspace_bytes(20, 100), [](const Gated& b) { return b.run(20, 100, 8); });
  CHECK(launched(1, "gated_gemm "));
  for (int64_t F : {8, 900})  // the hidden layer's codes, or the input's
    exact(g, bitlinear_gated_ffn_workspace_bytes(20, 100, F, 8), [F](const Gated& b) { return b.block(20, 100, F, 8); });
  CHECK(launched(6, "gated_gemm gated_gemm "));
  exact(l, bitlinear_adapters_workspace_bytes(300, 100, 8, 9), [](const Low& b) { return b.run(300, 100, 8, 4, 9); });
  exact(l, bitlinear_adapted_workspace_bytes(300, 100, 8, 9), [](const Low& b) { return b.whole(300, 100, 8, 4, 9); });
  exact(l, bitlinear_adapters_backward_workspace_bytes(300, 100, 70, 4, 9),
        [=](const Low& b) { return b.back(300, 100, 70, 4, 9, dX, dd, du); });
  CHECK(launched(0, "shrink expand first join adapted_gemm shrink expand grad grad "));
  const size_t need = bitlinear_gated_input_backward_workspace_bytes(33, 70, 8, 1);
  CHECK(dx(33, 70, 8, 0, at(8), need - 1) == BITLINEAR_ERR_WORKSPACE);
  CHECK(dx(33, 70, 8, 0, at(8), need) == BITLINEAR_OK && launched(0, "dx_copies "));
  CHECK(dx(33, 72, 8, 0, nullptr, 0) == BITLINEAR_OK && launched(0, "dx "));
  CHECK(dx(33, 72, 8, 1, nullptr, 0) == BITLINEAR_ERR_WORKSPACE && none());
  const size_t sums = bitlinear_gated_input_backward_workspace_bytes(33, 1024, 8, 0);
  CHECK(sums > 0 && dx(33, 1024, 8, 0, at(8), sums - 1) == BITLINEAR_ERR_WORKSPACE && none());
  CHECK(dx(33, 1024, 8, 0, at(8), sums) == BITLINEAR_OK && launched(0, "dx "));

  // the product of few tiles in parts of K
  exact(g, bitlinear_gated_ffn_workspace_bytes(64, 100, 11008, 8), [](const Gated& b) { return b.block(64, 100, 11008, 8); });
  CHECK(launched(2, "gated_gemm parts "));
  exact(l, bitlinear_adapted_workspace_bytes(64, 11008, 8, 9), [](const Low& b) { return b.whole(64, 11008, 8, 4, 9); });
  CHECK(launched(0, "first parts expand "));
  for (int64_t M : {int64_t(1), int64_t(16), int64_t(17), int64_t(64), int64_t(777), int64_t(100000), M31, I64MAX / 2})
    for (int64_t N : {int64_t(1), int64_t(128), int64_t(4096), int64_t(70000), M31, I64MAX / 2})
      for (int64_t K : {int64_t(1), int64_t(128), int64_t(255), int64_t(4096), int64_t(11008), K20, I64MAX / 2}) {
        const int p = bitlinear::prefill_parts(M, N, K).parts;
        CHECK(p >= 1 && p <= 16 && (p == 1 || (M > 16 && 2 * p <= (K + 127) / 128)));
        CHECK(p == 1 || bitlinear::prefill_parts_bytes(M, N, K) >= size_t(4) * p * M * N);
      }

  // which launches: paths, sizes and what is asked for
  {
    Gated b;
    CHECK(b.run(16, 100, 8) == BITLINEAR_OK && launched(0, "gated_decode "));
    CHECK(b.codes(16, 100, 8) == BITLINEAR_OK && launched(0, "gated_decode "));
    CHECK(b.codes(17, 100, 8) == BITLINEAR_OK && launched(0, "gated_gemm "));
    CHECK(b.block(16, 100, 8, 8, as<float>(9)) == BITLINEAR_OK && launched(2, "gated_decode "));
    CHECK(b.back(5, 8) == BITLINEAR_OK && launched(0, "gated_backward "));
    b.path = BITLINEAR_PATH_PREFILL;
    CHECK(b.run(16, 100, 8) == BITLINEAR_OK && launched(1, "gated_gemm "));
    CHECK(b.block(16, 100, 8, 8) == BITLINEAR_OK && launched(3, "gated_gemm "));
    CHECK(b.run(M31, 511, 1) == BITLINEAR_OK && b.run(1, K20, 4095) == BITLINEAR_OK &&
          launched(2, "gated_gemm gated_gemm "));
    Low c;
    CHECK(c.whole(4, 100, 8, 4, 9) == BITLINEAR_OK && launched(1, "shrink expand "));  // no piece
    g_piece = 4;
    CHECK(c.whole(4, 100, 8, 4, 9) == BITLINEAR_OK && launched(0, "adapted_decode "));
    c.path = BITLINEAR_PATH_PREFILL;
    CHECK(c.whole(256, 100, 8, 4, 9) == BITLINEAR_OK && launched(0, "first join adapted_gemm "));
    CHECK(c.whole(255, 100, 8, 4, 9) == BITLINEAR_OK && launched(1, "first expand "));
    CHECK(c.whole(2048, 100, 2048, 4, 64) == BITLINEAR_OK && launched(0, "first join adapted_gemm "));
    CHECK(c.whole(2048, 100, 2048, 4, 65) == BITLINEAR_OK && launched(1, "first expand "));
    CHECK(c.whole(128, 100, 8, 4, 17) == BITLINEAR_OK && launched(1, "first expand "));
    CHECK(c.whole(128, 7, 8, 4, 9) == BITLINEAR_OK && launched(2, "shrink expand "));
    CHECK(c.whole(128, 8, 7, 4, 9) == BITLINEAR_OK && launched(1, "first expand "));
    g_piece = 0;
    CHECK(l.back(5, 100, 9, 4, 8, dX, nullptr, nullptr, 1) == BITLINEAR_OK && launched(0, "shrink expand "));
    CHECK(l.back(5, 100, 9, 4, 8, nullptr, dd, nullptr) == BITLINEAR_OK && launched(0, "shrink join grad "));
    CHECK(l.back(5, 100, 9, 4, 8, nullptr, nullptr, du) == BITLINEAR_OK && launched(0, "grad "));
  }

  // a launch that fails: an error, and none after it
  g_fail = true;
  CHECK(g.run(2, 8, 8) == BITLINEAR_ERR_HIP && g.codes(2, 8, 8) == BITLINEAR_ERR_HIP && g.back(2, 8) == BITLINEAR_ERR_HIP);
  CHECK(launched(0, "gated_decode gated_decode gated_backward "));
  CHECK(g.block(2, 8, 8, 8) == BITLINEAR_ERR_HIP && launched(0, "gated_decode "));
  CHECK(dx(2, 8, 8, 0, nullptr, 0) == BITLINEAR_ERR_HIP && launched(0, "dx "));
  CHECK(l.run(2, 8, 8, 4, 8) == BITLINEAR_ERR_HIP && launched(0, "shrink "));
  CHECK(l.whole(300, 8, 8, 4, 8) == BITLINEAR_ERR_HIP && launched(0, "first "));
  CHECK(l.back(2, 8, 8, 4, 8, dX, dd, du) == BITLINEAR_ERR_HIP && launched(0, "shrink "));
  CHECK(l.back(2, 8, 8, 4, 8, nullptr, nullptr, du) == BITLINEAR_ERR_HIP && launched(0, "grad "));
  CHECK(drop(at(0), 0, nullptr, 0, 64, 0.5, at(1), 0) == BITLINEAR_ERR_HIP && launched(0, "dropout "));
  g_fail = false;
  stub_reset(0);
  CHECK(g.run(20, 8, 8) == BITLINEAR_ERR_HIP && launched(1, ""));
  stub_reset(0);
  CHECK(g.block(2, 8, 8, 8) == BITLINEAR_ERR_HIP && launched(1, "gated_decode "));
  stub_reset(0);
  CHECK(l.whole(300, 8, 8, 4, 17) == BITLINEAR_ERR_HIP && launched(1, "first "));

  // size queries saturate to 0
  for (int64_t v : {int64_t(0), int64_t(-1), I64MAX, I64MIN, (int64_t(1) << 40) + 1}) {
    CHECK(bitlinear_gated_ffn_workspace_bytes(v, 8, 8, 8) == 0 && bitlinear_gated_ffn_workspace_bytes(8, v, 8, 8) == 0 &&
          bitlinear_gated_ffn_workspace_bytes(8, 8, v, 8) == 0 && bitlinear_gated_ffn_workspace_bytes(8, 8, 8, v) == 0);
    for (int copies : {0, 1})
      CHECK(bitlinear_gated_input_backward_workspace_bytes(v, 8, 8, copies) == 0 &&
            bitlinear_gated_input_backward_workspace_bytes(8, v, 8, copies) == 0 &&
            bitlinear_gated_input_backward_workspace_bytes(8, 8, v, copies) == 0);
    CHECK(bitlinear_adapters_workspace_bytes(v, 8, 8, 8) == 0 && bitlinear_adapters_workspace_bytes(8, v, 8, 8) == 0 &&
          bitlinear_adapters_workspace_bytes(8, 8, v, 8) == 0 && bitlinear_adapters_workspace_bytes(8, 8, 8, v) == 0);
    CHECK(bitlinear_adapted_workspace_bytes(v, 8, 8, 8) == 0 && bitlinear_adapted_workspace_bytes(8, v, 8, 8) == 0 &&
          bitlinear_adapted_workspace_bytes(8, 8, v, 8) == 0 && bitlinear_adapted_workspace_bytes(8, 8, 8, v) == 0);
    CHECK(bitlinear_adapters_backward_workspace_bytes(v, 8, 8, 4, 8) == 0 &&
          bitlinear_adapters_backward_workspace_bytes(8, v, 8, 4, 8) == 0 &&
          bitlinear_adapters_backward_workspace_bytes(8, 8, v, 4, 8) == 0 &&
          bitlinear_adapters_backward_workspace_bytes(8, 8, 8, v, 8) == 0 &&
          bitlinear_adapters_backward_workspace_bytes(8, 8, 8, 4, v) == 0);
  }
  const int64_t huge = int64_t(1) << 40;
  CHECK(bitlinear_gated_ffn_workspace_bytes(huge, huge, huge, huge) == 0);
  CHECK(bitlinear_gated_input_backward_workspace_bytes(huge, huge, huge, 1) == 0);
  for (int64_t M : {int64_t(1), int64_t(55), int64_t(64), int64_t(300), int64_t(5000)})
    for (int64_t D : {int64_t(1), int64_t(64), int64_t(238), int64_t(4096), int64_t(70000)})
      for (int64_t F : {int64_t(1), int64_t(64), int64_t(255), int64_t(256), int64_t(10688), K20}) {
        const bitlinear::GatedDxPlan p = bitlinear::gated_dx_plan(M, F, D);
        CHECK(p.parts >= 1 && p.parts <= 64 && (p.parts == 1 || int64_t(p.parts) * 256 <= bitlinear::padded_k(F)));
        CHECK(bitlinear_gated_input_backward_workspace_bytes(M, F, D, 0) >=
              (p.parts == 1 ? 0 : size_t(4) * p.parts * M * D));
      }
  CHECK(bitlinear_adapted_workspace_bytes(huge, huge, 8, 256) == 0);
  CHECK(bitlinear_adapters_backward_workspace_bytes(huge, huge, huge, 65535, 256) > size_t(huge) * 256 * 8);

  // every plan: at least one part, none empty of its smallest piece, sizes agree
  for (int64_t M : {int64_t(1), int64_t(2), int64_t(15), int64_t(17), int64_t(255), int64_t(256), int64_t(777),
                    int64_t(2048), int64_t(100000), M31})
    for (int64_t C = 1; C <= K20; C = C < 40 ? C + 1 : 2 * C + 7)
      for (int64_t R : {1, 16, 17, 64, 255, 256}) {
        const bitlinear::ShrinkPlan s = bitlinear::shrink_plan(M, C);
        CHECK(s.parts >= 1 && s.parts <= 16 && (s.parts == 1 || int64_t(s.parts) * 256 < C + 256) && s.spread >= 1 &&
              s.spread <= 16 && (s.blocks == 1 || s.blocks == 4));
        CHECK(bitlinear::shrink_ws_bytes(M, C, R) >= size_t(M) * bitlinear::padded_r(R) * (4 * s.parts + 6));
        for (int64_t A : {1, 5, 65535}) {
          const bitlinear::GradPlan p = bitlinear::grad_plan(M, C, A, R);
          CHECK(p.parts >= 1 && p.parts <= 16 && (p.parts == 1 || int64_t(p.parts) * 256 < M + 256) &&
                int64_t(p.tiles) * 64 >= C && p.groups * 64 >= R);
          CHECK(p.parts == 1 || bitlinear::grad_ws_bytes(M, C, A, R) >= size_t(p.parts) * 4 * A * R * C);
        }
      }
  printf("%d checks, %d failed\n", g_run, g_failed);
  return g_failed != 0;
}
