// Device helpers of the gated feed-forward block (include/bitlinear_gated.h).
#pragma once

#include "block_device.hpp"

namespace bitlinear {

constexpr int kActRelu2 = 0, kActSilu = 1;

// sigmoid(g) = 1 / (1 + exp(-g)), within a few float32 roundings.  exp(-g) is
// 2^t with t = -g log2(e) held in two float32 (a single one would be off by
// |g| 2^-24 of the result), on the hardware's exp2 and reciprocal: nine
// instructions, two of them quarter rate, where the library's expf and an IEEE
// division take about 40.  Beyond |t| = 126 the tail is left out: there the
// result is 1 or below 2^-126, and infinities must not meet the tail's zeros.
__device__ __forceinline__ float sigmoid(float g) {
  constexpr float kHi = -1.44269502162933349609375f;  // fp32(-log2(e))
  constexpr float kLo = -1.92596299112661746887e-8f;  // -log2(e) - kHi
  const float t = __fmul_rn(g, kHi);
  const float rest = __fmaf_rn(g, kLo, __fmaf_rn(g, kHi, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  // 2^(t + rest) = 2^t (1 + rest ln 2) (|rest| < 2^-16)
  const float whole = __fmaf_rn(e, __fmul_rn(rest, 0.693147182464599609375f), e);
  return __builtin_amdgcn_rcpf(__fadd_rn(1.0f, fabsf(t) <= 126.0f ? whole : e));
}

// act(g) * u: fp32(fp32(r * r) * u), r = max(g, 0), or g sigmoid(g) u
__device__ __forceinline__ float gated_value(int act, float g, float u) {
  float a;
  if (act == kActRelu2) {
    const float r = g <= 0.0f ? 0.0f : g;
    a = __fmul_rn(r, r);
  } else {
    a = __fmul_rn(g, sigmoid(g));
  }
  return __fmul_rn(a, u);
}

__device__ __forceinline__ void store_one(void* p, int dtype, int64_t at, float v) {
  if (dtype == kF32)
    static_cast<float*>(p)[at] = v;
  else
    static_cast<uint16_t*>(p)[at] = static_cast<uint16_t>(bf16_pair(v, v));
}

}  // namespace bitlinear
