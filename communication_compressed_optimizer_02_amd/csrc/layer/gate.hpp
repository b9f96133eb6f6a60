// gate.hpp -- the gate functions of a gated linear layer and their derivatives.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "layer.hpp"

namespace oba {

namespace {

// The first four are the activation functions' numbers.
constexpr int kGateSilu = 4, kGateSigmoid = 5;

// The logistic function s and 1 - s, each with its relative accuracy: from
// z = exp(-|p|) <= 1, 1 / (1 + z) and z / (1 + z), which change places with p's
// sign.  z is off by what rounds its exponent, |p| 2^-24 of it, and the
// hardware's exp2 and reciprocal by 2^-22 each: at |p| = 32 together 2^-18, far
// below half a step of the 16-bit results.  Below 2^-126 z is taken as 0.
__device__ __forceinline__ float logistic(float p, float& other) {
  const float z = exp2_hw(-kLog2E * __builtin_fabsf(p)), t = rcp_hw(1.0f + z), zt = z * t;
  other = p < 0.0f ? t : zt;
  return p < 0.0f ? zt : t;
}

// f(p) in place, eight values at a time: one branch on the kind.  Without 1 - s
// the logistic function is 1 / (1 + exp(-p)), as exact: where exp(-p) is large its
// error is the result's, and past 2^126 the result is 0.
__device__ __forceinline__ void gate_value(float (&v)[8], int kind) {
  if (kind == kGateSilu) {
    for (int j = 0; j < 8; ++j) v[j] *= rcp_hw(1.0f + exp2_hw(-kLog2E * v[j]));
  } else if (kind == kGateSigmoid) {
    for (int j = 0; j < 8; ++j) v[j] = rcp_hw(1.0f + exp2_hw(-kLog2E * v[j]));
  } else {
    activate(v, kind);
  }
}

// f(p) in place, and f'(p).
__device__ __forceinline__ void gate_both(float (&v)[8], float (&d)[8], int kind) {
  if (kind == kGateSilu) {
    for (int j = 0; j < 8; ++j) {
      float o;
      const float s = logistic(v[j], o);
      d[j] = s * __builtin_fmaf(v[j], o, 1.0f);
      v[j] *= s;
    }
  } else if (kind == kGateSigmoid) {
    for (int j = 0; j < 8; ++j) {
      float o;
      const float s = logistic(v[j], o);
      d[j] = s * o;
      v[j] = s;
    }
  } else if (kind == kActGelu) {
    for (int j = 0; j < 8; ++j) {
      float g;
      const float c = normal_cdf(v[j], g);
      d[j] = __builtin_fmaf(v[j] * kInvSqrt2Pi, g, c);
      v[j] *= c;
    }
  } else if (kind == kActNone) {
    for (int j = 0; j < 8; ++j) d[j] = 1.0f;
  } else {
    for (int j = 0; j < 8; ++j) d[j] = v[j];
    activate_grad(d, kind);
    activate(v, kind);
  }
}

}  // namespace
}  // namespace oba
