// layer.hpp -- device helpers shared by the layer operators (act8.hip,
// norm.hip, linear.hip): vectors of a row, the 8-bit format of kept
// activations, and the activation functions with their derivatives.
//
// Kept activations.  A group of 32 consecutive columns of a row whose largest
// magnitude is f * 2^k (1 <= f < 2) has the step 2^max(k-6, -126); an element
// is the integer x / step rounded to nearest even, held to +-127.  The scale
// is a power of two and not amax/127 because the value an integer stands for
// then has at most 7 significant bits: it is exact in bfloat16 (and, for rows
// that were binary16, in binary16), so the weight gradient's matrix
// instructions take it without a second rounding, and quantising is a shift
// of the exponent followed by one rounding.  The cost is up to one bit of the
// eight (half a bit on average).
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "kernels.hpp"

namespace oba {

namespace {

typedef float lf4 __attribute__((ext_vector_type(4)));
typedef uint32_t lu2 __attribute__((ext_vector_type(2)));
typedef uint32_t lu4 __attribute__((ext_vector_type(4)));

// Elements of a row that one lane holds: 16 bytes.
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

// Unpack 16 bytes of T to binary32 (exact).
__device__ __forceinline__ void unpack(const lu4 u, float (&v)[4], const float*) {
  for (int j = 0; j < 4; ++j) {
    const uint32_t w = u[j];  // (bit-casting the element itself takes the vector's first)
    v[j] = __builtin_bit_cast(float, w);
  }
}
__device__ __forceinline__ void unpack(const lu4 u, float (&v)[8], const _Float16*) {
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = (float)__builtin_bit_cast(_Float16, (uint16_t)(u[j] & 0xFFFFu));
    v[2 * j + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(u[j] >> 16));
  }
}
__device__ __forceinline__ void unpack(const lu4 u, float (&v)[8], const __bf16*) {
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __builtin_bit_cast(float, u[j] << 16);
    v[2 * j + 1] = __builtin_bit_cast(float, u[j] & 0xFFFF0000u);
  }
}

// Two binary32 values rounded to T (nearest, ties to even), packed by one
// instruction.
typedef float lf2 __attribute__((ext_vector_type(2)));
typedef _Float16 lh2 __attribute__((ext_vector_type(2)));
typedef __bf16 lb2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack2(float a, float b, const _Float16*) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(lf2{a, b}, lh2));
}
__device__ __forceinline__ uint32_t pack2(float a, float b, const __bf16*) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(lf2{a, b}, lb2));
}
__device__ __forceinline__ lu4 pack(const float (&v)[4], const float*) {
  lu4 u;
  for (int j = 0; j < 4; ++j) u[j] = __builtin_bit_cast(uint32_t, v[j]);
  return u;
}
template <typename T>
__device__ __forceinline__ lu4 pack(const float (&v)[8], const T* t) {
  lu4 u;
  for (int j = 0; j < 4; ++j) u[j] = pack2(v[2 * j], v[2 * j + 1], t);
  return u;
}

// The lane's 16 bytes of a row from column col.  Rows hold memory up to cols
// rounded up to 8 (the calls' contract), so they are readable whenever
// col < cols; what lies past cols is cut off when it is unpacked.
template <typename T>
__device__ __forceinline__ lu4 load_raw(const T* __restrict__ row, int col, int cols) {
  return col < cols ? *reinterpret_cast<const lu4*>(row + col) : lu4{0u, 0u, 0u, 0u};
}
template <typename T>
__device__ __forceinline__ void unpack_row(const lu4 u, int col, int cols, float (&v)[kVec<T>]) {
  unpack(u, v, (const T*)nullptr);
  if (col + kVec<T> > cols) {
    for (int j = 0; j < kVec<T>; ++j)
      if (col + j >= cols) v[j] = 0.0f;
  }
}

// The lane's elements col .. col+kVec-1 of a row; those at or past cols read
// as 0.
template <typename T>
__device__ __forceinline__ void load_row(const T* __restrict__ row, int col, int cols,
                                         float (&v)[kVec<T>]) {
  unpack_row<T>(load_raw(row, col, cols), col, cols, v);
}

// Writes the elements before cols and no others.
template <typename T>
__device__ __forceinline__ void store_row(T* __restrict__ row, int col, int cols,
                                          const float (&v)[kVec<T>]) {
  if (col + kVec<T> <= cols) {
    *reinterpret_cast<lu4*>(row + col) = pack(v, (const T*)nullptr);
  } else {
    for (int j = 0; j < kVec<T>; ++j)
      if (col + j < cols) row[col + j] = (T)v[j];
  }
}

// ---- across lanes, by data-parallel primitives: no trip through LDS ---------
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ float dppf(float v) {
  return __builtin_bit_cast(float, dpp<CTRL>(__builtin_bit_cast(uint32_t, v)));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

// The largest of L neighbouring lanes (L = 4 or 8), in all of them.
template <int L>
__device__ __forceinline__ uint32_t max_lanes(uint32_t v) {
  v = max(v, dpp<kXor1>(v));
  v = max(v, dpp<kXor2>(v));
  if constexpr (L == 8) v = max(v, dpp<kHalfMirror>(v));
  return v;
}

// The sum of a wave's 64 lanes, in all of them: rows of 16 by exchanges, the
// four rows' sums in order.
__device__ __forceinline__ float wave_sum(float v) {
  v += dppf<kXor1>(v);
  v += dppf<kXor2>(v);
  v += dppf<kHalfMirror>(v);
  v += dppf<kMirror>(v);
  const int b = __builtin_bit_cast(int, v);
  float s = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 0));
  s += __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 16));
  s += __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 32));
  s += __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 48));
  return s;
}

template <int CTRL>
__device__ __forceinline__ double dppd(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)dpp<CTRL>((uint32_t)(u >> 32)) << 32 |
                                        dpp<CTRL>((uint32_t)u));
}
__device__ __forceinline__ double lane_of(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum(double v) {
  v += dppd<kXor1>(v);
  v += dppd<kXor2>(v);
  v += dppd<kHalfMirror>(v);
  v += dppd<kMirror>(v);
  return lane_of(v, 0) + lane_of(v, 16) + lane_of(v, 32) + lane_of(v, 48);
}

// ---- kept activations ------------------------------------------------------
__device__ __forceinline__ uint32_t magnitude(float x) {
  return __builtin_bit_cast(uint32_t, x) & 0x7FFFFFFFu;
}

// The largest magnitude bits of eight values.  As signed integers the largest
// is the largest positive value, as unsigned ones the most negative value if
// there is one: two three-way maxima for two values, and no masking of signs.
__device__ __forceinline__ uint32_t magnitude8(const float (&v)[8]) {
  int32_t p = 0;
  uint32_t m = 0;
  for (int j = 0; j < 8; ++j) {
    p = max(p, __builtin_bit_cast(int32_t, v[j]));
    m = max(m, __builtin_bit_cast(uint32_t, v[j]));
  }
  return max((uint32_t)p, m > 0x80000000u ? m & 0x7FFFFFFFu : 0u);
}

// The exponent byte of a group with largest magnitude bits `top`: the step is
// 2^(byte-127); 255 for a group that holds an infinity or a NaN.
__device__ __forceinline__ uint32_t group_exp(uint32_t top) {
  const int b = (int)(top >> 23) - 6;
  return top >= 0x7F800000u ? 255u : (uint32_t)(b < 1 ? 1 : b);
}

__device__ __forceinline__ float step_of(uint32_t e) {
  return __builtin_bit_cast(float, e << 23);  // 255: infinity, so that 0 * step is NaN
}
// 1 / step; 0 for the byte 255, whose integers are all 0
__device__ __forceinline__ float inv_step_of(uint32_t e) {
  return e == 255u ? 0.0f : __builtin_bit_cast(float, (254u - e) << 23);
}

// Four integers, packed.  The values are held to 127 steps before they are
// scaled (exactly) and rounded: adding 1.5 * 2^23 rounds to an integer, ties
// to even, whose two's complement byte is the sum's last.
__device__ __forceinline__ uint32_t quant4(const float* v, float inv, float step, bool finite) {
  constexpr float kRound = 12582912.0f;
  uint32_t u[4];
  for (int j = 0; j < 4; ++j) {
    const float x = __builtin_amdgcn_fmed3f(v[j], -127.0f * step, 127.0f * step);
    u[j] = __builtin_bit_cast(uint32_t, __builtin_fmaf(x, inv, kRound));
  }
  const uint32_t lo = __builtin_amdgcn_perm(u[1], u[0], 0x0c0c0400u);
  const uint32_t hi = __builtin_amdgcn_perm(u[3], u[2], 0x04000c0cu);
  return finite ? lo | hi : 0u;
}
__device__ __forceinline__ float dequant(uint32_t u, int j, float step) {
  return (float)(int8_t)(u >> (8 * j)) * step;
}

// ---- activation functions ----------------------------------------------------
constexpr int kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3;

// The results go to 16 bits (half a step: 2^-8 of the value in bfloat16, 2^-11
// in binary16), so the functions are evaluated with the hardware's exp2 and
// reciprocal.  Their error grows with the exponent, whose argument is rounded
// in binary32: Phi is within (32 + 1.5 x^2) 2^-24 of its value, 2^-19 near 0
// and 2^-17 at x = -8 (observed 2^-18); the tanh form's factor within
// (8 + 16 |u|) 2^-24 for u < 0, 2^-15 at u = -24 (x = -8; observed 2^-17).  The
// epilogue of a product computes one per result: erfcf and a correctly rounded
// division made GELU 94 of 241 us at 16384 x 1024 -> 4096, these make it 20 of
// 167.
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_hw(float x) { return __builtin_amdgcn_rcpf(x); }

constexpr float kLog2E = 1.4426950408889634f, kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTanhA = 0.79788456080286536f, kTanhC = 0.044715f;  // sqrt(2/pi)

// (1 + tanh u) / 2 = 1 / (1 + exp(-2u)), which keeps its relative accuracy
// where it nears 0
__device__ __forceinline__ float sigmoid2(float u) {
  return rcp_hw(1.0f + exp2_hw(-2.0f * kLog2E * u));
}

// The normal distribution function Phi and exp(-x^2/2).  For z = |x|,
// Phi(-z) = exp(-z^2/2) R(z) keeps its relative accuracy in the tail; R, the
// Mills ratio over sqrt(2 pi), is a polynomial in t = 1 / (1 + 0.36 z) without
// a constant term (the form of Hastings' approximations), its coefficients
// fitted by iteratively reweighted least squares to 9e-7 of R on 0 <= z <= 14.
__device__ __forceinline__ float normal_cdf(float x, float& gauss) {
  const float t = rcp_hw(__builtin_fmaf(0.36f, __builtin_fabsf(x), 1.0f));
  float r = 0.04705954f;
  r = __builtin_fmaf(r, t, -0.17977609f);
  r = __builtin_fmaf(r, t, 0.18096979f);
  r = __builtin_fmaf(r, t, 0.02653834f);
  r = __builtin_fmaf(r, t, 0.13972329f);
  r = __builtin_fmaf(r, t, 0.14177172f);
  r = __builtin_fmaf(r, t, 0.1437131f);
  gauss = exp2_hw((-0.5f * kLog2E) * x * x);
  const float tail = gauss * (r * t);
  return x < 0.0f ? tail : 1.0f - tail;
}

// Eight values at a time: one branch on the kind.
__device__ __forceinline__ void activate(float (&v)[8], int kind) {
  if (kind == kActGelu) {
    float g;
    for (int j = 0; j < 8; ++j) v[j] *= normal_cdf(v[j], g);
  } else if (kind == kActGeluTanh) {
    for (int j = 0; j < 8; ++j)
      v[j] *= sigmoid2(kTanhA * __builtin_fmaf(kTanhC * v[j], v[j] * v[j], v[j]));
  } else if (kind == kActRelu) {
    for (int j = 0; j < 8; ++j) v[j] = v[j] < 0.0f ? 0.0f : v[j];  // NaN stays
  }
}

// The derivatives, in place of their arguments.
__device__ __forceinline__ void activate_grad(float (&v)[8], int kind) {
  if (kind == kActGelu) {
    for (int j = 0; j < 8; ++j) {
      float g;
      const float c = normal_cdf(v[j], g);
      v[j] = __builtin_fmaf(v[j] * kInvSqrt2Pi, g, c);
    }
  } else if (kind == kActGeluTanh) {
    for (int j = 0; j < 8; ++j) {
      const float x = v[j], xx = x * x, s = sigmoid2(kTanhA * __builtin_fmaf(kTanhC * x, xx, x));
      // x s (1 - s) is 0 long before xx passes 2^100: d stays finite, so that
      // their product is 0 there and not 0 * infinity
      const float d = __builtin_fmaf(6.0f * kTanhA * kTanhC, __builtin_fminf(xx, 0x1p100f),
                                     2.0f * kTanhA);
      v[j] = __builtin_fmaf(x * s * (1.0f - s), d, s);
    }
  } else if (kind == kActRelu) {
    for (int j = 0; j < 8; ++j) v[j] = v[j] > 0.0f ? 1.0f : (v[j] != v[j] ? v[j] : 0.0f);
  }
}

}  // namespace
}  // namespace oba
