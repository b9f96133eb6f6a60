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

// Two binary32 values rounded to T (nearest, ties to even), packed.
__device__ __forceinline__ uint32_t pack2(float a, float b, const _Float16*) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)a) |
         (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)b) << 16;
}
__device__ __forceinline__ uint32_t pack2(float a, float b, const __bf16*) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)a) |
         (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)b) << 16;
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

// The lane's elements col .. col+kVec-1 of a row; those at or past cols read
// as 0.  Rows hold memory up to cols rounded up to 8 (the calls' contract),
// so the 16 bytes are readable whenever col < cols.
template <typename T>
__device__ __forceinline__ void load_row(const T* __restrict__ row, int col, int cols,
                                         float (&v)[kVec<T>]) {
  if (col + kVec<T> <= cols) {
    unpack(*reinterpret_cast<const lu4*>(row + col), v, (const T*)nullptr);
  } else if (col < cols) {
    unpack(*reinterpret_cast<const lu4*>(row + col), v, (const T*)nullptr);
    for (int j = 0; j < kVec<T>; ++j)
      if (col + j >= cols) v[j] = 0.0f;
  } else {
    for (int j = 0; j < kVec<T>; ++j) v[j] = 0.0f;
  }
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

// ---- kept activations ------------------------------------------------------
__device__ __forceinline__ uint32_t magnitude(float x) {
  return __builtin_bit_cast(uint32_t, x) & 0x7FFFFFFFu;
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

__device__ __forceinline__ uint32_t quant(float x, float inv) {
  // x * inv is exact (a power of two); a NaN (inf * 0) becomes 0
  const float r = __builtin_rintf(x * inv);
  const int i = (int)__builtin_fminf(__builtin_fmaxf(r, -127.0f), 127.0f);
  return (uint32_t)i & 0xFFu;
}
__device__ __forceinline__ uint32_t quant4(const float* v, float inv, bool finite) {
  const uint32_t u = quant(v[0], inv) | quant(v[1], inv) << 8 | quant(v[2], inv) << 16 |
                     quant(v[3], inv) << 24;
  return finite ? u : 0u;
}
__device__ __forceinline__ float dequant(uint32_t u, int j, float step) {
  return (float)(int8_t)(u >> (8 * j)) * step;
}

// ---- activation functions ----------------------------------------------------
constexpr int kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3;

constexpr float kSqrtHalf = 0.70710678118654752f, kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTanhA = 0.79788456080286536f, kTanhC = 0.044715f;  // sqrt(2/pi)

// 1 / (1 + exp(-2u)), the form of (1 + tanh u) / 2 that keeps its relative
// accuracy where it nears 0
__device__ __forceinline__ float sigmoid2(float u) {
  return 1.0f / (1.0f + __expf(-2.0f * u));
}

// GELU is x * Phi(x) with Phi from erfc, which keeps its relative accuracy in
// the tail where 1 + erf cancels.
__device__ __forceinline__ float act(float x, int kind) {
  switch (kind) {
    case kActRelu: return x < 0.0f ? 0.0f : x;  // NaN stays
    case kActGelu: return 0.5f * x * erfcf(-kSqrtHalf * x);
    case kActGeluTanh: return x * sigmoid2(kTanhA * (x + kTanhC * x * x * x));
    default: return x;
  }
}

__device__ __forceinline__ float act_grad(float x, int kind) {
  switch (kind) {
    case kActRelu: return x > 0.0f ? 1.0f : (x != x ? x : 0.0f);
    case kActGelu:
      return 0.5f * erfcf(-kSqrtHalf * x) + x * (kInvSqrt2Pi * __expf(-0.5f * x * x));
    case kActGeluTanh: {
      const float s = sigmoid2(kTanhA * (x + kTanhC * x * x * x));
      return s + x * s * (1.0f - s) * (2.0f * kTanhA) * (1.0f + 3.0f * kTanhC * x * x);
    }
    default: return 1.0f;
  }
}

}  // namespace
}  // namespace oba
