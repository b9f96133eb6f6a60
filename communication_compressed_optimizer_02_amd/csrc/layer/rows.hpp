// rows.hpp -- a layer norm's rows (norm.hip): how they lie over the lanes of one
// wave or of several, parameter vectors, whose pieces join.hip reads too (Four),
// and taking the mean off.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "layer.hpp"

namespace oba {

namespace {

// A lane's columns: chunk c holds kVec consecutive columns from
// (c * W * 64 + thread) * kVec, W the waves that share a row (a power of two; a
// block holds four rows of one wave or one row).
template <typename T, int W>
__device__ __forceinline__ int32_t chunk_col(int c) {
  const int32_t t = (int32_t)threadIdx.x & (W * 64 - 1);
  return (c * W * 64 + t) * kVec<T>;
}

// Columns from a binary32 vector of any alignment (parameters live anywhere
// in the flat x); those past cols read as 0.
struct __attribute__((packed, aligned(4))) Four {
  float v[4];
};
template <typename T, int NC, int W>
__device__ __forceinline__ void load_params(const float* __restrict__ p, int32_t cols,
                                            float (&v)[NC][kVec<T>]) {
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int32_t col = chunk_col<T, W>(c);
#pragma unroll
    for (int j = 0; j < kVec<T>; j += 4) {
      if (col + j + 4 <= cols) {
        const Four f = *reinterpret_cast<const Four*>(p + col + j);
        for (int i = 0; i < 4; ++i) v[c][j + i] = f.v[i];
      } else {
        for (int i = 0; i < 4; ++i) v[c][j + i] = col + j + i < cols ? p[col + j + i] : 0.0f;
      }
    }
  }
}

// v - m - off (m rounded to binary32 and what that left), 0 stays at and past
// cols: lanes that hold none of the row subtract 0, and elements are looked at
// one by one only where a row ends inside a lane.
template <int V>
__device__ __forceinline__ void centre(float (&v)[V], float m, float off, int32_t col,
                                       int32_t cols) {
  m = col < cols ? m : 0.0f;
  off = col < cols ? off : 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = (v[j] - m) - off;
  if (cols % V != 0) {  // the same for every lane
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = col + j < cols ? v[j] : 0.0f;
  }
}

}  // namespace
}  // namespace oba
