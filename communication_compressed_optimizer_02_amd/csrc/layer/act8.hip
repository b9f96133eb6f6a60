// act8.hip -- activations kept in 8 bits (gfx950): rows to integers with a
// power-of-two step per 32 columns, and back.  The format is described in
// layer.hpp and include/oba.h.  Both are bound by memory: 32768 x 4096 of
// bfloat16 (407 MB) encode in 88 us (4.6 TB/s) and decode in 68 us (6.0 TB/s,
// part of the integers still in cache); a large copy reaches 5.0 TB/s.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "layer.hpp"
#include "layer_kernels.hpp"

namespace oba {

namespace {

constexpr int kA8Block = 256;
constexpr int kA8Unroll = 4;  // pieces of 16 bytes per lane, all loaded before the first is used

// A matrix is walked as one list of pieces of 16 bytes, `per_row` to a row
// (whole groups, so the lanes of a group are neighbours in a wave).  A block
// takes kA8Block * kA8Unroll pieces in a row; its first piece's row comes
// from one uniform 64-bit division, a lane's from a binary32 reciprocal: the
// quotient is at most 1 off, and is put right.
struct Walk {
  int64_t row0;
  int32_t rem0, per_row;
  float inv;
};

__device__ __forceinline__ Walk walk(int64_t first, int32_t per_row) {
  Walk w;
  w.row0 = first / per_row;
  w.rem0 = (int32_t)(first - w.row0 * per_row);
  w.per_row = per_row;
  w.inv = 1.0f / (float)per_row;
  return w;
}

__device__ __forceinline__ void place(const Walk& w, int32_t i, int64_t& row, int32_t& piece) {
  const int32_t r = w.rem0 + i;  // below per_row + kA8Block * kA8Unroll, far below 2^24
  int32_t q = (int32_t)((float)r * w.inv);
  int32_t p = r - q * w.per_row;
  if (p < 0) {
    --q;
    p += w.per_row;
  } else if (p >= w.per_row) {
    ++q;
    p -= w.per_row;
  }
  row = w.row0 + q;
  piece = p;
}

template <typename T>
__global__ __launch_bounds__(kA8Block) void k_act8_encode(int64_t pieces, int32_t per_row,
                                                          int32_t cols,
                                                          const T* __restrict__ x, int64_t ldx,
                                                          uint8_t* __restrict__ q,
                                                          uint8_t* __restrict__ e) {
  constexpr int V = kVec<T>, L = kAct8Group / V;  // lanes of a group
  const int64_t first = (int64_t)blockIdx.x * (kA8Block * kA8Unroll);
  const Walk w = walk(first, per_row);
  float v[kA8Unroll][V];
  int64_t row[kA8Unroll];
  int32_t piece[kA8Unroll];
#pragma unroll
  for (int u = 0; u < kA8Unroll; ++u) {
    const int32_t i = u * kA8Block + threadIdx.x;
    place(w, i, row[u], piece[u]);
    if (first + i >= pieces) row[u] = -1;
    if (row[u] >= 0) load_row(x + row[u] * ldx, piece[u] * V, cols, v[u]);
    else
      for (int j = 0; j < V; ++j) v[u][j] = 0.0f;
  }
#pragma unroll
  for (int u = 0; u < kA8Unroll; ++u) {
    uint32_t top = 0;
    for (int j = 0; j < V; ++j) top = max(top, magnitude(v[u][j]));
    top = max_lanes<L>(top);
    const uint32_t ex = group_exp(top);
    const float inv = inv_step_of(ex), step = step_of(ex);
    if (row[u] < 0) continue;
    const int64_t at = (row[u] * per_row + piece[u]) * V;
    if constexpr (V == 8) {
      const lu2 o = {quant4(v[u], inv, step, ex != 255u), quant4(v[u] + 4, inv, step, ex != 255u)};
      *reinterpret_cast<lu2*>(q + at) = o;
    } else {
      *reinterpret_cast<uint32_t*>(q + at) = quant4(v[u], inv, step, ex != 255u);
    }
    if ((threadIdx.x & (L - 1)) == 0) e[at / kAct8Group] = (uint8_t)ex;
  }
}

template <typename T>
__global__ __launch_bounds__(kA8Block) void k_act8_decode(int64_t pieces, int32_t per_row,
                                                          int32_t cols,
                                                          const uint8_t* __restrict__ q,
                                                          const uint8_t* __restrict__ e,
                                                          T* __restrict__ x, int64_t ldx) {
  constexpr int V = kVec<T>;
  const int64_t first = (int64_t)blockIdx.x * (kA8Block * kA8Unroll);
  const Walk w = walk(first, per_row);
  lu2 b[kA8Unroll];
  uint32_t ex[kA8Unroll];
  int64_t row[kA8Unroll];
  int32_t piece[kA8Unroll];
#pragma unroll
  for (int u = 0; u < kA8Unroll; ++u) {
    const int32_t i = u * kA8Block + threadIdx.x;
    place(w, i, row[u], piece[u]);
    if (first + i >= pieces) row[u] = -1;
    if (row[u] < 0) continue;
    const int64_t at = (row[u] * per_row + piece[u]) * V;
    if constexpr (V == 8) b[u] = *reinterpret_cast<const lu2*>(q + at);
    else b[u][0] = *reinterpret_cast<const uint32_t*>(q + at);
    ex[u] = e[at / kAct8Group];
  }
#pragma unroll
  for (int u = 0; u < kA8Unroll; ++u) {
    if (row[u] < 0) continue;
    const float s = step_of(ex[u]);
    float v[V];
    for (int j = 0; j < V; ++j) v[j] = dequant(b[u][j / 4], j % 4, s);
    store_row(x + row[u] * ldx, piece[u] * V, cols, v);
  }
}

constexpr int64_t kPerBlock = kA8Block * kA8Unroll;

// Pieces of a row of vec elements: whole groups.
int32_t pieces_of(int64_t cols, int vec) {
  return (int32_t)((cols + kAct8Group - 1) / kAct8Group * (kAct8Group / vec));
}

template <typename T>
void encode(int64_t rows, int32_t cols, const void* x, int64_t ldx, int8_t* q, uint8_t* e,
            hipStream_t st) {
  const int32_t per_row = pieces_of(cols, kVec<T>);
  const int64_t pieces = rows * per_row;
  hipLaunchKernelGGL(HIP_KERNEL_NAME(k_act8_encode<T>),
                     dim3((uint32_t)((pieces + kPerBlock - 1) / kPerBlock)), dim3(kA8Block), 0, st,
                     pieces, per_row, cols, static_cast<const T*>(x), ldx,
                     reinterpret_cast<uint8_t*>(q), e);
}

template <typename T>
void decode(int64_t rows, int32_t cols, const int8_t* q, const uint8_t* e, void* x, int64_t ldx,
            hipStream_t st) {
  const int32_t per_row = pieces_of(cols, kVec<T>);
  const int64_t pieces = rows * per_row;
  hipLaunchKernelGGL(HIP_KERNEL_NAME(k_act8_decode<T>),
                     dim3((uint32_t)((pieces + kPerBlock - 1) / kPerBlock)), dim3(kA8Block), 0, st,
                     pieces, per_row, cols,
                     reinterpret_cast<const uint8_t*>(q), e, static_cast<T*>(x), ldx);
}

}  // namespace

int64_t act8_blocks(int64_t rows, int64_t cols, int dtype) {
  return (rows * pieces_of(cols, dtype == kGradF32 ? 4 : 8) + kPerBlock - 1) / kPerBlock;
}

void launch_act8_encode(int64_t rows, int32_t cols, const void* x, int64_t ldx, int dtype,
                        int8_t* q, uint8_t* e, hipStream_t st) {
  if (dtype == kGradF32) encode<float>(rows, cols, x, ldx, q, e, st);
  else if (dtype == kGradF16) encode<_Float16>(rows, cols, x, ldx, q, e, st);
  else encode<__bf16>(rows, cols, x, ldx, q, e, st);
}

void launch_act8_decode(int64_t rows, int32_t cols, const int8_t* q, const uint8_t* e, void* x,
                        int64_t ldx, int dtype, hipStream_t st) {
  if (dtype == kGradF32) decode<float>(rows, cols, q, e, x, ldx, st);
  else if (dtype == kGradF16) decode<_Float16>(rows, cols, q, e, x, ldx, st);
  else decode<__bf16>(rows, cols, q, e, x, ldx, st);
}

}  // namespace oba
