// dropout.hip -- dropout from a counter-based generator (gfx950):
//   y = (kept ? x * scale : 0) + add
// The bits of an element are a function of its place, the seed, the step and
// the site (philox.hpp), so nothing is stored and the backward pass is the same
// call on dy.  Bound by the memory, the generator's ten rounds for eight columns run
// under it: 32768 x 4096 bfloat16 98 us, 5.4 TB/s; 4099 x 1609 binary32 with add 15.3
// us, 5.2 TB/s.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "layer.hpp"
#include "philox.hpp"
#include "sublayer_kernels.hpp"

namespace oba {

namespace {

constexpr int kDropBlock = 256;
constexpr int kDropUnroll = 4;  // pieces of 16 bytes per lane, all loaded before the first is used
constexpr int64_t kDropPerBlock = kDropBlock * kDropUnroll;

// The matrix is one list of pieces of 16 bytes, whole blocks of eight columns
// to a row; a block of threads takes kDropPerBlock in a row.
template <typename T>
__global__ __launch_bounds__(kDropBlock) void k_dropout(int64_t pieces, int32_t per_row,
                                                        int32_t cols, const T* __restrict__ x,
                                                        int64_t ldx, Dropout d,
                                                        const T* __restrict__ add, int64_t ldadd,
                                                        T* __restrict__ y, int64_t ldy) {
  constexpr int V = kVec<T>;
  const int64_t first = (int64_t)blockIdx.x * kDropPerBlock;
  const RngKey key = load_key(d);
  lu4 xr[kDropUnroll], ar[kDropUnroll];
  int64_t row[kDropUnroll];
  int32_t col[kDropUnroll];
#pragma unroll
  for (int u = 0; u < kDropUnroll; ++u) {
    const int64_t i = first + u * kDropBlock + threadIdx.x;
    row[u] = i / per_row;
    col[u] = (int32_t)(i - row[u] * per_row) * V;
    if (i >= pieces) col[u] = cols;  // none of a row
    if (col[u] >= cols) continue;
    xr[u] = load_raw(x + row[u] * ldx, col[u], cols);
    if (add) ar[u] = load_raw(add + row[u] * ldadd, col[u], cols);
  }
#pragma unroll
  for (int u = 0; u < kDropUnroll; ++u) {
    if (col[u] >= cols) continue;
    float v[V];
    unpack(xr[u], v, (const T*)nullptr);
    if (d.threshold) drop<V>(d, key, row[u], (cols + 7) / 8, col[u], v);
    if (add) {
      float w[V];
      unpack(ar[u], w, (const T*)nullptr);
      for (int j = 0; j < V; ++j) v[j] += w[j];
    }
    store_row(y + row[u] * ldy, col[u], cols, v);
  }
}

int32_t per_row_of(int64_t cols, int vec) { return (int32_t)((cols + 7) / 8 * (8 / vec)); }

template <typename T>
void run(int64_t rows, int32_t cols, const void* x, int64_t ldx, const Dropout& d, const void* add,
         int64_t ldadd, void* y, int64_t ldy, hipStream_t st) {
  const int32_t per_row = per_row_of(cols, kVec<T>);
  const int64_t pieces = rows * per_row;
  hipLaunchKernelGGL(HIP_KERNEL_NAME(k_dropout<T>),
                     dim3((uint32_t)((pieces + kDropPerBlock - 1) / kDropPerBlock)),
                     dim3(kDropBlock), 0, st, pieces, per_row, cols, static_cast<const T*>(x), ldx,
                     d, static_cast<const T*>(add), ldadd, static_cast<T*>(y), ldy);
}

}  // namespace

int64_t dropout_blocks(int64_t rows, int64_t cols, int dtype) {
  return (rows * per_row_of(cols, dtype == kGradF32 ? 4 : 8) + kDropPerBlock - 1) / kDropPerBlock;
}

void launch_dropout(int64_t rows, int32_t cols, const void* x, int64_t ldx, int dtype,
                    const Dropout& d, const void* add, int64_t ldadd, void* y, int64_t ldy,
                    hipStream_t st) {
  if (dtype == kGradF32) run<float>(rows, cols, x, ldx, d, add, ldadd, y, ldy, st);
  else if (dtype == kGradF16) run<_Float16>(rows, cols, x, ldx, d, add, ldadd, y, ldy, st);
  else run<__bf16>(rows, cols, x, ldx, d, add, ldadd, y, ldy, st);
}

}  // namespace oba
