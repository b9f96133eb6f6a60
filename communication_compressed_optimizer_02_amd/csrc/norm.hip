// norm.hip -- layer norm of rows, forward and backward (gfx950).
//
// Forward, per row: mean, rstd = 1/sqrt(var + eta) with the variance summed
// from the centred values (two passes over registers, one over memory), then
// y = xhat * gamma + beta and, if wanted, xhat kept in 8 bits.  Backward, per
// row, with a = dy * gamma:
//   dx = rstd * (a - mean(a) - xhat * mean(a * xhat)) + add
// and, per worker and column, dgamma = sum dy * xhat, dbeta = sum dy.
// Everything is bound by the rows' bytes: a row is read once into registers.
//
// A row belongs to one wave up to 2048 columns, to a block of 4 waves up to
// 8192 and of 8 waves up to 16384.  A wave walks many rows, so that gamma
// and beta are read once and, in the backward pass, the column sums stay in
// binary32 registers until the wave's last row; blocks write them as partial
// sums, which a second kernel adds per column in binary64 in a fixed order.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "layer.hpp"
#include "layer_kernels.hpp"

namespace oba {

namespace {

// A lane's columns: chunk c holds kVec consecutive columns from
// (c * W * 64 + thread) * kVec, W the waves that share a row.
template <typename T, int W>
__device__ __forceinline__ int32_t chunk_col(int c) {
  const int32_t t = W == 1 ? (int32_t)(threadIdx.x & 63) : (int32_t)threadIdx.x;
  return (c * W * 64 + t) * kVec<T>;
}

__device__ __forceinline__ float wave_sum32(float v) {
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

// Sums of two values over the waves of a row; every lane gets them.  `lds`
// holds 2 * W floats; the sums of the waves are added in wave order.
template <int W>
__device__ __forceinline__ void row_sum2(float& a, float& b, float* lds) {
  a = wave_sum32(a);
  b = wave_sum32(b);
  if constexpr (W > 1) {
    __syncthreads();  // the last sums have been read by all
    if ((threadIdx.x & 63) == 0) {
      lds[threadIdx.x >> 6] = a;
      lds[W + (threadIdx.x >> 6)] = b;
    }
    __syncthreads();
    a = b = 0.0f;
    for (int w = 0; w < W; ++w) {
      a += lds[w];
      b += lds[W + w];
    }
  }
}

// Columns from a binary32 vector of any alignment (parameters live anywhere
// in the flat x); those past cols read as 0.
template <typename T, int NC, int W>
__device__ __forceinline__ void load_params(const float* __restrict__ p, int32_t cols,
                                            float (&v)[NC][kVec<T>]) {
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int32_t col = chunk_col<T, W>(c);
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j) v[c][j] = col + j < cols ? p[col + j] : 0.0f;
  }
}

template <typename T, int NC, int W, bool KEEP>
__global__ __launch_bounds__(W == 1 ? 256 : W * 64) void k_norm_fwd(
    int64_t rows, int32_t cols, const T* __restrict__ x, int64_t ldx,
    const float* __restrict__ gamma, const float* __restrict__ beta, float eta,
    T* __restrict__ y, int64_t ldy, float* __restrict__ mean, float* __restrict__ rstd,
    uint8_t* __restrict__ q, uint8_t* __restrict__ e) {
  constexpr int V = kVec<T>, R = W == 1 ? 4 : 1;  // rows a block works on at a time
  __shared__ float lds[2 * W];
  const int32_t groups = (cols + kAct8Group - 1) / kAct8Group;
  float ga[NC][V], be[NC][V];
  load_params<T, NC, W>(gamma, cols, ga);
  load_params<T, NC, W>(beta, cols, be);
  const float n = (float)cols;
  for (int64_t r = (int64_t)blockIdx.x * R + (W == 1 ? threadIdx.x >> 6 : 0); r < rows;
       r += (int64_t)gridDim.x * R) {
    float v[NC][V];
    float s = 0.0f, z = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      load_row(x + r * ldx, chunk_col<T, W>(c), cols, v[c]);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < V; ++j) s += v[c][j];
    row_sum2<W>(s, z, lds);
    const float mu = s / n;
    float s2 = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int32_t col = chunk_col<T, W>(c);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        v[c][j] = col + j < cols ? v[c][j] - mu : 0.0f;
        s2 += v[c][j] * v[c][j];
      }
    }
    row_sum2<W>(s2, z, lds);
    const float rs = 1.0f / __builtin_sqrtf(s2 / n + eta);
    if ((W == 1 ? threadIdx.x & 63 : threadIdx.x) == 0) {
      mean[r] = mu;
      rstd[r] = rs;
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int32_t col = chunk_col<T, W>(c);
      float o[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        v[c][j] *= rs;
        o[j] = v[c][j] * ga[c][j] + be[c][j];
      }
      if (col < cols) store_row(y + r * ldy, col, cols, o);
      if constexpr (KEEP) {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) top = max(top, magnitude(v[c][j]));
#pragma unroll
        for (int m = 1; m < kAct8Group / V; m <<= 1)
          top = max(top, (uint32_t)__shfl_xor((int)top, m));
        const uint32_t ex = group_exp(top);
        const float inv = inv_step_of(ex);
        if (col < groups * kAct8Group) {  // a started group is written whole
          uint8_t* at = q + r * (int64_t)groups * kAct8Group + col;
          if constexpr (V == 8)
            *reinterpret_cast<lu2*>(at) =
                lu2{quant4(v[c], inv, ex != 255u), quant4(v[c] + 4, inv, ex != 255u)};
          else
            *reinterpret_cast<uint32_t*>(at) = quant4(v[c], inv, ex != 255u);
          if (col % kAct8Group == 0) e[r * groups + col / kAct8Group] = (uint8_t)ex;
        }
      }
    }
  }
}

// ---- backward ------------------------------------------------------------------
template <typename T, int NC, int W, bool KEPT>
__global__ __launch_bounds__(W == 1 ? 256 : W * 64) void k_norm_bwd(NormBwd a) {
  constexpr int V = kVec<T>, R = W == 1 ? 4 : 1;
  __shared__ float lds[2 * W];
  const int32_t cols = a.cols, groups = (cols + kAct8Group - 1) / kAct8Group;
  const int32_t worker = blockIdx.y;
  const int64_t base = (int64_t)worker * a.rows;
  float ga[NC][V], dg[NC][V], db[NC][V];
  load_params<T, NC, W>(a.gamma, cols, ga);
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < V; ++j) dg[c][j] = db[c][j] = 0.0f;
  const float n = (float)cols;
  for (int64_t i = (int64_t)blockIdx.x * R + (W == 1 ? threadIdx.x >> 6 : 0); i < a.rows;
       i += (int64_t)gridDim.x * R) {
    const int64_t r = base + i;
    float h[NC][V], d[NC][V];
    const float rs = a.rstd[r];
#pragma unroll
    for (int c = 0; c < NC; ++c)
      load_row(static_cast<const T*>(a.dy) + r * a.lddy, chunk_col<T, W>(c), cols, d[c]);
    if constexpr (KEPT) {
      const uint8_t* qr = reinterpret_cast<const uint8_t*>(a.q) + r * (int64_t)groups * kAct8Group;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int32_t col = chunk_col<T, W>(c);
        lu2 u = {0u, 0u};
        float step = 0.0f;
        if (col < cols) {
          if constexpr (V == 8) u = *reinterpret_cast<const lu2*>(qr + col);
          else u[0] = *reinterpret_cast<const uint32_t*>(qr + col);
          step = step_of(a.e[r * groups + col / kAct8Group]);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) h[c][j] = dequant(u[j / 4], j % 4, step);
      }
    } else {
      const float mu = a.mean[r];
#pragma unroll
      for (int c = 0; c < NC; ++c)
        load_row(static_cast<const T*>(a.x) + r * a.ldx, chunk_col<T, W>(c), cols, h[c]);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int32_t col = chunk_col<T, W>(c);
#pragma unroll
        for (int j = 0; j < V; ++j) h[c][j] = col + j < cols ? (h[c][j] - mu) * rs : 0.0f;
      }
    }
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float t = d[c][j] * ga[c][j];
        dg[c][j] += d[c][j] * h[c][j];
        db[c][j] += d[c][j];
        s1 += t;
        s2 += t * h[c][j];
        d[c][j] = t;
      }
    row_sum2<W>(s1, s2, lds);
    const float m1 = s1 / n, m2 = s2 / n;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int32_t col = chunk_col<T, W>(c);
      float o[V];
      if (a.add) load_row(static_cast<const T*>(a.add) + r * a.ldadd, col, cols, o);
      else
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] += rs * (d[c][j] - m1 - h[c][j] * m2);
      if (col < cols) store_row(static_cast<T*>(a.dx) + r * a.lddx, col, cols, o);
    }
  }
  // the block's column sums: the waves of a block add theirs in wave order
  float* part = a.part + ((int64_t)worker * gridDim.x + blockIdx.x) * 2 * cols;
  if constexpr (W == 1) {
    __shared__ float sums[2][NC * 64 * V];
    for (int w = 0; w < R; ++w) {
      if ((int)(threadIdx.x >> 6) == w) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const int32_t at = chunk_col<T, W>(c) + j;
            sums[0][at] = (w ? sums[0][at] : 0.0f) + dg[c][j];
            sums[1][at] = (w ? sums[1][at] : 0.0f) + db[c][j];
          }
      }
      __syncthreads();
    }
    for (int32_t col = threadIdx.x; col < cols; col += 256) {
      part[col] = sums[0][col];
      part[cols + col] = sums[1][col];
    }
  } else {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int32_t col = chunk_col<T, W>(c) + j;
        if (col < cols) {
          part[col] = dg[c][j];
          part[cols + col] = db[c][j];
        }
      }
  }
}

// Column sums of a worker from its blocks' partial sums, in binary64: 64
// columns to a block, 4 waves that each add every fourth partial, joined in
// wave order.
template <typename G>
__global__ __launch_bounds__(256) void k_norm_wgrad(const float* __restrict__ part,
                                                    int32_t blocks, int32_t cols,
                                                    G* __restrict__ dgamma,
                                                    G* __restrict__ dbeta, int64_t ldg) {
  __shared__ double lds[4][64];
  const int32_t col = blockIdx.x * 64 + (threadIdx.x & 63), w = threadIdx.x >> 6;
  const float* p = part + (int64_t)blockIdx.y * blocks * 2 * cols;
  double s = 0.0;
  if (col < 2 * cols)
    for (int32_t b = w; b < blocks; b += 4) s += p[(int64_t)b * 2 * cols + col];
  lds[w][threadIdx.x & 63] = s;
  __syncthreads();
  if (w == 0 && col < 2 * cols) {
    const int l = threadIdx.x;
    const float t = (float)(((lds[0][l] + lds[1][l]) + lds[2][l]) + lds[3][l]);
    if (col < cols) dgamma[(int64_t)blockIdx.y * ldg + col] = (G)t;
    else dbeta[(int64_t)blockIdx.y * ldg + col - cols] = (G)t;
  }
}

// ---- launchers -------------------------------------------------------------------
template <typename T, int NC, int W>
void fwd_keep(const NormFwd& a, hipStream_t st) {
  constexpr int R = W == 1 ? 4 : 1;
  const int64_t want = (a.rows + R - 1) / R;
  const uint32_t grid = (uint32_t)std::min<int64_t>(want, W == 1 ? 2048 : W == 4 ? 2048 : 512);
  const dim3 block(W == 1 ? 256 : W * 64);
  auto* q = reinterpret_cast<uint8_t*>(a.q);
  if (a.q)
    hipLaunchKernelGGL(HIP_KERNEL_NAME(k_norm_fwd<T, NC, W, true>), dim3(grid), block, 0, st,
                       a.rows, a.cols, static_cast<const T*>(a.x), a.ldx, a.gamma, a.beta, a.eta,
                       static_cast<T*>(a.y), a.ldy, a.mean, a.rstd, q, a.e);
  else
    hipLaunchKernelGGL(HIP_KERNEL_NAME(k_norm_fwd<T, NC, W, false>), dim3(grid), block, 0, st,
                       a.rows, a.cols, static_cast<const T*>(a.x), a.ldx, a.gamma, a.beta, a.eta,
                       static_cast<T*>(a.y), a.ldy, a.mean, a.rstd, q, a.e);
}

// The smallest instance that holds a row; M = 1 for 16-byte pieces of eight
// elements, 2 for binary32's four.
template <typename T>
void fwd(const NormFwd& a, hipStream_t st) {
  constexpr int M = 8 / kVec<T>;
  if (a.cols <= 512) fwd_keep<T, M, 1>(a, st);
  else if (a.cols <= 1024) fwd_keep<T, 2 * M, 1>(a, st);
  else if (a.cols <= 2048) fwd_keep<T, 4 * M, 1>(a, st);
  else if (a.cols <= 4096) fwd_keep<T, 2 * M, 4>(a, st);
  else if (a.cols <= 8192) fwd_keep<T, 4 * M, 4>(a, st);
  else fwd_keep<T, 4 * M, 8>(a, st);
}

template <typename T, int NC, int W>
void bwd_kept(const NormBwd& a, hipStream_t st) {
  const dim3 grid(norm_bwd_blocks(a.n, a.rows, a.cols), a.n), block(W == 1 ? 256 : W * 64);
  if (a.q) hipLaunchKernelGGL(HIP_KERNEL_NAME(k_norm_bwd<T, NC, W, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL(HIP_KERNEL_NAME(k_norm_bwd<T, NC, W, false>), grid, block, 0, st, a);
}

template <typename T>
void bwd(const NormBwd& a, hipStream_t st) {
  constexpr int M = 8 / kVec<T>;
  if (a.cols <= 512) bwd_kept<T, M, 1>(a, st);
  else if (a.cols <= 1024) bwd_kept<T, 2 * M, 1>(a, st);
  else if (a.cols <= 2048) bwd_kept<T, 4 * M, 1>(a, st);
  else if (a.cols <= 4096) bwd_kept<T, 2 * M, 4>(a, st);
  else if (a.cols <= 8192) bwd_kept<T, 4 * M, 4>(a, st);
  else bwd_kept<T, 4 * M, 8>(a, st);
}

template <typename G>
void wgrad(const NormBwd& a, hipStream_t st) {
  hipLaunchKernelGGL(HIP_KERNEL_NAME(k_norm_wgrad<G>), dim3((2 * a.cols + 63) / 64, a.n),
                     dim3(256), 0, st, a.part, a.rows ? norm_bwd_blocks(a.n, a.rows, a.cols) : 0,
                     a.cols, static_cast<G*>(a.dgamma), static_cast<G*>(a.dbeta), a.ldg);
}

}  // namespace

// About four blocks to a CU over all workers, and no more than a worker has
// rows for.
int32_t norm_bwd_blocks(int32_t n, int64_t rows, int32_t cols) {
  const int64_t per = cols <= 2048 ? 4 : 1;
  const int64_t most = std::max<int64_t>(1, (cols <= 8192 ? 1024 : 512) / n);
  return (int32_t)std::max<int64_t>(1, std::min<int64_t>((rows + per - 1) / per, most));
}

void launch_layer_norm(const NormFwd& a, hipStream_t st) {
  if (a.dtype == kGradF32) fwd<float>(a, st);
  else if (a.dtype == kGradF16) fwd<_Float16>(a, st);
  else fwd<__bf16>(a, st);
}

void launch_layer_norm_backward(const NormBwd& a, hipStream_t st) {
  if (a.dtype == kGradF32) bwd<float>(a, st);
  else if (a.dtype == kGradF16) bwd<_Float16>(a, st);
  else bwd<__bf16>(a, st);
}

void launch_layer_norm_weight_grad(const NormBwd& a, hipStream_t st) {
  if (a.g_dtype == kGradF32) wgrad<float>(a, st);
  else if (a.g_dtype == kGradF16) wgrad<_Float16>(a, st);
  else wgrad<__bf16>(a, st);
}

}  // namespace oba
