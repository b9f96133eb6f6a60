// norm.hip -- layer norm of rows, forward and backward (gfx950).
//
// Forward, per row: mean (a binary64 sum), rstd = 1/sqrt(var + eta) with the
// variance summed from the centred values (two passes over registers, one over
// memory), then
// y = xhat * gamma + beta and, if wanted, xhat kept in 8 bits.  Backward, per
// row, with a = dy * gamma:
//   dx = rstd * (a - mean(a) - xhat * mean(a * xhat)) + add
// and, per worker and column, dgamma = sum dy * xhat, dbeta = sum dy.
// A row is read once into registers.
//
// A row belongs to one wave up to 1024 columns, to a block of 4 waves up to
// 4096 and of 8 waves up to 16384.  A wave walks many rows, so that gamma
// and beta are read once and, in the backward pass, the column sums stay in
// binary32 registers until the wave's last row; blocks write them as partial
// sums, which a second kernel adds per column in binary64 in a fixed order.
// 32768 x 1024 in bfloat16: forward with xhat kept 32 us (169 MB, 5.3 TB/s),
// backward from 8 bits with add 50 us (236 MB, 4.7 TB/s) and 4.8 us for the
// columns' join; a large copy reaches 5.0 TB/s.
//
// What bounds it goes by the width.  2^25 elements in us, calls one after
// another, forward bare, forward kept, backward from the rows and from 8 bits
// (join included; the bytes at 4.96 TB/s take 27, 34, 41 and 34 in bfloat16, 54,
// 61, 81 and 61 in binary32):
//   columns      64   128   512  1024  2048  4096  8192 16384
//   bfloat16    183    93    29    27    32    27    27    28
//               214   113    37    34    38    35    34    39
//               200   107    45    44    51    55    57    66
//               237   129    48    43    58    56    61    74
//   binary32    167    90    49    48    51    49    50    52
//               201   107    57    58    59    58    59    63
//               178   101    84    83    86    88    84   100
//               176    98    65    69    69    75    88   115
// Forward, the bytes bound every row from 512 columns on.  A narrower row still
// takes a wave, whose sums and instructions bound it: at 64 columns 8 to 16 of
// the 64 lanes hold data.  Backward, the bytes bound binary32 rows of 512 to
// 4096 columns; other rows take 1.1 to 2.2 times the bytes' time, the more the
// wider they are: above 1024 columns a block has one row in flight.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "layer.hpp"
#include "layer_kernels.hpp"
#include "rows.hpp"

namespace oba {

namespace {

// Sums of two values over the waves of a row; every lane gets them.  `lds`
// holds 2 * W floats; the sums of the waves are added in wave order.
template <int W>
__device__ __forceinline__ void row_sum2(float& a, float& b, float* lds) {
  a = wave_sum(a);
  b = wave_sum(b);
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

// The same for one value, and for one in binary64 (`lds` holds W values).
template <int W, typename F>
__device__ __forceinline__ F row_sum(F a, F* lds) {
  a = wave_sum(a);
  if constexpr (W > 1) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = a;
    __syncthreads();
    a = 0;
    for (int w = 0; w < W; ++w) a += lds[w];
  }
  return a;
}

// The waves of a block: 4 rows at a time with a wave each, or one row.
template <int W>
constexpr int kThreads = W == 1 ? 256 : W * 64;
template <int W>
constexpr int kRows = W == 1 ? 4 : 1;

// Waves per SIMD asked of the compiler: what the registers of a row of NC
// pieces allow without spilling.  One instance spills all the same, the
// backward pass of binary32 rows above 8192 columns: 21 registers from the
// rows (24 bytes a lane), 90 from 8 bits (108 bytes), at two waves.
template <typename T, int NC>
constexpr int kFwdWaves = NC * kVec<T> <= 16 ? 4 : 2;
template <typename T, int NC>
constexpr int kBwdWaves = NC * kVec<T> <= 8 ? 4 : NC * kVec<T> <= 16 ? 3 : 2;

template <typename T, int NC, int W, bool KEEP>
__global__ __launch_bounds__((kThreads<W>), (kFwdWaves<T, NC>)) void k_norm_fwd(
    int64_t rows, int32_t cols, const T* __restrict__ x, int64_t ldx,
    const float* __restrict__ gamma, const float* __restrict__ beta, float eta,
    T* __restrict__ y, int64_t ldy, float* __restrict__ mean, float* __restrict__ rstd,
    uint8_t* __restrict__ q, uint8_t* __restrict__ e) {
  constexpr int V = kVec<T>, R = kRows<W>;
  __shared__ double lds64[W];
  __shared__ float lds[W];
  const int32_t groups = (cols + kAct8Group - 1) / kAct8Group;
  const int64_t stride = (int64_t)gridDim.x * R;
  int64_t r = (int64_t)blockIdx.x * R + (W == 1 ? threadIdx.x >> 6 : 0);
  // a row ahead: its loads are in flight while this one is worked on
  lu4 next[NC];
  if (r < rows) {
#pragma unroll
    for (int c = 0; c < NC; ++c) next[c] = load_raw(x + r * ldx, chunk_col<T, W>(c), cols);
  }
  float ga[NC][V], be[NC][V];
  load_params<T, NC, W>(gamma, cols, ga);
  load_params<T, NC, W>(beta, cols, be);
  const float n = (float)cols;
  const double n64 = (double)cols, inv64 = 1.0 / n64;
  for (; r < rows; r += stride) {
    float v[NC][V];
#pragma unroll
    for (int c = 0; c < NC; ++c) unpack_row<T>(next[c], chunk_col<T, W>(c), cols, v[c]);
    if (r + stride < rows) {
#pragma unroll
      for (int c = 0; c < NC; ++c)
        next[c] = load_raw(x + (r + stride) * ldx, chunk_col<T, W>(c), cols);
    }
    // The sum is binary64: a binary32 one is off by the rounding of values of
    // the mean's size, which xhat has in units of the spread (1e-3 of it at a
    // mean of 1000 spreads), and a mean near 0 by that of the values.  Its
    // quotient is put right by its remainder, so a constant row's is the value.
    double s = 0.0;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < V; ++j) s += (double)v[c][j];
    s = row_sum<W>(s, lds64);
    const double m = s * inv64, mean64 = __builtin_fma(__builtin_fma(-m, n64, s), inv64, m);
    const float mu = (float)mean64, off = (float)(mean64 - (double)mu);
    float s2 = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int32_t col = chunk_col<T, W>(c);
      centre(v[c], mu, off, col, cols);
#pragma unroll
      for (int j = 0; j < V; ++j) s2 += v[c][j] * v[c][j];
    }
    const float var = row_sum<W>(s2, lds) / n;
    const float rs = 1.0f / __builtin_sqrtf(var + eta);
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
        top = max_lanes<kAct8Group / V>(top);
        const uint32_t ex = group_exp(top);
        const float inv = inv_step_of(ex), step = step_of(ex);
        if (col < groups * kAct8Group) {  // a started group is written whole
          uint8_t* at = q + r * (int64_t)groups * kAct8Group + col;
          if constexpr (V == 8)
            *reinterpret_cast<lu2*>(at) =
                lu2{quant4(v[c], inv, step, ex != 255u), quant4(v[c] + 4, inv, step, ex != 255u)};
          else
            *reinterpret_cast<uint32_t*>(at) = quant4(v[c], inv, step, ex != 255u);
          if (col % kAct8Group == 0) e[r * groups + col / kAct8Group] = (uint8_t)ex;
        }
      }
    }
  }
}

// ---- backward ------------------------------------------------------------------
// What a row's backward pass reads, as it lies in memory.
template <typename T, int NC, bool KEPT>
struct BwdRow {
  lu4 dy[NC], add[NC];
  lu4 x[KEPT ? 1 : NC];
  lu2 q[KEPT ? NC : 1];
  uint32_t e[KEPT ? NC : 1];
  float rs, mu;
};

template <typename T, int NC, int W, bool KEPT>
__device__ __forceinline__ void load_bwd(const NormBwd& a, int64_t r, int32_t groups,
                                         BwdRow<T, NC, KEPT>& w) {
  w.rs = a.rstd[r];
#pragma unroll
  for (int c = 0; c < NC; ++c)
    w.dy[c] = load_raw(static_cast<const T*>(a.dy) + r * a.lddy, chunk_col<T, W>(c), a.cols);
  if constexpr (KEPT) {
    const uint8_t* qr = reinterpret_cast<const uint8_t*>(a.q) + r * (int64_t)groups * kAct8Group;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int32_t col = chunk_col<T, W>(c);
      w.q[c] = lu2{0u, 0u};
      w.e[c] = 0u;
      if (col < a.cols) {
        if constexpr (kVec<T> == 8) w.q[c] = *reinterpret_cast<const lu2*>(qr + col);
        else w.q[c][0] = *reinterpret_cast<const uint32_t*>(qr + col);
        w.e[c] = a.e[r * groups + col / kAct8Group];
      }
    }
  } else {
    w.mu = a.mean[r];
#pragma unroll
    for (int c = 0; c < NC; ++c)
      w.x[c] = load_raw(static_cast<const T*>(a.x) + r * a.ldx, chunk_col<T, W>(c), a.cols);
  }
  if (a.add) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
      w.add[c] = load_raw(static_cast<const T*>(a.add) + r * a.ldadd, chunk_col<T, W>(c), a.cols);
  }
}

template <typename T, int NC, int W, bool KEPT>
__global__ __launch_bounds__((kThreads<W>), (kBwdWaves<T, NC>)) void k_norm_bwd(NormBwd a) {
  constexpr int V = kVec<T>, R = kRows<W>;
  __shared__ float lds[2 * W];
  const int32_t cols = a.cols, groups = (cols + kAct8Group - 1) / kAct8Group;
  const int32_t worker = blockIdx.y;
  const int64_t base = (int64_t)worker * a.rows, stride = (int64_t)gridDim.x * R;
  int64_t i = (int64_t)blockIdx.x * R + (W == 1 ? threadIdx.x >> 6 : 0);
  // a row ahead where that leaves the registers for as many waves (at 16
  // columns a lane it cost a wave or spilled: 65 or 57 us against 50 for
  // 32768 x 1024 in bfloat16)
  constexpr bool kAhead = NC * V <= 8;
  BwdRow<T, NC, KEPT> next;
  if (kAhead && i < a.rows) load_bwd<T, NC, W, KEPT>(a, base + i, groups, next);
  float ga[NC][V], dg[NC][V], db[NC][V];
  load_params<T, NC, W>(a.gamma, cols, ga);
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < V; ++j) dg[c][j] = db[c][j] = 0.0f;
  const float n = (float)cols;
  for (; i < a.rows; i += stride) {
    const int64_t r = base + i;
    if (!kAhead) load_bwd<T, NC, W, KEPT>(a, r, groups, next);
    float h[NC][V], d[NC][V];
    lu4 add[NC];
    const float rs = next.rs, mu = next.mu;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int32_t col = chunk_col<T, W>(c);
      unpack_row<T>(next.dy[c], col, cols, d[c]);
      add[c] = next.add[c];
      if constexpr (KEPT) {
        const float step = step_of(next.e[c]);
#pragma unroll
        for (int j = 0; j < V; ++j) h[c][j] = dequant(next.q[c][j / 4], j % 4, step);
      } else {
        unpack_row<T>(next.x[c], col, cols, h[c]);
      }
    }
    if (kAhead && i + stride < a.rows) load_bwd<T, NC, W, KEPT>(a, r + stride, groups, next);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int32_t col = chunk_col<T, W>(c);
      if constexpr (!KEPT) {
#pragma unroll
        for (int j = 0; j < V; ++j) h[c][j] = col + j < cols ? (h[c][j] - mu) * rs : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float t = d[c][j] * ga[c][j];
        dg[c][j] += d[c][j] * h[c][j];
        db[c][j] += d[c][j];
        s1 += t;
        s2 += t * h[c][j];
        d[c][j] = t;
      }
    }
    row_sum2<W>(s1, s2, lds);
    const float m1 = s1 / n, m2 = s2 / n;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int32_t col = chunk_col<T, W>(c);
      float o[V];
      if (a.add) unpack(add[c], o, (const T*)nullptr);
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
// columns to a block of 16 waves that each add every 16th partial, joined in
// wave order.
constexpr int kJoinWaves = 16;
template <typename G>
__global__ __launch_bounds__(kJoinWaves * 64) void k_norm_wgrad(const float* __restrict__ part,
                                                                int32_t blocks, int32_t cols,
                                                                G* __restrict__ dgamma,
                                                                G* __restrict__ dbeta,
                                                                int64_t ldg) {
  __shared__ double lds[kJoinWaves][64];
  const int32_t l = threadIdx.x & 63, w = threadIdx.x >> 6, col = blockIdx.x * 64 + l;
  const float* p = part + (int64_t)blockIdx.y * blocks * 2 * cols;
  double s = 0.0;
  if (col < 2 * cols) {
#pragma unroll 4
    for (int32_t b = w; b < blocks; b += kJoinWaves) s += p[(int64_t)b * 2 * cols + col];
  }
  lds[w][l] = s;
  __syncthreads();
  if (w == 0 && col < 2 * cols) {
    s = 0.0;
    for (int v = 0; v < kJoinWaves; ++v) s += lds[v][l];
    if (col < cols) dgamma[(int64_t)blockIdx.y * ldg + col] = (G)(float)s;
    else dbeta[(int64_t)blockIdx.y * ldg + col - cols] = (G)(float)s;
  }
}

// ---- launchers -------------------------------------------------------------------
template <typename T, int NC, int W>
void fwd_keep(const NormFwd& a, hipStream_t st) {
  // one round of resident blocks: kFwdWaves waves on each of the 4 SIMDs of
  // 256 CUs, and no more than there are rows for
  const int64_t want = (a.rows + kRows<W> - 1) / kRows<W>;
  const int64_t most = 256 * 256 * kFwdWaves<T, NC> / kThreads<W>;
  const uint32_t grid = (uint32_t)std::min(want, most);
  const dim3 block(kThreads<W>);
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

// The instance that holds a row.  Binary32 rows take twice the pieces (M).
template <typename T>
void fwd(const NormFwd& a, hipStream_t st) {
  constexpr int M = 8 / kVec<T>;
  if (a.cols <= 512) fwd_keep<T, M, 1>(a, st);
  else if (a.cols <= 1024) fwd_keep<T, 2 * M, 1>(a, st);
  else if (a.cols <= 2048) fwd_keep<T, M, 4>(a, st);
  else if (a.cols <= 4096) fwd_keep<T, 2 * M, 4>(a, st);
  else if (a.cols <= 8192) fwd_keep<T, 2 * M, 8>(a, st);
  else fwd_keep<T, 4 * M, 8>(a, st);
}

template <typename T, int NC, int W>
void bwd_kept(const NormBwd& a, hipStream_t st) {
  const dim3 grid(norm_bwd_blocks(a.n, a.rows, a.cols), a.n), block(kThreads<W>);
  if (a.q) hipLaunchKernelGGL(HIP_KERNEL_NAME(k_norm_bwd<T, NC, W, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL(HIP_KERNEL_NAME(k_norm_bwd<T, NC, W, false>), grid, block, 0, st, a);
}

template <typename T>
void bwd(const NormBwd& a, hipStream_t st) {
  constexpr int M = 8 / kVec<T>;
  if (a.cols <= 512) bwd_kept<T, M, 1>(a, st);
  else if (a.cols <= 1024) bwd_kept<T, 2 * M, 1>(a, st);
  else if (a.cols <= 2048) bwd_kept<T, M, 4>(a, st);
  else if (a.cols <= 4096) bwd_kept<T, 2 * M, 4>(a, st);
  else if (a.cols <= 8192) bwd_kept<T, 2 * M, 8>(a, st);
  else bwd_kept<T, 4 * M, 8>(a, st);
}

template <typename G>
void wgrad(const NormBwd& a, hipStream_t st) {
  hipLaunchKernelGGL(HIP_KERNEL_NAME(k_norm_wgrad<G>), dim3((2 * a.cols + 63) / 64, a.n),
                     dim3(kJoinWaves * 64), 0, st, a.part, a.rows ? norm_bwd_blocks(a.n, a.rows, a.cols) : 0,
                     a.cols, static_cast<G*>(a.dgamma), static_cast<G*>(a.dbeta), a.ldg);
}

}  // namespace

// One round of resident blocks over all workers (kBwdWaves waves a SIMD), and
// no more than a worker has rows for.
int32_t norm_bwd_blocks(int32_t n, int64_t rows, int32_t cols) {
  const int64_t per = cols <= 1024 ? 4 : 1;  // rows of a block at a time
  const int64_t all = cols <= 512 ? 1024 : cols <= 1024 ? 768 : cols <= 2048 ? 1024
                      : cols <= 4096 ? 768 : 256;
  const int64_t most = std::max<int64_t>(1, all / n);
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
