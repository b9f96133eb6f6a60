// join.hip -- what lies between two blocks of a residual network, in one pass
// (gfx950): the norm behind a block, dropout, its gate, the residual sum and the
// norm before the next block.
//
// Forward, per row, every step optional but the sum:
//   n = norm(b) * gamma_b + beta_b,   r = alpha * x + gate * drop(n),
//   z = norm(r) * gamma + beta
// norm(v) = (v - mean) * rstd with rstd = 1 / sqrt(mean((v - mean)^2) + eta), or
// without the mean (kind kNormRms).  Backward, with h = norm(r) and k = norm(b)
// from 8 bits, per row and with a = dz * gamma:
//   D = rstd * (a - mean(a) - h * mean(a * h)) + dr,   dx = alpha * D
//   e = drop(D),   c = e * gate * gamma_b
//   db = rstd_b * (c - mean(c) - k * mean(c * k))
// (without mean(a) and mean(c) for kNormRms) and per worker and column four
// sums, from which all parameters' gradients come:
//   dgamma = sum dz * h, dbeta = sum dz, S = sum e * k, T = sum e:
//   dgamma_b = gate * S, dbeta_b = gate * T, dgate = gamma_b * S + beta_b * T
//
// A row is read once into registers: eight columns a lane, by 1 to 16 waves (16
// columns a lane above 8192).  A block walks many rows, so parameters are read
// once and the column sums stay in binary32 registers until its last row; they
// are written as partial sums and added per column in binary64 in a fixed
// order.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "layer.hpp"
#include "philox.hpp"
#include "rows.hpp"
#include "sublayer_kernels.hpp"

namespace oba {

namespace {

// W waves to a row; blocks of 8 waves hold 8 / W rows at a time, 16 waves one.
template <int W>
constexpr int kThreads = W == 16 ? 1024 : 512;
template <int W>
constexpr int kRows = kThreads<W> / 64 / W;

// Sums of two values over a row's W waves: every lane gets them, added in wave
// order.  One barrier: two calls in turn use the two halves of `lds`, and a wave
// that writes a half again has passed the barrier of the call between, behind
// every wave's reads of this half.  All waves of a block call it together.
template <int W, typename F>
__device__ __forceinline__ void row_sums(F& a, F& b, F (*lds)[2][kThreads<W> / 64], int& half) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (W > 1) {
    const int w = threadIdx.x >> 6, first = w & ~(W - 1);
    if ((threadIdx.x & 63) == 0) {
      lds[half][0][w] = a;
      lds[half][1][w] = b;
    }
    __syncthreads();
    a = b = 0;
#pragma unroll 4
    for (int i = 0; i < W; ++i) {
      a += lds[half][0][first + i];
      b += lds[half][1][first + i];
    }
    half ^= 1;
  }
}

// Columns of a row that its wave w holds.
template <typename T, int NC, int W>
__device__ __forceinline__ int32_t wave_cols(int32_t w, int32_t cols) {
  int32_t n = 0;
#pragma unroll
  for (int c = 0; c < NC; ++c) n += min(max(cols - (c * W + w) * 64 * kVec<T>, 0), 64 * kVec<T>);
  return n;
}

// What a norm divides by: columns of the row and of the lane's wave, with their
// reciprocals, which a division for each row would cost 20 instructions of
// binary64.  A quotient by a reciprocal is put right by its remainder.
struct Share {
  double n, inv;
};
__device__ __forceinline__ Share share_of(int32_t n) {
  auto uniform = [](double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)u);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(u >> 32));
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
  };
  return Share{uniform((double)n), uniform(n > 0 ? 1.0 / (double)n : 0.0)};
}
__device__ __forceinline__ double quotient(double s, double n, double inv) {
  const double m = s * inv;
  return __builtin_fma(__builtin_fma(-m, n, s), inv, m);
}
__device__ __forceinline__ float quotient(float s, float n, float inv) {
  const float m = s * inv;
  return __builtin_fmaf(__builtin_fmaf(-m, n, s), inv, m);
}

// The mean and the squares around it of the columns that a wave holds.  The sums
// are taken twice, the second time around the first one's mean m, so that the mean
// and the squares are off by what rounds differences, not values: m + sum(v - m) /
// n.  For binary32 rows the first sum is binary64 and the second needs no mean:
// a row of one value, whose sum binary32 does not hold, is then centred to 0.  For
// 16-bit rows (and r made of them) binary32 does.
template <typename T, int NC, int W>
__device__ __forceinline__ void wave_moments(const float (&v)[NC][kVec<T>], int32_t cols,
                                             const Share& part, double& mean, double& squares) {
  constexpr int V = kVec<T>;
  float m;
  if constexpr (V == 4) {
    double s = 0.0;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < V; ++j) s += (double)v[c][j];
    mean = quotient(wave_sum(s), part.n, part.inv);
    m = (float)mean;
  } else {
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < V; ++j) s += v[c][j];
    m = quotient(wave_sum(s), (float)part.n, (float)part.inv);
  }
  float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    // lanes that hold none of the row, and elements past its end, add nothing
    const int32_t col = chunk_col<T, W>(c);
    const float mc = col < cols ? m : 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float t = v[c][j] - mc;
      if (cols % V != 0) t = col + j < cols ? t : 0.0f;
      if constexpr (V == 8) s1 += t;
      s2 = __builtin_fmaf(t, t, s2);
    }
  }
  squares = (double)wave_sum(s2);
  if constexpr (V == 8) {
    const double d = (double)wave_sum(s1);
    mean = __builtin_fma(d, part.inv, (double)m);
    squares = __builtin_fma(-d * part.inv, d, squares);
  }
}

// Rows to their normalised form in place; the reciprocal of the spread.  The
// waves' squares are moved to the row's mean, n_w (mean_w - mean)^2 for each, so
// that one exchange between the waves serves mean and spread.
template <typename T, int NC, int W>
__device__ __forceinline__ float normalise(float (&v)[NC][kVec<T>], int32_t cols, int kind,
                                           float eta, const Share& row, const Share& part, double (*lds)[2][kThreads<W> / 64],
                                           int& half) {
  constexpr int V = kVec<T>;
  const int wave = threadIdx.x >> 6, first = wave & ~(W - 1);
  double squares;
  float mu = 0.0f, off = 0.0f;
  if (kind == kNormLayer) {
    double mean;
    wave_moments<T, NC, W>(v, cols, part, mean, squares);
    if constexpr (W > 1) {
      if ((threadIdx.x & 63) == 0) {
        lds[half][0][wave] = mean;
        lds[half][1][wave] = squares;
      }
      __syncthreads();
      double all = 0.0;
#pragma unroll 4
      for (int i = 0; i < W; ++i)
        all = __builtin_fma((double)wave_cols<T, NC, W>(i, cols), lds[half][0][first + i], all);
      mean = quotient(all, row.n, row.inv);
      squares = 0.0;
#pragma unroll 4
      for (int i = 0; i < W; ++i) {
        const double n = (double)wave_cols<T, NC, W>(i, cols);
        const double d = lds[half][0][first + i] - mean;
        squares += __builtin_fma(n * d, d, lds[half][1][first + i]);
      }
      half ^= 1;
    }
    mu = (float)mean;
    off = (float)(mean - (double)mu);
  } else {
    float s2 = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < V; ++j) s2 = __builtin_fmaf(v[c][j], v[c][j], s2);
    s2 = wave_sum(s2);
    squares = (double)s2;
    if constexpr (W > 1) {
      if ((threadIdx.x & 63) == 0) lds[half][0][wave] = squares;
      __syncthreads();
      squares = 0.0;
#pragma unroll 4
      for (int i = 0; i < W; ++i) squares += lds[half][0][first + i];
      half ^= 1;
    }
  }
  const float rs = 1.0f / __builtin_sqrtf((float)(squares * row.inv) + eta);
  if (kind == kNormLayer) {
    const float low = -off * rs;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
      for (int j = 0; j < V; ++j) v[c][j] = __builtin_fmaf(v[c][j] - mu, rs, low);
      if (cols % (NC * W * 64 * V) != 0) {  // 0 stays past the row's end
        const int32_t col = chunk_col<T, W>(c);
#pragma unroll
        for (int j = 0; j < V; ++j) v[c][j] = col + j < cols ? v[c][j] : 0.0f;
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < V; ++j) v[c][j] *= rs;
  }
  return rs;
}

// A lane's columns of a row to 8 bits; four or eight lanes hold a group.
template <typename T>
__device__ __forceinline__ void keep(const float (&v)[kVec<T>], int8_t* q, uint8_t* e, int64_t row,
                                     int32_t groups, int32_t col) {
  constexpr int V = kVec<T>;
  uint32_t top = 0;
  if constexpr (V == 8) {
    top = magnitude8(v);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) top = max(top, magnitude(v[j]));
  }
  top = max_lanes<kAct8Group / V>(top);
  const uint32_t ex = group_exp(top);
  const float inv = inv_step_of(ex), step = step_of(ex);
  const bool finite = ex != 255u;
  uint32_t w[V / 4];
  if (past_range(top)) {
    for (int j = 0; j < V / 4; ++j) w[j] = quant4(v + 4 * j, inv, step, finite);
  } else {
    for (int j = 0; j < V / 4; ++j) w[j] = quant4_in(v + 4 * j, inv, finite);
  }
  if (col >= groups * kAct8Group) return;  // a started group is written whole
  int8_t* at = q + row * (int64_t)groups * kAct8Group + col;
  if constexpr (V == 8) *reinterpret_cast<lu2*>(at) = lu2{w[0], w[1]};
  else *reinterpret_cast<uint32_t*>(at) = w[0];
  if (col % kAct8Group == 0) e[row * groups + col / kAct8Group] = (uint8_t)ex;
}

// A parameter vector's columns in a lane, `other` where there is no vector; 0
// past the last column.  Rows of 8 columns a lane hold them in registers from row
// to row; at 16 columns a lane they are read again for each row (from cache): held
// they spilled.
template <typename T, int NC, int W>
struct Params {
  static constexpr int V = kVec<T>;
  static constexpr bool kHold = NC * V <= 8;
  const float* p;
  float other;
  float held[kHold ? NC : 1][V];

  __device__ __forceinline__ void read(int c, int32_t cols, float (&v)[V]) const {
    const int32_t col = chunk_col<T, W>(c);
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      if (!p) {
        for (int i = 0; i < 4; ++i) v[j + i] = other;
      } else if (col + j + 4 <= cols) {
        const Four f = *reinterpret_cast<const Four*>(p + col + j);
        for (int i = 0; i < 4; ++i) v[j + i] = f.v[i];
      } else {
        for (int i = 0; i < 4; ++i) v[j + i] = col + j + i < cols ? p[col + j + i] : 0.0f;
      }
    }
  }
  __device__ __forceinline__ Params(const float* from, float without, int32_t cols)
      : p(from), other(without) {
    if constexpr (kHold) {
#pragma unroll
      for (int c = 0; c < NC; ++c) read(c, cols, held[c]);
    }
  }
  __device__ __forceinline__ void get(int c, int32_t cols, float (&v)[V]) const {
    if constexpr (kHold) {
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = held[c][j];
    } else {
      read(c, cols, v);
    }
  }
};

// Waves per SIMD asked of the compiler.  A row of 16 columns a lane has 16 waves
// in a block, so four to a SIMD too; its loads are not a row ahead, which spilled.
constexpr int kWaves = 4;
template <typename T, int NC>
constexpr bool kAhead = NC * kVec<T> <= 8;

// The row of a block's first round that a wave belongs to, the same for all its
// lanes: addresses of rows then need no vector registers.
template <int W>
__device__ __forceinline__ int32_t wave_row() {
  return __builtin_amdgcn_readfirstlane((int32_t)threadIdx.x / (W * 64));
}

template <typename T, int NC, int W>
__global__ __launch_bounds__((kThreads<W>), kWaves) void k_join_fwd(JoinFwd args) {
  JoinFwd a = arguments(args);
  constexpr int V = kVec<T>, R = kRows<W>;
  __shared__ double lds[2][2][kThreads<W> / 64];
  int half = 0;
  const int32_t cols = a.cols, groups = (cols + kAct8Group - 1) / kAct8Group;
  const int64_t rows = a.rows, stride = (int64_t)gridDim.x * R;
  const bool first_lane = (threadIdx.x & (W * 64 - 1)) == 0;
  const RngKey key = load_key(a.drop);
  int64_t r = (int64_t)blockIdx.x * R + wave_row<W>();
  constexpr bool A = kAhead<T, NC>;  // each loaded anew once the row before is taken out of it
  lu4 nx[NC], nb[NC];
  auto load = [&](const void* from, int64_t ld, int64_t row, lu4 (&to)[NC]) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
      to[c] = load_raw(global(static_cast<const T*>(from)) + row * ld, chunk_col<T, W>(c), cols);
  };
  if (A && r < a.rows) {
    load(a.x, a.ldx, r, nx);
    if (a.b) load(a.b, a.ldb, r, nb);
  }
  const Params<T, NC, W> gate(global(a.gate), 1.0f, cols), gb(global(a.gamma_b), 1.0f, cols),
      bb(global(a.beta_b), 0.0f, cols), ga(global(a.gamma), 1.0f, cols),
      be(global(a.beta), 0.0f, cols);
  const Share row = share_of(cols),
              part = share_of(wave_cols<T, NC, W>((threadIdx.x >> 6) & (W - 1), cols));
  // the rows of a block go round together: its waves meet at the sums' barriers
  for (int64_t r0 = (int64_t)blockIdx.x * R; r0 < rows; r0 += stride, r += stride) {
    const bool in = r < rows, more = r + stride < rows;
    a = arguments(args);
    const lu4 none = {0u, 0u, 0u, 0u};
    float v[NC][V];
    if (!A && a.b && in) load(a.b, a.ldb, r, nb);
#pragma unroll
    for (int c = 0; c < NC; ++c)
      unpack_row<T>(in && a.b ? nb[c] : none, chunk_col<T, W>(c), cols, v[c]);
    if (A && a.b && more) load(a.b, a.ldb, r + stride, nb);
    if (a.b) {
      if (a.gamma_b) {
        const float rs = normalise<T, NC, W>(v, cols, a.kind, a.eta, row, part, lds, half);
        if (in && first_lane) global(a.rstd_b)[r] = rs;
      }
      if (a.qb && in) {
#pragma unroll
        for (int c = 0; c < NC; ++c) keep<T>(v[c], global(a.qb), global(a.eb), r, groups, chunk_col<T, W>(c));
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float f[V], o[V];
        if (a.gamma_b) {
          gb.get(c, cols, f);
          bb.get(c, cols, o);
#pragma unroll
          for (int j = 0; j < V; ++j) v[c][j] = __builtin_fmaf(v[c][j], f[j], o[j]);
        }
        if (a.drop.threshold) drop<V>(a.drop, key, r, (cols + 7) / 8, chunk_col<T, W>(c), v[c]);
        if (a.gate) {
          gate.get(c, cols, f);
#pragma unroll
          for (int j = 0; j < V; ++j) v[c][j] *= f[j];
        }
      }
    }
    a = arguments(args);
    if (!A && in) load(a.x, a.ldx, r, nx);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float x[V];
      unpack_row<T>(in ? nx[c] : none, chunk_col<T, W>(c), cols, x);
#pragma unroll
      for (int j = 0; j < V; ++j) v[c][j] = __builtin_fmaf(a.alpha, x[j], v[c][j]);
    }
    if (A && more) load(a.x, a.ldx, r + stride, nx);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int32_t col = chunk_col<T, W>(c);
      if (a.r && in && col < cols) store_row(global(static_cast<T*>(a.r)) + r * a.ldr, col, cols, v[c]);
    }
    a = arguments(args);
    if (!a.gamma) continue;
    const float rs = normalise<T, NC, W>(v, cols, a.kind, a.eta, row, part, lds, half);
    if (!in) continue;
    if (first_lane) global(a.rstd)[r] = rs;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int32_t col = chunk_col<T, W>(c);
      if (a.q) keep<T>(v[c], global(a.q), global(a.e), r, groups, col);
      float f[V], o[V];
      ga.get(c, cols, f);
      be.get(c, cols, o);
#pragma unroll
      for (int j = 0; j < V; ++j) v[c][j] = __builtin_fmaf(v[c][j], f[j], o[j]);
      if (col < cols) store_row(global(static_cast<T*>(a.z)) + r * a.ldz, col, cols, v[c]);
    }
  }
}

// ---- backward ------------------------------------------------------------------
// What a row's backward pass reads, as it lies in memory, a row ahead: each half
// is loaded anew as soon as the row before has been taken out of it.
template <int NC>
struct BwdRow {
  lu4 dz[NC], dr[NC];
  lu2 q[NC], qb[NC];
  uint32_t e[NC], eb[NC];
  float rs, rsb;
};

template <typename T>
__device__ __forceinline__ void load_kept(const int8_t* q, const uint8_t* e, int64_t row,
                                          int32_t groups, int32_t col, int32_t cols, lu2& qr,
                                          uint32_t& er) {
  qr = lu2{0u, 0u};
  er = 0u;
  if (col < cols) {
    const int8_t* at = q + row * (int64_t)groups * kAct8Group + col;
    if constexpr (kVec<T> == 8) qr = *reinterpret_cast<const lu2*>(at);
    else qr[0] = *reinterpret_cast<const uint32_t*>(at);
    er = e[row * groups + col / kAct8Group];
  }
}

// The values; 0 where there are none.
template <typename T>
__device__ __forceinline__ void decode(bool there, lu2 q, uint32_t e, float (&v)[kVec<T>]) {
  const float step = there ? step_of(e) : 0.0f;
#pragma unroll
  for (int j = 0; j < kVec<T> / 4; ++j) dequant4(q[j], step, v + 4 * j);
}

template <typename T, int NC, int W>
__device__ __forceinline__ void load_upper(const JoinBwd& a, int64_t r, BwdRow<NC>& w) {
  if (!a.dz) return;
  const int32_t groups = (a.cols + kAct8Group - 1) / kAct8Group;
  w.rs = global(a.rstd)[r];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int32_t col = chunk_col<T, W>(c);
    w.dz[c] = load_raw(global(static_cast<const T*>(a.dz)) + r * a.lddz, col, a.cols);
    load_kept<T>(global(a.q), global(a.e), r, groups, col, a.cols, w.q[c], w.e[c]);
  }
}

template <typename T, int NC, int W>
__device__ __forceinline__ void load_lower(const JoinBwd& a, int64_t r, BwdRow<NC>& w) {
  const int32_t groups = (a.cols + kAct8Group - 1) / kAct8Group;
  if (a.gamma_b) w.rsb = global(a.rstd_b)[r];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int32_t col = chunk_col<T, W>(c);
    if (a.dr) w.dr[c] = load_raw(global(static_cast<const T*>(a.dr)) + r * a.lddr, col, a.cols);
    if (a.qb) load_kept<T>(global(a.qb), global(a.eb), r, groups, col, a.cols, w.qb[c], w.eb[c]);
  }
}

// The norm's input gradient from that of its normalised rows, in place.  What it
// leaves past a row's end reaches no result: the sums of the branch there are not
// stored, and the parameters, 0 there, keep it out of the next row sums.
template <typename T, int NC, int W>
__device__ __forceinline__ void through(float (&d)[NC][kVec<T>], const float (&h)[NC][kVec<T>],
                                        float rs, int32_t cols, int kind,
                                        float (*lds)[2][kThreads<W> / 64], int& half) {
  constexpr int V = kVec<T>;
  float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      s1 += d[c][j];
      s2 = __builtin_fmaf(d[c][j], h[c][j], s2);
    }
  row_sums<W>(s1, s2, lds, half);
  const float n = (float)cols;
  const float m1 = kind == kNormLayer ? -rs * (s1 / n) : 0.0f, m2 = -s2 / n;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < V; ++j)
      d[c][j] = __builtin_fmaf(__builtin_fmaf(m2, h[c][j], d[c][j]), rs, m1);
}

template <typename T, int NC, int W>
__global__ __launch_bounds__((kThreads<W>), kWaves) void k_join_bwd(JoinBwd args) {
  JoinBwd a = arguments(args);
  constexpr int V = kVec<T>, R = kRows<W>;
  __shared__ float lds[2][2][kThreads<W> / 64];
  int half = 0;
  const int32_t cols = a.cols, worker = blockIdx.y;
  const int64_t rows = a.rows, base = worker * rows, stride = (int64_t)gridDim.x * R;
  const RngKey key = load_key(a.drop);
  int64_t i = (int64_t)blockIdx.x * R + wave_row<W>();
  constexpr bool A = kAhead<T, NC>;
  BwdRow<NC> next;
  if (A && i < rows) {
    load_upper<T, NC, W>(a, base + i, next);
    load_lower<T, NC, W>(a, base + i, next);
  }
  const Params<T, NC, W> ga(global(a.gamma), 1.0f, cols), gate(global(a.gate), 1.0f, cols),
      gb(global(a.gamma_b), 1.0f, cols);
  float sums[4][NC][V];
#pragma unroll
  for (int s = 0; s < 4; ++s)
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < V; ++j) sums[s][c][j] = 0.0f;
  for (int64_t i0 = (int64_t)blockIdx.x * R; i0 < rows; i0 += stride, i += stride) {
    const bool in = i < rows, more = i + stride < rows;
    const int64_t r = base + i;
    const lu4 none = {0u, 0u, 0u, 0u};
    float d[NC][V];
    a = arguments(args);
    if (!A && in) load_upper<T, NC, W>(a, r, next);
    if (a.dz) {
      float h[NC][V];
      const float rs = in ? next.rs : 0.0f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        unpack_row<T>(in ? next.dz[c] : none, chunk_col<T, W>(c), cols, d[c]);
        decode<T>(in, next.q[c], next.e[c], h[c]);
      }
      if (A && more) load_upper<T, NC, W>(a, r + stride, next);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float f[V];
        ga.get(c, cols, f);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          sums[0][c][j] = __builtin_fmaf(d[c][j], h[c][j], sums[0][c][j]);
          sums[1][c][j] += d[c][j];
          d[c][j] *= f[j];
        }
      }
      through<T, NC, W>(d, h, rs, cols, a.kind, lds, half);
    } else {
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < V; ++j) d[c][j] = 0.0f;
    }
    a = arguments(args);
    if (!A && in) load_lower<T, NC, W>(a, r, next);
    float k[NC][V];
    const float rsb = in ? next.rsb : 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (a.dr) {
        float o[V];
        unpack_row<T>(in ? next.dr[c] : none, chunk_col<T, W>(c), cols, o);
#pragma unroll
        for (int j = 0; j < V; ++j) d[c][j] += o[j];
      }
      decode<T>(in && a.qb, next.qb[c], next.eb[c], k[c]);
    }
    if (A && more) load_lower<T, NC, W>(a, r + stride, next);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int32_t col = chunk_col<T, W>(c);
      float o[V];
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] = a.alpha * d[c][j];
      if (in && col < cols) store_row(global(static_cast<T*>(a.dx)) + r * a.lddx, col, cols, o);
      if (a.drop.threshold) drop<V>(a.drop, key, r, (cols + 7) / 8, col, d[c]);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        sums[2][c][j] = __builtin_fmaf(d[c][j], k[c][j], sums[2][c][j]);
        sums[3][c][j] += d[c][j];
      }
      if (a.gate) {
        gate.get(c, cols, o);
#pragma unroll
        for (int j = 0; j < V; ++j) d[c][j] *= o[j];
      }
      if (a.gamma_b) {
        gb.get(c, cols, o);
#pragma unroll
        for (int j = 0; j < V; ++j) d[c][j] *= o[j];
      }
    }
    if (!a.db) continue;
    if (a.gamma_b) through<T, NC, W>(d, k, rsb, cols, a.kind, lds, half);
    if (!in) continue;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int32_t col = chunk_col<T, W>(c);
      if (col < cols) store_row(global(static_cast<T*>(a.db)) + r * a.lddb, col, cols, d[c]);
    }
  }
  // the block's column sums: its rows add theirs in order
  if (!a.part) return;
  float* part = global(a.part) + ((int64_t)worker * gridDim.x + blockIdx.x) * 4 * cols;
  if constexpr (R > 1) {
    __shared__ float all[4][NC * W * 64 * V];
    for (int g = 0; g < R; ++g) {
      if ((int)threadIdx.x / (W * 64) == g) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < V; ++j) {
              const int32_t at = chunk_col<T, W>(c) + j;
              all[s][at] = (g ? all[s][at] : 0.0f) + sums[s][c][j];
            }
      }
      __syncthreads();
    }
    for (int32_t col = threadIdx.x; col < cols; col += kThreads<W>)
      for (int s = 0; s < 4; ++s) part[s * cols + col] = all[s][col];
  } else {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int32_t col = chunk_col<T, W>(c) + j;
          if (col < cols) part[s * cols + col] = sums[s][c][j];
        }
  }
}

// The parameters' gradients of a worker from its blocks' partial sums, in
// binary64: 64 columns to a block of 16 waves that each add every 16th partial,
// joined in wave order.  blockIdx.z: the sums of the norm before the next block,
// or those of the branch.
constexpr int kJoinWaves = 16;
template <typename G>
__global__ __launch_bounds__(kJoinWaves * 64) void k_join_wgrad(JoinBwd a, int32_t blocks) {
  __shared__ double lds[kJoinWaves][2][64];
  const int32_t l = threadIdx.x & 63, w = threadIdx.x >> 6, col = blockIdx.x * 64 + l;
  const int64_t cols = a.cols, worker = blockIdx.y;
  const float* p = a.part + (worker * blocks * 4 + blockIdx.z * 2) * cols + col;
  double s = 0.0, t = 0.0;
  if (col < cols) {
#pragma unroll 4
    for (int32_t b = w; b < blocks; b += kJoinWaves) {
      s += p[(int64_t)b * 4 * cols];
      t += p[((int64_t)b * 4 + 1) * cols];
    }
  }
  lds[w][0][l] = s;
  lds[w][1][l] = t;
  __syncthreads();
  if (w > 0 || col >= cols) return;
  s = t = 0.0;
  for (int v = 0; v < kJoinWaves; ++v) {
    s += lds[v][0][l];
    t += lds[v][1][l];
  }
  const int64_t at = worker * a.ldg + col;
  auto store = [&](void* to, double v) {
    if (to) static_cast<G*>(to)[at] = (G)(float)v;
  };
  if (blockIdx.z == 0) {
    store(a.dgamma, s);
    store(a.dbeta, t);
  } else {
    const double gate = a.gate ? a.gate[col] : 1.0;
    store(a.dgate, (a.gamma_b ? s * a.gamma_b[col] : s) + (a.beta_b ? t * a.beta_b[col] : 0.0));
    store(a.dgamma_b, s * gate);
    store(a.dbeta_b, t * gate);
  }
}

// ---- launchers -------------------------------------------------------------------
// One round of resident blocks, and no more than there are rows for.
constexpr int64_t kResident = 512;  // blocks of 512 threads, 4 waves a SIMD

template <typename T, int NC, int W>
void fwd(const JoinFwd& a, hipStream_t st) {
  const int64_t want = (a.rows + kRows<W> - 1) / kRows<W>;
  const int64_t most = kResident * 512 / kThreads<W>;
  hipLaunchKernelGGL(HIP_KERNEL_NAME(k_join_fwd<T, NC, W>), dim3((uint32_t)std::min(want, most)),
                     dim3(kThreads<W>), 0, st, a);
}

template <typename T, int NC, int W>
void bwd(const JoinBwd& a, hipStream_t st) {
  hipLaunchKernelGGL(HIP_KERNEL_NAME(k_join_bwd<T, NC, W>),
                     dim3(join_bwd_blocks(a.n, a.rows, a.cols), a.n), dim3(kThreads<W>), 0, st, a);
}

// The instance that holds a row: 8 columns a lane, 16 above 8192 columns.
// Binary32 rows take twice the pieces (M).
template <typename T, class A, class F>
void pick(const A& a, F&& f) {
  constexpr int M = 8 / kVec<T>;
  if (a.cols <= 512) f(std::integral_constant<int, M>{}, std::integral_constant<int, 1>{});
  else if (a.cols <= 1024) f(std::integral_constant<int, M>{}, std::integral_constant<int, 2>{});
  else if (a.cols <= 2048) f(std::integral_constant<int, M>{}, std::integral_constant<int, 4>{});
  else if (a.cols <= 4096) f(std::integral_constant<int, M>{}, std::integral_constant<int, 8>{});
  else if (a.cols <= 8192) f(std::integral_constant<int, M>{}, std::integral_constant<int, 16>{});
  else f(std::integral_constant<int, 2 * M>{}, std::integral_constant<int, 16>{});
}

template <typename T>
void fwd(const JoinFwd& a, hipStream_t st) {
  pick<T>(a, [&](auto nc, auto w) { fwd<T, nc.value, w.value>(a, st); });
}
template <typename T>
void bwd(const JoinBwd& a, hipStream_t st) {
  pick<T>(a, [&](auto nc, auto w) { bwd<T, nc.value, w.value>(a, st); });
}

template <typename G>
void wgrad(const JoinBwd& a, hipStream_t st) {
  const int32_t blocks = a.rows ? join_bwd_blocks(a.n, a.rows, a.cols) : 0;
  hipLaunchKernelGGL(HIP_KERNEL_NAME(k_join_wgrad<G>), dim3((a.cols + 63) / 64, a.n, 2),
                     dim3(kJoinWaves * 64), 0, st, a, blocks);
}

}  // namespace

int32_t join_bwd_blocks(int32_t n, int64_t rows, int32_t cols) {
  const int64_t per = cols <= 512 ? 8 : cols <= 1024 ? 4 : cols <= 2048 ? 2 : 1;
  const int64_t all = cols <= 4096 ? kResident : kResident / 2;
  const int64_t most = std::max<int64_t>(1, all / n);
  return (int32_t)std::max<int64_t>(1, std::min<int64_t>((rows + per - 1) / per, most));
}

void launch_join(const JoinFwd& a, hipStream_t st) {
  if (a.dtype == kGradF32) fwd<float>(a, st);
  else if (a.dtype == kGradF16) fwd<_Float16>(a, st);
  else fwd<__bf16>(a, st);
}

void launch_join_backward(const JoinBwd& a, hipStream_t st) {
  if (a.dtype == kGradF32) bwd<float>(a, st);
  else if (a.dtype == kGradF16) bwd<_Float16>(a, st);
  else bwd<__bf16>(a, st);
}

void launch_join_weight_grad(const JoinBwd& a, hipStream_t st) {
  if (a.g_dtype == kGradF32) wgrad<float>(a, st);
  else if (a.g_dtype == kGradF16) wgrad<_Float16>(a, st);
  else wgrad<__bf16>(a, st);
}

}  // namespace oba
