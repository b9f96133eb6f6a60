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
// A row is read once into registers: eight columns a lane, by as many waves as it
// has 512 columns (16 columns a lane above 8192).  A block walks many rows, so
// parameters are read once and the column sums stay in binary32 until its last
// row; they are written as partial sums and added per column in binary64 in a
// fixed order.
//
// Bound by the memory and, nearly as much, by the vector unit: a wave's 512 columns
// take 630 instructions forward with both norms, dropout and both kept forms (a
// sixth of them the random bits, whose 32-bit products are four times as long), 78 %
// of the unit's time at 32768 x 1024.  So waves without columns are what costs most:
// with the waves a row rounded up to 1, 2, 4, 8 or 16, 33.5 million bfloat16 elements
// of 2500 columns took 157 us, of 4500 199 us, and 93 and 136 with the waves counted
// out; a row narrower than a wave takes a wave all the same (256 columns 121 us, 64 437).
// Measured, both norms, dropout, all kept, bfloat16: 32768 x 1024 80 us (4.2 TB/s), 8192 x
// 4096 82 us (4.1 TB/s), back 79 and 88 us; binary32, the RMS norm of 2048 x 8192 58 us
// (5.0 TB/s).
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

// Columns of a wave: 8 a lane, or 16 where a row has more than 16 such waves.
// Rows of one wave, ONE, need no exchange.
template <typename T, int NC>
constexpr int32_t kWaveCols = NC * kVec<T> * 64;

// Rows to a block: forward, four of one wave, else one (its waves wait for no
// other row's).  Backward, where a block's rows share one partial sum, eight waves'
// if they are whole rows, else what 16 waves hold: fewer partial sums, but all wait
// for one another (1600 columns: 91 us against 100 with 16; 2500: 132 against 95,
// 4096: 97 against 88, for 2^25 elements).
template <bool BACK>
__host__ __device__ inline int32_t block_rows(int32_t waves) {
  if (!BACK) return waves == 1 ? 4 : 1;
  return waves == 1 || waves == 2 || waves == 4 ? 8 / waves : 16 / waves;
}

// Where a lane's columns lie: chunk c at `at` + c * `step`; its wave is number
// `wave` of the `waves` of the block's row number `row`, whose first wave is
// `first`.  All but `at` is the same for a wave's lanes.
template <typename T, int NC, bool ONE>
struct Where {
  int32_t waves, wave, first, row, at, step;
  __device__ __forceinline__ explicit Where(int32_t cols) {
    const int32_t w = __builtin_amdgcn_readfirstlane((int32_t)threadIdx.x >> 6);
    waves = ONE ? 1 : (cols + kWaveCols<T, NC> - 1) / kWaveCols<T, NC>;
    row = ONE ? w : __builtin_amdgcn_readfirstlane(w / waves);
    first = row * waves;
    wave = w - first;
    at = (wave * 64 + ((int32_t)threadIdx.x & 63)) * kVec<T>;
    step = waves * 64 * kVec<T>;
  }
  __device__ __forceinline__ int32_t col(int c) const { return at + c * step; }
  // columns of the row that its wave w holds
  __device__ __forceinline__ int32_t part(int32_t w, int32_t cols) const {
    int32_t n = 0;
#pragma unroll
    for (int c = 0; c < NC; ++c)
      n += min(max(cols - c * step - w * 64 * kVec<T>, 0), 64 * kVec<T>);
    return n;
  }
};

// Of a lane's columns from col those past the row's end to 0.
template <int V>
__device__ __forceinline__ void clear_past(float (&v)[V], int32_t col, int32_t cols) {
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = col + j < cols ? v[j] : 0.0f;
}

// Over the waves of a row: each wave's two values are laid into LDS, and lane i of
// every 16 takes wave i's, so that sums over the waves are four exchanges however
// many waves there are.  One barrier: two meetings in turn use the two halves of
// `lds`, and a wave that writes a half again has passed the barrier of the meeting
// between, behind every wave's reads of this half.  All waves of a block meet
// together.
template <typename F>
using Meet = F __attribute__((ext_vector_type(2)));

template <typename T, int NC, typename F>
__device__ __forceinline__ Meet<F> meet(F a, F b, const Where<T, NC, false>& at,
                                        Meet<F> (*lds)[16], int& half) {
  if ((threadIdx.x & 63) == 0) lds[half][at.first + at.wave] = Meet<F>{a, b};
  __syncthreads();
  const int32_t i = (int32_t)threadIdx.x & 15;
  Meet<F> v = lds[half][at.first + min(i, at.waves - 1)];
  half ^= 1;
  if (i >= at.waves) v[1] = 0;
  return v;
}
// The sum of 16 neighbouring lanes, in all of them.
__device__ __forceinline__ float sum16(float v) {
  v += dppf<kXor1>(v);
  v += dppf<kXor2>(v);
  v += dppf<kHalfMirror>(v);
  return v + dppf<kMirror>(v);
}
__device__ __forceinline__ double sum16(double v) {
  v += dppd<kXor1>(v);
  v += dppd<kXor2>(v);
  v += dppd<kHalfMirror>(v);
  return v + dppd<kMirror>(v);
}

// The sum of a wave's 64 lanes, in all of them: rows of 16 by exchanges, then the
// first row's sum to the second and the third's to the fourth, and the second's to
// the fourth, whose last lane has it all: 7 instructions.
__device__ __forceinline__ float wave_total(float v) {
  v = sum16(v);
  auto from = [](float x, auto row, auto mask) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
        0, __builtin_bit_cast(int, x), decltype(row)::value, decltype(mask)::value, 0xF, false));
  };
  v += from(v, std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{});
  v += from(v, std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xC>{});
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// 1 / sqrt(v): the estimate, one unit off, and one step of Newton's method; small
// values are scaled into the range of normal ones.
__device__ __forceinline__ float inv_root(float v) {
  const bool tiny = v < 0x1p-100f;
  v = tiny ? v * 0x1p100f : v;
  float y = __builtin_amdgcn_rsqf(v);
  const float e = __builtin_fmaf(-v * y, y, 1.0f);
  if (v > 0.0f && v < __builtin_inff()) y = __builtin_fmaf(0.5f * y, e, y);
  return tiny ? y * 0x1p50f : y;
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
template <typename T, int NC, bool ONE>
__device__ __forceinline__ void wave_moments(const float (&v)[NC][kVec<T>], int32_t cols,
                                             const Where<T, NC, ONE>& at, const Share& part,
                                             double& mean, double& squares) {
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
    m = quotient(wave_total(s), (float)part.n, (float)part.inv);
  }
  float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    // lanes that hold none of the row, and elements past its end, add nothing
    const int32_t col = at.col(c);
    const float mc = col < cols ? m : 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float t = v[c][j] - mc;
      if (cols % V != 0) t = col + j < cols ? t : 0.0f;
      if constexpr (V == 8) s1 += t;
      s2 = __builtin_fmaf(t, t, s2);
    }
  }
  squares = (double)wave_total(s2);
  if constexpr (V == 8) {
    const double d = (double)wave_total(s1);
    mean = __builtin_fma(d, part.inv, (double)m);
    squares = __builtin_fma(-d * part.inv, d, squares);
  }
}

// Rows to their normalised form in place; the reciprocal of the spread.  The
// waves' squares are moved to the row's mean, n_w (mean_w - mean)^2 for each, so
// that one meeting serves mean and spread; their means are taken as differences
// from the first wave's.  n: the columns of the wave whose values the lane takes.
template <typename T, int NC, bool ONE>
__device__ __forceinline__ float normalise(float (&v)[NC][kVec<T>], int32_t cols,
                                           const Where<T, NC, ONE>& at, int kind, float eta,
                                           const Share& row, const Share& part, float n,
                                           Meet<double> (*lds)[16], int& half) {
  constexpr int V = kVec<T>;
  double squares;
  float mu = 0.0f, off = 0.0f;
  if (kind == kNormLayer) {
    double mean;
    wave_moments(v, cols, at, part, mean, squares);
    if constexpr (!ONE) {
      const Meet<double> m = meet(mean, squares, at, lds, half);
      const double from = lane_of(m[0], 0);
      float apart;
      if constexpr (V == 4) {
        const double d = m[0] - from;
        const double moved = quotient(sum16((double)n * d), row.n, row.inv);
        mean = from + moved;
        apart = (float)(d - moved);
      } else {  // the waves' sums are binary32's already
        const float inv = (float)row.inv, d = (float)(m[0] - from), moved = sum16(n * d) * inv;
        apart = d - moved;
        mean = from + ((double)moved + (double)(sum16(n * apart) * inv));
      }
      squares = (double)sum16(__builtin_fmaf(n * apart, apart, (float)m[1]));
    }
    mu = (float)mean;
    off = (float)(mean - (double)mu);
  } else {
    float s2 = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < V; ++j) s2 = __builtin_fmaf(v[c][j], v[c][j], s2);
    s2 = wave_total(s2);
    squares = (double)s2;
    if constexpr (!ONE) squares = (double)sum16((float)meet(0.0, squares, at, lds, half)[1]);
  }
  // the squares around the mean are a difference and, for equal values, may be less than 0
  const float var = (float)(squares * row.inv), rs = inv_root((var < 0.0f ? 0.0f : var) + eta);
  if (kind == kNormLayer) {
    const float low = -off * rs;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
      for (int j = 0; j < V; ++j) v[c][j] = __builtin_fmaf(v[c][j] - mu, rs, low);
      if (cols != at.waves * kWaveCols<T, NC>) {  // 0 stays past the row's end
        const int32_t col = at.col(c);
#pragma unroll
        for (int j = 0; j < V; ++j) v[c][j] = col + j < cols ? v[c][j] : 0.0f;
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < V; ++j) v[c][j] *= rs;
    // 0 stays past the row's end also where rs is infinite or NaN: where all of such a
    // branch is dropped, the norm of r would take it in
    if (!(rs < __builtin_inff())) {
#pragma unroll
      for (int c = 0; c < NC; ++c) clear_past(v[c], at.col(c), cols);
    }
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
template <typename T, int NC, bool ONE>
struct Params {
  static constexpr int V = kVec<T>;
  static constexpr bool kHold = NC * V <= 8;
  const float* p;
  float other;
  float held[kHold ? NC : 1][V];

  __device__ __forceinline__ void read(int32_t col, int32_t cols, float (&v)[V]) const {
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
  __device__ __forceinline__ Params(const float* from, float without, int32_t cols,
                                    const Where<T, NC, ONE>& at)
      : p(from), other(without) {
    if constexpr (kHold) {
#pragma unroll
      for (int c = 0; c < NC; ++c) read(at.col(c), cols, held[c]);
    }
  }
  __device__ __forceinline__ void get(int c, int32_t col, int32_t cols,
                                      float (&v)[V]) const {
    if constexpr (kHold) {
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = held[c][j];
    } else {
      read(col, cols, v);
    }
  }
};

// Waves per SIMD asked of the compiler.  A row of 16 columns a lane has 16 waves
// in a block, so four to a SIMD too; its loads are not a row ahead, which spilled.
constexpr int kWaves = 4;
template <typename T, int NC>
constexpr bool kAhead = NC * kVec<T> <= 8;

template <typename T, int NC, bool ONE>
__global__ __launch_bounds__(1024, kWaves) void k_join_fwd(JoinFwd args) {
  JoinFwd a = arguments(args);
  constexpr int V = kVec<T>;
  __shared__ Meet<double> lds[2][16];
  int half = 0;
  const int32_t cols = a.cols, groups = (cols + kAct8Group - 1) / kAct8Group;
  const Where<T, NC, ONE> at(cols);
  const int32_t R = block_rows<false>(at.waves);
  const int64_t rows = a.rows, stride = (int64_t)gridDim.x * R;
  const bool first_lane = at.at == 0;
  const RngKey key = load_key(a.drop);
  int64_t r = (int64_t)blockIdx.x * R + at.row;
  constexpr bool A = kAhead<T, NC>;  // each loaded anew once the row before is taken out of it
  lu4 nx[NC], nb[NC];
  auto load = [&](const void* from, int64_t ld, int64_t row, lu4 (&to)[NC]) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
      to[c] = load_raw(global(static_cast<const T*>(from)) + row * ld, at.col(c), cols);
  };
  if (A && r < a.rows) {
    load(a.x, a.ldx, r, nx);
    if (a.b) load(a.b, a.ldb, r, nb);
  }
  const Params<T, NC, ONE> gate(global(a.gate), 1.0f, cols, at),
      gb(global(a.gamma_b), 1.0f, cols, at), bb(global(a.beta_b), 0.0f, cols, at),
      ga(global(a.gamma), 1.0f, cols, at), be(global(a.beta), 0.0f, cols, at);
  const Share row = share_of(cols),
              part = share_of(at.part(at.wave, cols));
  const int32_t other = (int32_t)threadIdx.x & 15;
  const float n = other < at.waves ? (float)at.part(other, cols) : 0.0f;
  // the rows of a block go round together: its waves meet at the sums' barriers
  for (int64_t r0 = (int64_t)blockIdx.x * R; r0 < rows; r0 += stride, r += stride) {
    const bool in = r < rows, more = r + stride < rows;
    a = arguments(args);
    const lu4 none = {0u, 0u, 0u, 0u};
    float v[NC][V];
    if (!A && a.b && in) load(a.b, a.ldb, r, nb);
#pragma unroll
    for (int c = 0; c < NC; ++c)
      unpack_row<T>(in && a.b ? nb[c] : none, at.col(c), cols, v[c]);
    if (A && a.b && more) load(a.b, a.ldb, r + stride, nb);
    if (a.b) {
      if (a.gamma_b) {
        const float rs = normalise(v, cols, at, a.kind, a.eta, row, part, n, lds, half);
        if (in && first_lane) global(a.rstd_b)[r] = rs;
      }
      if (a.qb && in) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
          keep<T>(v[c], global(a.qb), global(a.eb), r, groups, at.col(c));
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float f[V], o[V];
        if (a.gamma_b) {
          gb.get(c, at.col(c), cols, f);
          bb.get(c, at.col(c), cols, o);
#pragma unroll
          for (int j = 0; j < V; ++j) v[c][j] = __builtin_fmaf(v[c][j], f[j], o[j]);
        }
        if (a.drop.threshold) drop<V>(a.drop, key, r, (cols + 7) / 8, at.col(c), v[c]);
        if (a.gate) {
          gate.get(c, at.col(c), cols, f);
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
      unpack_row<T>(in ? nx[c] : none, at.col(c), cols, x);
#pragma unroll
      for (int j = 0; j < V; ++j) v[c][j] = __builtin_fmaf(a.alpha, x[j], v[c][j]);
    }
    if (A && more) load(a.x, a.ldx, r + stride, nx);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int32_t col = at.col(c);
      if (a.r && in && col < cols)
        store_row(global(static_cast<T*>(a.r)) + r * a.ldr, col, cols, v[c]);
    }
    a = arguments(args);
    if (!a.gamma) continue;
    const float rs = normalise(v, cols, at, a.kind, a.eta, row, part, n, lds, half);
    if (!in) continue;
    if (first_lane) global(a.rstd)[r] = rs;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int32_t col = at.col(c);
      if (a.q) keep<T>(v[c], global(a.q), global(a.e), r, groups, col);
      float f[V], o[V];
      ga.get(c, at.col(c), cols, f);
      be.get(c, at.col(c), cols, o);
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

template <typename T, int NC, bool ONE>
__device__ __forceinline__ void load_upper(const JoinBwd& a, const Where<T, NC, ONE>& at,
                                           int64_t r, BwdRow<NC>& w) {
  if (!a.dz) return;
  const int32_t groups = (a.cols + kAct8Group - 1) / kAct8Group;
  w.rs = global(a.rstd)[r];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int32_t col = at.col(c);
    w.dz[c] = load_raw(global(static_cast<const T*>(a.dz)) + r * a.lddz, col, a.cols);
    load_kept<T>(global(a.q), global(a.e), r, groups, col, a.cols, w.q[c], w.e[c]);
  }
}

template <typename T, int NC, bool ONE>
__device__ __forceinline__ void load_lower(const JoinBwd& a, const Where<T, NC, ONE>& at,
                                           int64_t r, BwdRow<NC>& w) {
  const int32_t groups = (a.cols + kAct8Group - 1) / kAct8Group;
  if (a.gamma_b) w.rsb = global(a.rstd_b)[r];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int32_t col = at.col(c);
    if (a.dr) w.dr[c] = load_raw(global(static_cast<const T*>(a.dr)) + r * a.lddr, col, a.cols);
    if (a.qb) load_kept<T>(global(a.qb), global(a.eb), r, groups, col, a.cols, w.qb[c], w.eb[c]);
  }
}

// The norm's input gradient from that of its normalised rows, in place, and what it
// leaves past the row's end.  That reaches no result: the sums of the branch there
// are not stored, and the parameters, 0 there, keep it out of the next row sums, if
// it is finite.
template <typename T, int NC, bool ONE>
__device__ __forceinline__ float through(float (&d)[NC][kVec<T>], const float (&h)[NC][kVec<T>],
                                         float rs, const Share& row, const Where<T, NC, ONE>& at,
                                         int kind, Meet<float> (*lds)[16], int& half) {
  constexpr int V = kVec<T>;
  float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      s1 += d[c][j];
      s2 = __builtin_fmaf(d[c][j], h[c][j], s2);
    }
  s1 = wave_total(s1);
  s2 = wave_total(s2);
  if constexpr (!ONE) {
    const Meet<float> m = meet(s1, s2, at, lds, half);
    s1 = sum16(((int32_t)threadIdx.x & 15) < at.waves ? m[0] : 0.0f);
    s2 = sum16(m[1]);
  }
  const float n = (float)row.n, inv = (float)row.inv;
  const float m1 = kind == kNormLayer ? -rs * quotient(s1, n, inv) : 0.0f;
  const float m2 = -quotient(s2, n, inv);
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < V; ++j)
      d[c][j] = __builtin_fmaf(__builtin_fmaf(m2, h[c][j], d[c][j]), rs, m1);
  return __builtin_fmaf(m2 * 0.0f, rs, m1);
}

template <typename T, int NC, bool ONE>
__global__ __launch_bounds__(1024, kWaves) void k_join_bwd(JoinBwd args) {
  JoinBwd a = arguments(args);
  constexpr int V = kVec<T>;
  __shared__ Meet<float> lds[2][16];
  int half = 0;
  const int32_t cols = a.cols, worker = blockIdx.y;
  const Where<T, NC, ONE> at(cols);
  const int32_t R = block_rows<true>(at.waves);
  const int64_t rows = a.rows, base = worker * rows, stride = (int64_t)gridDim.x * R;
  const RngKey key = load_key(a.drop);
  int64_t i = (int64_t)blockIdx.x * R + at.row;
  constexpr bool A = kAhead<T, NC>;
  BwdRow<NC> next;
  if (A && i < rows) {
    load_upper(a, at, base + i, next);
    load_lower(a, at, base + i, next);
  }
  const Params<T, NC, ONE> ga(global(a.gamma), 1.0f, cols, at),
      gate(global(a.gate), 1.0f, cols, at), gb(global(a.gamma_b), 1.0f, cols, at);
  const Share row = share_of(cols);
  // At 16 columns a lane registers do not hold four sums (8 x 256 of 16384: 349 us,
  // spilled, against 168): the branch's two lie in LDS, each lane's in its own place.
  constexpr bool kLow = NC * V > 8;
  constexpr int S = kLow ? 2 : 4;
  using Low = float __attribute__((ext_vector_type(4)));
  __shared__ Low low[kLow ? 2 : 1][kLow ? NC * V / 4 : 1][kLow ? 1024 : 1];
  float sums[S][NC][V];
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < V; ++j) sums[s][c][j] = 0.0f;
  if constexpr (kLow) {
    for (int s = 0; s < 2; ++s)
      for (int i = 0; i < NC * V / 4; ++i) low[s][i][threadIdx.x] = Low{0.0f, 0.0f, 0.0f, 0.0f};
  }
  for (int64_t i0 = (int64_t)blockIdx.x * R; i0 < rows; i0 += stride, i += stride) {
    const bool in = i < rows, more = i + stride < rows;
    const int64_t r = base + i;
    const lu4 none = {0u, 0u, 0u, 0u};
    float d[NC][V], past = 0.0f;
    a = arguments(args);
    if (!A && in) load_upper(a, at, r, next);
    if (a.dz) {
      float h[NC][V];
      const float rs = in ? next.rs : 0.0f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        unpack_row<T>(in ? next.dz[c] : none, at.col(c), cols, d[c]);
        decode<T>(in, next.q[c], next.e[c], h[c]);
      }
      if (A && more) load_upper(a, at, r + stride, next);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float f[V];
        ga.get(c, at.col(c), cols, f);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          sums[0][c][j] = __builtin_fmaf(d[c][j], h[c][j], sums[0][c][j]);
          sums[1][c][j] += d[c][j];
          d[c][j] *= f[j];
        }
      }
      past = through(d, h, rs, row, at, a.kind, lds, half);
    } else {
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < V; ++j) d[c][j] = 0.0f;
    }
    a = arguments(args);
    if (!A && in) load_lower(a, at, r, next);
    float k[NC][V];
    const float rsb = in ? next.rsb : 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (a.dr) {
        float o[V];
        unpack_row<T>(in ? next.dr[c] : none, at.col(c), cols, o);
#pragma unroll
        for (int j = 0; j < V; ++j) d[c][j] += o[j];
      }
      decode<T>(in && a.qb, next.qb[c], next.eb[c], k[c]);
    }
    if (A && more) load_lower(a, at, r + stride, next);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int32_t col = at.col(c);
      float o[V];
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] = a.alpha * d[c][j];
      if (in && col < cols) store_row(global(static_cast<T*>(a.dx)) + r * a.lddx, col, cols, o);
      // 0 times a parameter's 0 is no 0 for an infinity or a NaN, and where the row's own
      // are dropped, the branch's gradient is 0 (chunk by chunk here: for the whole row
      // behind the sums it spilled, 9000 binary32 columns 137 -> 164 us)
      if (!(__builtin_fabsf(past) < __builtin_inff())) clear_past(d[c], col, cols);
      if (a.drop.threshold) drop<V>(a.drop, key, r, (cols + 7) / 8, col, d[c]);
      if constexpr (kLow) {
#pragma unroll
        for (int j = 0; j < V; j += 4) {
          Low s = low[0][(c * V + j) / 4][threadIdx.x], t = low[1][(c * V + j) / 4][threadIdx.x];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[i] = __builtin_fmaf(d[c][j + i], k[c][j + i], s[i]);
            t[i] += d[c][j + i];
          }
          low[0][(c * V + j) / 4][threadIdx.x] = s;
          low[1][(c * V + j) / 4][threadIdx.x] = t;
        }
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          sums[2][c][j] = __builtin_fmaf(d[c][j], k[c][j], sums[2][c][j]);
          sums[3][c][j] += d[c][j];
        }
      }
      if (a.gate) {
        gate.get(c, at.col(c), cols, o);
#pragma unroll
        for (int j = 0; j < V; ++j) d[c][j] *= o[j];
      }
      if (a.gamma_b) {
        gb.get(c, at.col(c), cols, o);
#pragma unroll
        for (int j = 0; j < V; ++j) d[c][j] *= o[j];
      }
    }
    if (!a.db) continue;
    if (a.gamma_b) through(d, k, rsb, row, at, a.kind, lds, half);
    if (!in) continue;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int32_t col = at.col(c);
      if (col < cols) store_row(global(static_cast<T*>(a.db)) + r * a.lddb, col, cols, d[c]);
    }
  }
  // the block's column sums: its rows' in order
  if (!a.part) return;
  using Four4 = float __attribute__((ext_vector_type(4)));
  const int64_t pc = join_part_cols(cols);
  float* part = global(a.part) + ((int64_t)worker * gridDim.x + blockIdx.x) * 4 * pc;
  if constexpr (!kLow) {
    __shared__ Four4 all[2][16 * kWaveCols<T, NC> / 4];
    if (R > 1) {
      const int32_t row_cols = at.waves * kWaveCols<T, NC>;
#pragma unroll
      for (int s = 0; s < 4; s += 2) {  // the norm's two, then the branch's
        if (s) __syncthreads();
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < V; j += 4) {
              const float(&v)[V] = sums[s + t][c];
              all[t][(at.row * row_cols + at.col(c) + j) / 4] =
                  Four4{v[j], v[j + 1], v[j + 2], v[j + 3]};
            }
        __syncthreads();
        for (int32_t i = threadIdx.x; i < row_cols / 2; i += blockDim.x) {
          const int32_t t = i / (row_cols / 4), four = i % (row_cols / 4);
          Four4 v = all[t][four];
          for (int32_t g = 1; g < R; ++g) v += all[t][g * (row_cols / 4) + four];
          if (four * 4 < cols) *reinterpret_cast<Four4*>(part + (s + t) * pc + four * 4) = v;
        }
      }
      return;
    }
  }
#pragma unroll
  for (int s = 0; s < 4; ++s)
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        Four4 v;
        if (kLow && s >= 2) {
          v = low[s & 1][kLow ? (c * V + j) / 4 : 0][kLow ? threadIdx.x : 0];
        } else {
          const float(&w)[V] = sums[kLow ? s & 1 : s][c];
          v = Four4{w[j], w[j + 1], w[j + 2], w[j + 3]};
        }
        const int32_t col = at.col(c) + j;
        if (col < cols) *reinterpret_cast<Four4*>(part + s * pc + col) = v;
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
  const int64_t cols = a.cols, pc = join_part_cols(cols), worker = blockIdx.y;
  const float* p = a.part + (worker * blocks * 4 + blockIdx.z * 2) * pc + col;
  double s = 0.0, t = 0.0;
  if (col < cols) {
#pragma unroll 4
    for (int32_t b = w; b < blocks; b += kJoinWaves) {
      s += p[(int64_t)b * 4 * pc];
      t += p[((int64_t)b * 4 + 1) * pc];
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
// One round of resident blocks and no more than there are rows for: 16 waves to a
// CU, which their registers allow; 20 forward of 16-bit rows, where blocks of up to
// four waves fill the four SIMDs evenly (32768 x 1024 84 -> 79 us, 30203 x 1111 120 ->
// 113; but 5 waves to a row 93 -> 116).
constexpr int64_t kCus = 256, kCuWaves = 16, kCuWaves16 = 20;

struct Shape {
  int32_t waves, rows;  // to a row, and rows to a block
  int64_t resident;
};
template <bool BACK>
Shape shape_of(int32_t cols, bool two_bytes = false) {
  const int32_t wave = cols <= 16 * 512 ? 512 : 1024;
  Shape s;
  s.waves = (cols + wave - 1) / wave;
  s.rows = block_rows<BACK>(s.waves);
  const int64_t all = !BACK && two_bytes && s.waves <= 4 ? kCuWaves16 : kCuWaves;
  s.resident = kCus * (all / (s.waves * s.rows));
  return s;
}

// The instance that holds a row: 8 columns a lane, 16 above 8192 columns.
// Binary32 rows take twice the pieces (M).
template <typename T, class F>
void pick(int32_t cols, F&& f) {
  constexpr int M = 8 / kVec<T>;
  if (cols <= 512) f(std::integral_constant<int, M>{}, std::true_type{});
  else if (cols <= 16 * 512) f(std::integral_constant<int, M>{}, std::false_type{});
  else f(std::integral_constant<int, 2 * M>{}, std::false_type{});
}

template <typename T>
void fwd(const JoinFwd& a, hipStream_t st) {
  const Shape s = shape_of<false>(a.cols, sizeof(T) == 2);
  const int64_t blocks = std::min((a.rows + s.rows - 1) / s.rows, s.resident);
  pick<T>(a.cols, [&](auto nc, auto one) {
    hipLaunchKernelGGL(HIP_KERNEL_NAME(k_join_fwd<T, nc.value, one.value>), dim3((uint32_t)blocks),
                       dim3(s.waves * s.rows * 64), 0, st, a);
  });
}

template <typename T>
void bwd(const JoinBwd& a, hipStream_t st) {
  const Shape s = shape_of<true>(a.cols);
  pick<T>(a.cols, [&](auto nc, auto one) {
    hipLaunchKernelGGL(HIP_KERNEL_NAME(k_join_bwd<T, nc.value, one.value>),
                       dim3(join_bwd_blocks(a.n, a.rows, a.cols), a.n),
                       dim3(s.waves * s.rows * 64), 0, st, a);
  });
}

template <typename G>
void wgrad(const JoinBwd& a, hipStream_t st) {
  const int32_t blocks = a.rows ? join_bwd_blocks(a.n, a.rows, a.cols) : 0;
  hipLaunchKernelGGL(HIP_KERNEL_NAME(k_join_wgrad<G>), dim3((a.cols + 63) / 64, a.n, 2),
                     dim3(kJoinWaves * 64), 0, st, a, blocks);
}

}  // namespace

int32_t join_bwd_blocks(int32_t n, int64_t rows, int32_t cols) {
  const Shape s = shape_of<true>(cols);
  const int64_t most = std::max<int64_t>(1, s.resident / n), want = (rows + s.rows - 1) / s.rows;
  if (want <= most) return (int32_t)std::max<int64_t>(1, want);
  const int64_t rounds = (want + most - 1) / most;  // no more blocks than these need
  return (int32_t)((want + rounds - 1) / rounds);
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
