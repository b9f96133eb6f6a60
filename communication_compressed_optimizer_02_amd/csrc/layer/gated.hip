// gated.hip -- the products of a gated feed-forward block on the matrix cores
// (gfx950), the gate in their epilogue.
//
//   forward      p = x wg^T + bg, u = x wu^T + bu, y = f(p) * u
//   hidden grad  d = dy w, dp = d * u * f'(p), du = d * f(p)
//
// Forward, a tile holds the same columns of p and u, so that both meet in one
// wave and neither goes to memory as 16 bits: p, u and y are kept in 8 bits where
// the backward pass needs them.  Backward, p and u are read from 8 bits.
// Operands and layouts are those of tile.hpp.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "gate.hpp"
#include "layer.hpp"
#include "sublayer_kernels.hpp"
#include "tile.hpp"

namespace oba {

namespace {

constexpr int kMaxSplits = 8;

struct Tiles {
  int32_t ta, tb;    // tiles along the hidden columns and the rows
  int32_t splits;
  int32_t ksteps;    // steps of kBK of one split
};

__device__ __forceinline__ int32_t groups_of(int32_t cols) {
  return (cols + kAct8Group - 1) / kAct8Group;
}

// Eight columns from c of row r to 8 bits; four neighbouring lanes hold a group,
// those past the last column 0.
__device__ __forceinline__ void keep8(const float (&v)[8], bool in_rows, int64_t r, int32_t c,
                                      int32_t cols, int8_t* q, uint8_t* e) {
  const uint32_t top = max_lanes<4>(magnitude8(v));
  const uint32_t ex = group_exp(top);
  const float inv = inv_step_of(ex), step = step_of(ex);
  const int32_t groups = groups_of(cols);
  if (in_rows && c / kAct8Group < groups) {
    const int64_t g = r * groups + c / kAct8Group;
    *reinterpret_cast<lu2*>(q + g * kAct8Group + c % kAct8Group) =
        lu2{quant4(v, inv, step, ex != 255u), quant4(v + 4, inv, step, ex != 255u)};
    if (c % kAct8Group == 0) e[g] = (uint8_t)ex;
  }
}

__device__ __forceinline__ void load_bias(const Gated& a, int32_t c, float (&bp)[8],
                                          float (&bu)[8]) {
  for (int j = 0; j < 8; ++j) {
    const bool in = a.bias && c + j < a.cols;
    bp[j] = in ? a.bias[c + j] : 0.0f;
    bu[j] = in ? a.bias[a.cols + c + j] : 0.0f;
  }
}

// Forward results of eight columns from both products.
template <typename T>
__device__ __forceinline__ void finish_forward(const Gated& a, int64_t r, int32_t c,
                                               const float (&bp)[8], const float (&bu)[8],
                                               float (&p)[8], float (&u)[8]) {
  const int n = a.cols - c;
  const bool in_rows = r < a.rows;
  for (int j = 0; j < 8; ++j) {
    p[j] = j < n ? p[j] + bp[j] : 0.0f;
    u[j] = j < n ? u[j] + bu[j] : 0.0f;
  }
  if (a.qp) {
    keep8(p, in_rows, r, c, a.cols, a.qp, a.ep);
    keep8(u, in_rows, r, c, a.cols, a.qu, a.eu);
  }
  gate_value(p, a.gate);
  for (int j = 0; j < 8; ++j) p[j] *= u[j];
  if (a.q) {  // as rounded: what reading y and encoding it would give
    const lu4 w = pack(p, (const T*)nullptr);
    float y[8];
    unpack(w, y, (const T*)nullptr);
    if (n < 8)
      for (int j = 0; j < 8; ++j) y[j] = j < n ? y[j] : 0.0f;
    keep8(y, in_rows, r, c, a.cols, a.q, a.e);
  }
  if (in_rows && n > 0) store8(static_cast<T*>(a.c) + r * a.ldc + c, n, p);
}

// Eight kept pre-activations of each kind.
struct Kept {
  lu2 p, u;
  uint32_t ep, eu;
};
__device__ __forceinline__ void load_kept(const Gated& a, int64_t r, int32_t c, Kept& k) {
  if (r >= a.rows || c >= a.cols) return;
  const int64_t g = r * groups_of(a.cols) + c / kAct8Group;
  k.p = *reinterpret_cast<const lu2*>(a.qp + g * kAct8Group + c % kAct8Group);
  k.u = *reinterpret_cast<const lu2*>(a.qu + g * kAct8Group + c % kAct8Group);
  k.ep = a.ep[g];
  k.eu = a.eu[g];
}

template <typename T>
__device__ __forceinline__ void finish_grad(const Gated& a, int64_t r, int32_t c, const Kept& k,
                                            const float (&d)[8]) {
  const int n = a.cols - c;
  if (r >= a.rows || n <= 0) return;
  const float sp = step_of(k.ep), su = step_of(k.eu);
  float f[8], df[8];
  for (int j = 0; j < 8; ++j) f[j] = dequant(k.p[j / 4], j % 4, sp);
  gate_both(f, df, a.gate);
  for (int j = 0; j < 8; ++j) {
    df[j] *= d[j] * dequant(k.u[j / 4], j % 4, su);
    f[j] *= d[j];
  }
  T* row = static_cast<T*>(a.c) + r * a.ldc;
  store8(row + c, n, df);
  if (a.cols % 8 == 0) {
    store8(row + a.cols + c, n, f);
  } else {  // the second half begins inside a vector
    for (int j = 0; j < 8; ++j)
      if (j < n) row[a.cols + c + j] = (T)f[j];
  }
}

// Partial sums of a split product: [split][rows][halves][cols8].
__device__ __forceinline__ int64_t part_cols(const Gated& a) { return (a.cols + 7) / 8 * 8; }

template <typename T, GatedKind KIND, int BA, int BB, int WA, int WB>
__global__ __launch_bounds__(WA* WB * 64, 3) void k_gated(Gated a, Tiles t) {
  constexpr int NT = WA * WB * 64;
  constexpr bool FWD = KIND == GatedKind::kForward;
  constexpr int ASRC = FWD ? kKRow : kKCol;
  constexpr int HC = FWD ? BA / 2 : BA;  // hidden columns of a tile
  constexpr int TA = BA / WA / 16, TB = BB / WB / 16;
  constexpr int kA = BA * kBK * 2, kStageBytes = kA + BB * kBK * 2;  // of a step in LDS
  __shared__ __align__(1024) char lds[kStageBytes];

  const int64_t work = xcd_order(blockIdx.x, gridDim.x);
  const int32_t tiles = t.ta * t.tb;
  const int32_t tile = (int32_t)(work % tiles), split = (int32_t)(work / tiles);
  // four rows of tiles together, along the columns: the tiles that run at one
  // time share operands of both sides
  const int32_t super = tile / (4 * t.ta), in = tile - super * 4 * t.ta;
  const int32_t high = min(4, t.tb - super * 4);
  const int32_t r0 = (super * 4 + in % high) * BB, c0 = in / high * HC;

  const int64_t kbeg = (int64_t)split * t.ksteps * kBK;
  const int64_t kend = min(a.k, kbeg + (int64_t)t.ksteps * kBK);
  // forward: half a tile's rows from the gate's weights, half from the others'
  const char *ap, *ap2;
  int64_t astep;
  if constexpr (FWD) {
    ap = static_cast<const char*>(a.a) + ((int64_t)c0 * a.lda + kbeg) * 2;
    ap2 = ap + (int64_t)a.cols * a.lda * 2;
    astep = kBK * 2;
  } else {
    ap = static_cast<const char*>(a.a) + (kbeg * a.lda + c0) * 2;
    ap2 = ap;
    astep = kBK * a.lda * 2;
  }
  const char* bp = static_cast<const char*>(a.b) + ((int64_t)r0 * a.ldb + kbeg) * 2;

  // the operand's parts have the same offsets from their origins
  Stage<T, ASRC, HC, NT> sa;
  Stage<T, kKRow, BB, NT> sb;
  sa.init(c0, a.cols, (uint32_t)a.lda, 0);
  sb.init(r0, (int32_t)min(a.rows, (int64_t)0x7FFFFFFF), (uint32_t)a.ldb, 0);

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // uniform
  const int wa = wave % WA, wb = wave / WA;
  lf4 acc[TA][TB];
#pragma unroll
  for (int i = 0; i < TA; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j) acc[i][j] = lf4{0.0f, 0.0f, 0.0f, 0.0f};

  // the direct loads of a wave have landed in LDS (a barrier alone does not
  // wait for them)
  auto landed = [] { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); };
  auto compute = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int ks = 0; ks < kBK / 32; ++ks) {
      lu4 fa[TA], fb[TB];
#pragma unroll
      for (int i = 0; i < TA; ++i) {
        if constexpr (FWD)  // the first half of a wave's tiles are p's, the others u's
          fa[i] = fragment<kKRow, HC>(lds + (i < TA / 2 ? 0 : kA / 2),
                                      (wa * (TA / 2) + i % (TA / 2)) * 16, ks);
        else
          fa[i] = fragment<kKCol, HC>(lds, (wa * TA + i) * 16, ks);
      }
#pragma unroll
      for (int j = 0; j < TB; ++j) fb[j] = fragment<kKRow, BB>(lds + kA, (wb * TB + j) * 16, ks);
#pragma unroll
      for (int j = 0; j < TB; ++j)
#pragma unroll
        for (int i = 0; i < TA; ++i) acc[i][j] = mfma(fa[i], fb[j], acc[i][j], (const T*)nullptr);
    }
  };
  const int32_t full = (int32_t)((kend - kbeg) / kBK), rest = (int32_t)((kend - kbeg) % kBK);
  for (int32_t s = 0; s < full; ++s) {
    if (s > 0) __syncthreads();  // every wave is done with the last step's tile
    sa.direct(ap, lds);
    if constexpr (FWD) sa.direct(ap2, lds + kA / 2);
    sb.direct(bp, lds + kA);
    ap += astep;
    ap2 += astep;
    bp += kBK * 2;
    landed();
    __syncthreads();
    compute();
  }
  if (rest > 0) {
    if (full > 0) __syncthreads();
    sa.tail(ap, lds, rest);
    if constexpr (FWD) sa.tail(ap2, lds + kA / 2, rest);
    sb.tail(bp, lds + kA, rest);
    __syncthreads();
    compute();
  }

  // The results go through LDS, 16 rows of a wave at a time and within the
  // wave alone: lane l holds row l % 16 and four columns of each tile, and
  // takes back eight consecutive columns (forward, of both halves).
  constexpr int kRow = TA * 16 + 4;         // floats of a row in LDS, off the bank period
  constexpr int kCols = HC / WA;            // hidden columns of a wave
  constexpr int kLanes = kCols / 8;         // lanes of a row
  constexpr int kIter = 16 * kLanes / 64;
  static_assert(WA * WB * 16 * kRow * 4 <= kStageBytes, "epilogue rows fit the tile");
  static_assert(kIter >= 1 && kCols % kAct8Group == 0, "whole groups to a wave");
  const int l = threadIdx.x & 63;
  float* rows = reinterpret_cast<float*>(lds) + wave * 16 * kRow;
  const int64_t pc = part_cols(a);
  constexpr int kHalves = FWD ? 2 : 1;
  __syncthreads();  // every wave has read its last fragments
  const int rr = l / kLanes, cc = l % kLanes * 8;  // the lane's first row, and its columns
  const int32_t c = c0 + wa * kCols + cc;
  float bgate[8], blin[8];
  if constexpr (FWD) load_bias(a, c, bgate, blin);
#pragma unroll 1
  for (int j = 0; j < TB; ++j) {
    const int64_t rj = r0 + (wb * TB + j) * 16;
    Kept kept[kIter];
    if constexpr (!FWD) {
      if (t.splits == 1) {
#pragma unroll
        for (int i = 0; i < kIter; ++i) load_kept(a, rj + rr + i * (64 / kLanes), c, kept[i]);
      }
    }
#pragma unroll
    for (int jj = 0; jj < TB; ++jj) {
      if (jj != j) continue;  // a constant index into the accumulators
#pragma unroll
      for (int i = 0; i < TA; ++i)
        *reinterpret_cast<lf4*>(rows + (l & 15) * kRow + i * 16 + (l >> 4) * 4) = acc[i][jj];
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int ri = rr + i * (64 / kLanes);
      const int64_t r = rj + ri;
      float v[kHalves][8];
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const lf4* x = reinterpret_cast<const lf4*>(rows + ri * kRow + h * kCols + cc);
        const lf4 lo = x[0], hi = x[1];
        for (int m = 0; m < 4; ++m) {
          v[h][m] = lo[m];
          v[h][4 + m] = hi[m];
        }
        if (t.splits > 1 && r < a.rows && c < a.cols) {
          lf4* to = reinterpret_cast<lf4*>(
              a.part + (((int64_t)split * a.rows + r) * kHalves + h) * pc + c);
          to[0] = lo;
          to[1] = hi;
        }
      }
      if (t.splits == 1) {
        if constexpr (FWD) finish_forward<T>(a, r, c, bgate, blin, v[0], v[1]);
        else finish_grad<T>(a, r, c, kept[i], v[0]);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

// ---- joining a split product ------------------------------------------------------
// A thread adds eight columns' sums in split order and finishes them as above;
// four lanes hold a group of 32 columns.
template <typename T, GatedKind KIND>
__global__ __launch_bounds__(256) void k_gated_join(Gated a, int32_t splits) {
  constexpr int kHalves = KIND == GatedKind::kForward ? 2 : 1;
  const int32_t per_row = groups_of(a.cols) * 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t r = i / per_row;
  const int32_t c = (int32_t)(i - r * per_row) * 8;
  const int64_t pc = part_cols(a);
  if (r >= a.rows) return;  // whole groups of lanes
  float v[kHalves][8] = {};
  if (c < a.cols) {
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      lf4 x[kMaxSplits], y[kMaxSplits];
#pragma unroll
      for (int s = 0; s < kMaxSplits; ++s)  // all loads before the first sum
        if (s < splits) {
          const lf4* p = reinterpret_cast<const lf4*>(
              a.part + (((int64_t)s * a.rows + r) * kHalves + h) * pc + c);
          x[s] = p[0];
          y[s] = p[1];
        }
#pragma unroll
      for (int s = 0; s < kMaxSplits; ++s)
        if (s < splits)
          for (int j = 0; j < 4; ++j) {
            v[h][j] += x[s][j];
            v[h][4 + j] += y[s][j];
          }
    }
  }
  if constexpr (KIND == GatedKind::kForward) {
    float bp[8], bu[8];
    load_bias(a, c, bp, bu);
    finish_forward<T>(a, r, c, bp, bu, v[0], v[1]);
  } else {
    Kept k;
    load_kept(a, r, c, k);
    finish_grad<T>(a, r, c, k, v[0]);
  }
}

// ---- host side ----------------------------------------------------------------------
constexpr int kCUs = 256;
constexpr int kTile = 128;

Tiles choose(GatedKind kind, int64_t rows, int32_t cols, int64_t k) {
  const int32_t wide = kind == GatedKind::kForward ? kTile / 2 : kTile;
  Tiles t;
  t.ta = (cols + wide - 1) / wide;
  t.tb = (int32_t)((rows + kTile - 1) / kTile);
  const int64_t all = (int64_t)t.ta * t.tb, steps = (k + kBK - 1) / kBK;
  int64_t splits = 1;
  if (all > 0 && all <= kCUs) {
    const int64_t least = all <= kCUs / 2 ? 4 : 10;
    splits = std::max<int64_t>(
        1, std::min<int64_t>({2 * kCUs / all, steps / least, (int64_t)kMaxSplits}));
  }
  t.ksteps = (int32_t)std::max<int64_t>(1, (steps + splits - 1) / splits);
  t.splits = (int32_t)std::max<int64_t>(1, (steps + t.ksteps - 1) / t.ksteps);
  return t;
}

template <typename T, GatedKind KIND>
void product(const Gated& a, hipStream_t st) {
  const Tiles t = choose(KIND, a.rows, a.cols, a.k);
  const uint32_t grid = (uint32_t)gated_blocks(KIND, a.rows, a.cols, a.k);
  hipLaunchKernelGGL(HIP_KERNEL_NAME(k_gated<T, KIND, kTile, kTile, 2, 2>), dim3(grid), dim3(256),
                     0, st, a, t);
}

template <typename T, GatedKind KIND>
void join(const Gated& a, hipStream_t st) {
  const Tiles t = choose(KIND, a.rows, a.cols, a.k);
  const int64_t lanes = a.rows * ((a.cols + kAct8Group - 1) / kAct8Group) * 4;
  hipLaunchKernelGGL(HIP_KERNEL_NAME(k_gated_join<T, KIND>), dim3((uint32_t)((lanes + 255) / 256)),
                     dim3(256), 0, st, a, t.splits);
}

}  // namespace

int32_t gated_splits(GatedKind kind, int64_t rows, int32_t cols, int64_t k) {
  return choose(kind, rows, cols, k).splits;
}

int64_t gated_blocks(GatedKind kind, int64_t rows, int32_t cols, int64_t k) {
  const Tiles t = choose(kind, rows, cols, k);
  return (int64_t)t.ta * t.tb * t.splits;
}

size_t gated_workspace(GatedKind kind, int64_t rows, int32_t cols, int64_t k) {
  const int32_t s = gated_splits(kind, rows, cols, k);
  if (s <= 1) return 0;
  return (size_t)s * rows * ((size_t)(cols + 7) / 8 * 8) *
         (kind == GatedKind::kForward ? 2 : 1) * 4;
}

void launch_gated(GatedKind kind, const Gated& a, hipStream_t st) {
  if (kind == GatedKind::kForward) {
    if (a.dtype == kGradF16) product<_Float16, GatedKind::kForward>(a, st);
    else product<__bf16, GatedKind::kForward>(a, st);
  } else {
    if (a.dtype == kGradF16) product<_Float16, GatedKind::kHiddenGrad>(a, st);
    else product<__bf16, GatedKind::kHiddenGrad>(a, st);
  }
}

void launch_gated_join(GatedKind kind, const Gated& a, hipStream_t st) {
  if (kind == GatedKind::kForward) {
    if (a.dtype == kGradF16) join<_Float16, GatedKind::kForward>(a, st);
    else join<__bf16, GatedKind::kForward>(a, st);
  } else {
    if (a.dtype == kGradF16) join<_Float16, GatedKind::kHiddenGrad>(a, st);
    else join<__bf16, GatedKind::kHiddenGrad>(a, st);
  }
}

}  // namespace oba
