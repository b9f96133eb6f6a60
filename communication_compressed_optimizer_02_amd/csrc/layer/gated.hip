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
#include <type_traits>

#include "gate.hpp"
#include "layer.hpp"
#include "sublayer_kernels.hpp"
#include "tile.hpp"
#include "wide.hpp"

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

// A block to a tile, or to a part of its sum; the loads of STAGES - 1 steps ahead.
// Of 128 x 128 one stage, so that a CU's blocks hide each other's loads (3000 x 700 ->
// 2 x 1500 27 us; two to four stages, fewer blocks, 35 to 46); of 64 x 64 three (four
// and five gain nothing).
template <typename T, GatedKind KIND, int BA, int BB, int WA, int WB, int STAGES>
__global__ __launch_bounds__(WA* WB * 64, 3) void k_gated(Gated a, Tiles t) {
  constexpr int NT = WA * WB * 64;
  constexpr bool FWD = KIND == GatedKind::kForward;
  constexpr int ASRC = FWD ? kKRow : kKCol;
  constexpr int HC = FWD ? BA / 2 : BA;  // hidden columns of a tile
  constexpr int TA = BA / WA / 16, TB = BB / WB / 16;
  constexpr int kA = BA * kBK * 2, kStageBytes = kA + BB * kBK * 2;  // of a step in LDS
  __shared__ __align__(1024) char lds[STAGES * kStageBytes];

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
  AheadStage<ASRC, HC, NT> sa;
  AheadStage<kKRow, BB, NT> sb;
  sa.init(threadIdx.x, c0, a.cols, (uint32_t)a.lda);
  sb.init(threadIdx.x, r0, (int32_t)min(a.rows, (int64_t)0x7FFFFFFF), (uint32_t)a.ldb);

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // uniform
  const int wa = wave % WA, wb = wave / WA;
  lf4 acc[TA][TB];
#pragma unroll
  for (int i = 0; i < TA; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j) acc[i][j] = lf4{0.0f, 0.0f, 0.0f, 0.0f};

  auto compute = [&](const char* at) __attribute__((always_inline)) {
#pragma unroll
    for (int ks = 0; ks < kBK / 32; ++ks) {
      lu4 fa[TA], fb[TB];
#pragma unroll
      for (int i = 0; i < TA; ++i) {
        if constexpr (FWD)  // the first half of a wave's tiles are p's, the others u's
          fa[i] = fragment<kKRow, HC>(at + (i < TA / 2 ? 0 : kA / 2),
                                      (wa * (TA / 2) + i % (TA / 2)) * 16, ks);
        else
          fa[i] = fragment<kKCol, HC>(at, (wa * TA + i) * 16, ks);
      }
#pragma unroll
      for (int j = 0; j < TB; ++j) fb[j] = fragment<kKRow, BB>(at + kA, (wb * TB + j) * 16, ks);
#pragma unroll
      for (int j = 0; j < TB; ++j)
#pragma unroll
        for (int i = 0; i < TA; ++i) acc[i][j] = mfma(fa[i], fb[j], acc[i][j], (const T*)nullptr);
    }
  };
  // Step s lies in part s % STAGES of LDS.  A sum whose length is no multiple of the
  // step begins with what is left over, through registers.
  const int32_t full = (int32_t)((kend - kbeg) / kBK), rest = (int32_t)((kend - kbeg) % kBK);
  const int32_t steps = full + (rest > 0);
  auto issue = [&](int32_t s, int32_t part) __attribute__((always_inline)) {
    char* to = lds + part * kStageBytes;
    if (s == 0 && rest > 0) {
      sa.tail(threadIdx.x, ap + full * astep, to, rest);
      if constexpr (FWD) sa.tail(threadIdx.x, ap2 + full * astep, to + kA / 2, rest);
      sb.tail(threadIdx.x, bp + (int64_t)full * kBK * 2, to + kA, rest);
    } else {
      sa.ahead(wave, ap, to);
      if constexpr (FWD) sa.ahead(wave, ap2, to + kA / 2);
      sb.ahead(wave, bp, to + kA);
      ap += astep;
      ap2 += astep;
      bp += kBK * 2;
    }
  };
  constexpr int kLoads = (FWD ? 2 : 1) * decltype(sa)::P + decltype(sb)::P;  // of a step
  int32_t part = 0;
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s)
    if (s < steps) issue(s, s);
#pragma unroll 1
  for (int32_t s = 0; s < steps; ++s) {
    if constexpr (STAGES == 1) {
      if (s > 0) meet();  // every wave is done with the last step
      issue(s, 0);
      wait_loads();
      meet();
    } else {
      // step s has landed, those behind it may be on their way
      if (s + STAGES - 2 < steps) wait_loads<(STAGES - 2) * kLoads>();
      else wait_loads();
      meet();  // and every wave is done with step s - 1, whose part is free
      if (s + STAGES - 1 < steps) issue(s + STAGES - 1, part == 0 ? STAGES - 1 : part - 1);
    }
    compute(lds + part * kStageBytes);
    part = part == STAGES - 1 ? 0 : part + 1;
  }

  // The results go through LDS, 16 rows of a wave at a time and within the
  // wave alone: lane l holds row l % 16 and four columns of each tile, and
  // takes back eight consecutive columns (forward, of both halves).
  constexpr int kRow = TA * 16 + 4;         // floats of a row in LDS, off the bank period
  constexpr int kCols = HC / WA;            // hidden columns of a wave
  constexpr int kLanes = kCols / 8;         // lanes of a row
  constexpr int kIter = 16 * kLanes / 64;
  static_assert(WA * WB * 16 * kRow * 4 <= STAGES * kStageBytes, "epilogue rows fit");
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

// ---- the products of many tiles ------------------------------------------------------
// Blocks of eight waves, one to a CU, walk tiles of 256 rows by 256 rows of the
// other operand: forward 128 columns of p and of u, back 256 hidden columns.  A
// wave holds 64 hidden columns (forward of p and of u) in four tiles of 16 and 64
// or 128 rows.
//
// A step's products are in two halves of 32 along k.  The first half's fragments
// are in registers when the step begins, the second's are read under the first's
// products; then all waves meet, the step's parts of LDS take loads of later steps,
// and the next step's first fragments are read under the second half's products.
//
// The epilogue works in the registers that the products leave: a lane has four
// columns of each of four tiles, groups of 32 columns are in four lanes, and a
// transposition between the four groups of 16 lanes gives each lane 16 columns to
// store.
//
// Bound by the products, and between them by the memory: all CUs end a tile at one
// time, so its stores (and back its loads) run at 4.4 TB/s with the matrix cores
// idle.  16384 x 1024 -> 2 x 4096 bfloat16: nothing kept 231 us, all kept (340 MB)
// 283 to 312; the hidden gradient 120 us of products, 203 to 217 with its 400 MB.
// 8192 x 4096 -> 2 x 4096, nothing kept, 414 us, 1.33 PFLOP/s, the matrix cores busy
// for 70 % of the cycles.  Two blocks of half the tile to a CU, one's epilogue under
// the other's products, read half as much again from L2 and lost: 360 and 227.
__device__ __forceinline__ int32_t persistent_tile(int32_t round, int32_t tiles) {
  // each XCD (blocks are handed to the 8 in turn) walks a range of neighbouring
  // tiles, so that its L2 sees an operand's rows once
  const int32_t x = blockIdx.x & 7, i = (blockIdx.x >> 3) + round * (int32_t)(gridDim.x >> 3);
  const int32_t q = tiles / 8, r = tiles % 8, mine = q + (x < r ? 1 : 0);
  return i < mine ? x * q + min(x, r) + i : -1;
}

// 16 values of a lane (four of each of four tiles) to 8 bits, 16 bytes a lane;
// tiles 0 and 1 are one group of 32 columns, 2 and 3 the next.
__device__ __forceinline__ void keep16(const float (&v)[2][8], bool store, int64_t at_q,
                                       int64_t at_e, bool store_e, int8_t* q, uint8_t* e) {
  uint32_t w[4], ex[2], top[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    top[h] = max_groups(magnitude8(v[h]));
    ex[h] = group_exp(top[h]);
  }
  const bool held = past_range(top[0]) || past_range(top[1]);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float inv = inv_step_of(ex[h]), step = step_of(ex[h]);
    const bool finite = ex[h] != 255u;
    if (held) {
      w[2 * h] = quant4(v[h], inv, step, finite);
      w[2 * h + 1] = quant4(v[h] + 4, inv, step, finite);
    } else {
      w[2 * h] = quant4_in(v[h], inv, finite);
      w[2 * h + 1] = quant4_in(v[h] + 4, inv, finite);
    }
  }
  transpose4(w);
  if (store)
    __builtin_nontemporal_store(lu4{w[0], w[1], w[2], w[3]}, reinterpret_cast<lu4*>(q + at_q));
  // groups of 16 lanes 0 and 2 hold tiles 0 and 2
  if (store_e) e[at_e] = (uint8_t)((threadIdx.x & 32) ? ex[1] : ex[0]);
}

// 16 results of a lane (four of each of four tiles).  Exchanged between
// neighbouring groups of 16 lanes each lane has eight columns of one of the first
// two tiles and of one of the others, so that a store fills 64 bytes of a row.
// ONCE: past the caches, which hold the operands (forward, 242 -> 231 us at 16384 x
// 1024 -> 2 x 4096; the hidden gradient, with twice the bytes, lost: 212 -> 222).
template <typename T, bool ONCE>
__device__ __forceinline__ void store16(const float (&v)[2][8], bool whole, bool in_rows, T* row,
                                        int32_t cw, int32_t lg, int32_t cols, bool vec) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t a0 = pack2(v[h][0], v[h][1], (const T*)nullptr);
    uint32_t b0 = pack2(v[h][2], v[h][3], (const T*)nullptr);
    uint32_t a1 = pack2(v[h][4], v[h][5], (const T*)nullptr);
    uint32_t b1 = pack2(v[h][6], v[h][7], (const T*)nullptr);
    swap16(a0, a1);
    swap16(b0, b1);
    const int32_t c = cw + h * 32 + (lg & 1) * 16 + (lg >> 1) * 8;
    const uint32_t w[4] = {a0, b0, a1, b1};
    if (whole) {  // the same for all lanes
      const lu4 u = {w[0], w[1], w[2], w[3]};
      if constexpr (ONCE) __builtin_nontemporal_store(u, reinterpret_cast<lu4*>(row + c));
      else *reinterpret_cast<lu4*>(row + c) = u;
    } else if (in_rows && vec && c + 8 <= cols) {
      *reinterpret_cast<lu4*>(row + c) = lu4{w[0], w[1], w[2], w[3]};
    } else if (in_rows) {
      uint16_t* p = reinterpret_cast<uint16_t*>(row + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (c + 2 * i < cols) p[2 * i] = (uint16_t)w[i];
        if (c + 2 * i + 1 < cols) p[2 * i + 1] = (uint16_t)(w[i] >> 16);
      }
    }
  }
}

// GATE: the gate function, the identity's number also for relu (the epilogue is
// unrolled, and all six in it would fill the instruction cache).
template <typename T, GatedKind KIND, int GATE>
__global__ __launch_bounds__(kWideThreads, 2) void k_gated_wide(Gated args, Tiles t) {
  constexpr bool FWD = KIND == GatedKind::kForward;
  constexpr int ASRC = FWD ? kKRow : kKCol;
  constexpr int HC = FWD ? kWideTile / 2 : kWideTile;  // hidden columns of a tile
  constexpr int WA = HC / 64, WB = 8 / WA;             // waves along the columns and the rows
  constexpr int TA = FWD ? 8 : 4, TB = kWideTile / 16 / WB;
  __shared__ __align__(1024) char lds[kWideLds];

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wa = wave % WA, wb = wave / WA;
  const int32_t tiles = t.ta * t.tb;
  const int32_t full = (int32_t)(args.k / kBK), rest = (int32_t)(args.k % kBK);
  const int32_t steps = full + (rest > 0);

  AheadStage<ASRC, HC, kWideThreads> sa;
  AheadStage<kKRow, kWideTile, kWideThreads> sb;
  const char *ap, *ap2, *bp;  // of the step to be loaded next
  const char *rest_a, *rest_b;
  int64_t astep;
  int32_t r0, c0;
  // the operands of the tile to be loaded next
  auto begin = [&](int32_t tile) __attribute__((always_inline)) {
    const Gated a = arguments(args);
    // four rows of tiles together, along the columns: the tiles that run at one
    // time share operands of both sides
    const int32_t super = tile / (4 * t.ta), in = tile - super * 4 * t.ta;
    const int32_t high = min(4, t.tb - super * 4);
    r0 = (super * 4 + in % high) * kWideTile;
    c0 = in / high * HC;
    if constexpr (FWD) {
      ap = static_cast<const char*>(a.a) + (int64_t)c0 * a.lda * 2;
      ap2 = ap + (int64_t)a.cols * a.lda * 2;
      astep = kBK * 2;
    } else {
      ap = ap2 = static_cast<const char*>(a.a) + (int64_t)c0 * 2;
      astep = kBK * a.lda * 2;
    }
    bp = static_cast<const char*>(a.b) + (int64_t)r0 * a.ldb * 2;
    rest_a = ap + full * astep;
    rest_b = bp + (int64_t)full * kBK * 2;
    const uint32_t tid = thread_anew();
    sa.init(tid, c0, a.cols, (uint32_t)a.lda);
    sb.init(tid, r0, (int32_t)min(a.rows, (int64_t)0x7FFFFFFF), (uint32_t)a.ldb);
  };
  // the next step's loads to a part of LDS, operand by operand, a piece of each
  // thread's four at a time
  auto issue_a = [&](int32_t slot, bool to_next, int p) __attribute__((always_inline)) {
    char* to = lds + slot;
    if constexpr (FWD) sa.ahead(wave, p < 2 ? ap : ap2, to + (p < 2 ? 0 : kWideHalf / 2), p & 1, 1);
    else sa.ahead(wave, ap, to, p, 1);
    if (p == 3) {
      ap += to_next ? astep : 0;
      if constexpr (FWD) ap2 += to_next ? astep : 0;
    }
  };
  auto issue_b = [&](int32_t slot, bool to_next, int p) __attribute__((always_inline)) {
    sb.ahead(wave, bp, lds + kWideA + slot, p, 1);
    if (p == 3) bp += to_next ? kBK * 2 : 0;
  };
  // A sum whose length is no multiple of the step begins with what is left over: its
  // elements, 0 past them, go over what step 0 loaded there (the first whole step).
  auto put_rest = [&](int32_t slot_a, int32_t slot_b) __attribute__((always_inline)) {
    const uint32_t tid = thread_anew();
    sa.tail(tid, rest_a, lds + slot_a, rest);
    if constexpr (FWD) sa.tail(tid, rest_a + (ap2 - ap), lds + slot_a + kWideHalf / 2, rest);
    sb.tail(tid, rest_b, lds + kWideA + slot_b, rest);
  };
  Frags<ASRC> ga;
  Frags<kKRow> gb;
  ga.init(wa * 64);
  gb.init(wb * TB * 16);
#if defined(__HIP_DEVICE_COMPILE__)
  typedef __attribute__((address_space(3))) char* lp;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lp)lds;
#else
  const uint32_t lds0 = 0;
#endif
  // Of half a step's fragments the four of one operand are used throughout, the
  // eight of the other four products long each: read in this order, behind these
  // products of the half before, a fragment takes the registers of one that is done.
  constexpr bool kAlong = TA > TB;  // whether the first operand has the eight
  auto read_behind = [&](int m, int32_t slot_a, int32_t slot_b, int ks, lu4 (&fa)[TA],
                         lu4 (&fb)[TB]) __attribute__((always_inline)) {
    const int n = m < 4 ? m : m % 4 == 0 ? 3 + m / 4 : m == 30 ? 11 : -1;
    if (n < 0) return;
    const bool first = (n < 4) != kAlong;  // whether it is one of the first operand's
    const int i = n < 4 ? n : n - 4;
    if (!first) {
      fb[i % TB] = gb.read(lds0 + kWideA + (uint32_t)slot_b, ks, i);
    } else if constexpr (FWD) {  // the first four of a wave's tiles are p's, the others u's
      fa[i % TA] = ga.read(lds0 + (uint32_t)slot_a + (i < 4 ? 0 : kWideHalf / 2), ks, i % 4);
    } else {
      fa[i % TA] = ga.read(lds0 + (uint32_t)slot_a, ks, i);
    }
  };
  // The products of half a step, with a piece of other work behind each: a wave
  // issues in order, and what it issues between products that could follow each
  // other at once leaves the matrix cores idle.
  lf4 acc[TA][TB];
  auto products = [&](const lu4 (&fa)[TA], const lu4 (&fb)[TB], auto&& behind)
                      __attribute__((always_inline)) {
#pragma unroll
    for (int m = 0; m < TA * TB; ++m) {
      const int i = kAlong ? m / 4 : m % 4, j = kAlong ? m % 4 : m / 4;
      acc[i][j] = mfma(fa[i], fb[j], acc[i][j], (const T*)nullptr);
      behind(m);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto after = [](int32_t slot) { return slot == 2 * kWideHalf ? 0 : slot + kWideHalf; };
  int32_t round = 0, tile = persistent_tile(0, tiles);
  if (tile < 0) return;
  begin(tile);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
#pragma unroll
    for (int p = 0; p < 4; ++p) issue_a(s * kWideHalf, s > 0 || rest == 0, p);
#pragma unroll
    for (int p = 0; p < 4; ++p) issue_b(s * kWideHalf, s > 0 || rest == 0, p);
  }
  wait_loads();
  if (rest > 0) put_rest(0, 0);
  meet();
  // Step s of a tile lies in a ring of three parts and one of two; its loads are
  // issued under step s - 2, a tile's first two under the last two of the tile
  // before (after the last tile once more its own).
  int32_t slot_a = 0, slot_b = 0;
  while (true) {
    const int32_t rt = r0, cw = c0 + wa * 64;  // the wave's first column
    {
      const Gated a = arguments(args);
      const int32_t lg = (thread_anew() & 63) >> 4;
#pragma unroll
      for (int i = 0; i < TA; ++i) {
        lf4 first = {0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (FWD) {
          if (a.bias) {
            const float* b = global(a.bias) + (i < 4 ? 0 : a.cols);
            for (int m = 0; m < 4; ++m)
              first[m] = b[min(cw + i % 4 * 16 + lg * 4 + m, a.cols - 1)];
          }
        }
#pragma unroll
        for (int j = 0; j < TB; ++j) acc[i][j] = first;
      }
    }
    lu4 fa0[TA], fb0[TB], fa1[TA], fb1[TB];
#pragma unroll
    for (int m = 0; m < 32; ++m) read_behind(m, slot_a, slot_b, 0, fa0, fb0);
    const int32_t next = persistent_tile(round + 1, tiles);
#pragma unroll 1
    for (int32_t s = 0; s < steps; ++s) {
      if (s == steps - 2) begin(next >= 0 ? next : tile);
      const bool to_next = rest == 0 || s != steps - 2;
      const int32_t a1 = after(slot_a), a2 = after(a1), b1 = slot_b ^ kWideHalf;
      // the first half's products over the reads of the second's fragments and the
      // loads of the first operand's step s + 2
      products(fa0, fb0, [&](int m) __attribute__((always_inline)) {
        read_behind(m, slot_a, slot_b, 1, fa1, fb1);
        if (m % 8 == 5) issue_a(a2, to_next, m / 8);
      });
      // step s + 1 has landed: the second operand's loads of it are the last before
      // those of the first operand's step s + 2
      if (s > 0) wait_loads<4>();
      meet();  // every wave has read all of step s
      // the second half's over the next step's first fragments and the loads of the
      // second operand's step s + 2
      products(fa1, fb1, [&](int m) __attribute__((always_inline)) {
        read_behind(m, a1, b1, 0, fa0, fb0);
        if (m % 8 == 5) issue_b(slot_b, to_next, m / 8);
      });
      slot_a = a1;
      slot_b = b1;
    }

    // ---- the tile's results ----
    const Gated a = arguments(args);
    const uint32_t tid = thread_anew();
    const int32_t l = tid & 63, lg = l >> 4;
    const int64_t groups = groups_of(a.cols);
    const int32_t cl = cw + lg * 16;  // the lane's columns after transposing
    const bool edge = cw + 64 > a.cols;
    const bool vec = FWD || a.cols % 8 == 0;
    const bool whole = vec && !edge && (int64_t)rt + kWideTile <= a.rows;
    const int gate = GATE == kActNone ? min(a.gate, kActRelu) : GATE;
    // kept pre-activations of the row's 16 columns, two rows of tiles ahead (one
    // ahead, each was waited for)
    constexpr int kDeep = 3;
    struct Pre {
      lu4 p, u;
      uint32_t e;  // of p's two groups and of u's, in the four groups of 16 lanes
    } pre[FWD ? 1 : kDeep];
    const int32_t last = (int32_t)groups - 1;
    auto load_pre = [&](int j, Pre& k) __attribute__((always_inline)) {
      const int64_t r = min((int64_t)rt + (wb * TB + j) * 16 + (l & 15), a.rows - 1);
      const int64_t at = (r * groups + min(cl / kAct8Group, last)) * kAct8Group + (cl & 16);
      k.p = *reinterpret_cast<const lu4*>(global(a.qp) + at);
      k.u = *reinterpret_cast<const lu4*>(global(a.qu) + at);
      k.e = global(lg < 2 ? a.ep : a.eu)[r * groups + min(cw / kAct8Group + (lg & 1), last)];
    };
    // the next tile's steps, before stores that would be waited for; back, the kept
    // rows' first loads are behind them and waited for before the first store
    if constexpr (FWD) {
      wait_loads();
    } else {
#pragma unroll
      for (int j = 0; j < kDeep; ++j) load_pre(j, pre[j]);
    }
#pragma unroll
    for (int j = 0; j < TB; ++j) {  // the results of 16 rows
      const int64_t r = (int64_t)rt + (wb * TB + j) * 16 + (l & 15);
      const bool in_rows = r < a.rows;
      T* row = global(static_cast<T*>(a.c)) + r * a.ldc;
      float x[TA / 2][8];
#pragma unroll
      for (int i = 0; i < TA; ++i)
        for (int m = 0; m < 4; ++m) x[i / 2][i % 2 * 4 + m] = acc[i][j][m];
      if constexpr (FWD) {
        if (edge) {  // columns past the last are kept as 0
#pragma unroll
          for (int i = 0; i < 8; ++i)
            for (int m = 0; m < 4; ++m)
              if (cw + i % 4 * 16 + lg * 4 + m >= a.cols) x[i / 2][i % 2 * 4 + m] = 0.0f;
        }
        float (&p)[2][8] = reinterpret_cast<float (&)[2][8]>(x[0]);
        float (&u)[2][8] = reinterpret_cast<float (&)[2][8]>(x[2]);
        const int64_t at_e = r * groups + cl / kAct8Group;
        const int64_t at_q = at_e * kAct8Group + (cl & 16);
        const bool in = in_rows && cl / kAct8Group < groups, in_e = in && (lg & 1) == 0;
        if (a.qp) {
          keep16(p, in, at_q, at_e, in_e, global(a.qp), global(a.ep));
          keep16(u, in, at_q, at_e, in_e, global(a.qu), global(a.eu));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          gate_value(p[h], gate);
          for (int m = 0; m < 8; ++m) p[h][m] *= u[h][m];
        }
        if (a.q) {  // as rounded: what reading y and encoding it would give
          float y[2][8];
#pragma unroll
          for (int h = 0; h < 2; ++h) unpack(pack(p[h], (const T*)nullptr), y[h], (const T*)nullptr);
          keep16(y, in, at_q, at_e, in_e, global(a.q), global(a.e));
        }
        store16<T, true>(p, whole, in_rows, row, cw, lg, a.cols, vec);
      } else {
        float (&d)[2][8] = reinterpret_cast<float (&)[2][8]>(x[0]);
        Pre& k = pre[j % kDeep];
        uint32_t wp[4] = {k.p[0], k.p[1], k.p[2], k.p[3]};
        uint32_t wu[4] = {k.u[0], k.u[1], k.u[2], k.u[3]};
        uint32_t ex[4];
        spread4(k.e, ex);
        const float sp[2] = {step_of(ex[0]), step_of(ex[1])};
        const float su[2] = {step_of(ex[2]), step_of(ex[3])};
        if (j + kDeep < TB) load_pre(j + kDeep, k);
        transpose4(wp);
        transpose4(wu);
        float f[2][8], df[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float u[8];
          dequant4(wp[2 * h], sp[h], f[h]);
          dequant4(wp[2 * h + 1], sp[h], f[h] + 4);
          dequant4(wu[2 * h], su[h], u);
          dequant4(wu[2 * h + 1], su[h], u + 4);
          gate_both(f[h], df[h], gate);
#pragma unroll
          for (int m = 0; m < 8; ++m) {
            df[h][m] *= d[h][m] * u[m];
            f[h][m] *= d[h][m];
          }
        }
        store16<T, false>(df, whole, in_rows, row, cw, lg, a.cols, true);
        store16<T, false>(f, whole, in_rows, row + a.cols, cw, lg, a.cols, vec);
      }
    }
    if (next < 0) break;
    tile = next;
    ++round;
    if (rest > 0) put_rest(slot_a, slot_b);
    meet();  // every wave's part of the next tile's first steps is there
  }
}

// ---- the forward product of few rows ----------------------------------------------
// Up to 64 rows cost what reading w costs.  A block owns 16 columns, or 32 (a group)
// where 8 bits are kept: their rows of the gate's weights and of the others', one
// or two fragments each.  Its 8 waves share k in lines of 64, each wave's fragments
// straight from memory (a line of w is used by one wave, once), all of a batch's
// loads before its products.  The waves' sums meet in LDS, added in wave order.
// 1 x 1600 -> 2 x 6400 (41 MB of w) takes 10.6 us, 3.9 TB/s, what the call takes on
// the host too.
constexpr int kFewWaves = 8;

template <typename T, int NB, int NA>
__global__ __launch_bounds__(kFewWaves * 64, 2) void k_gated_few(Gated a) {
  constexpr int U = NB <= 2 ? 4 : 2;  // lines of a batch
  constexpr int HC = NA * 8;          // columns of the block
  __shared__ lf4 lds[kFewWaves][NB][NA][64];
  const int l = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t c0 = blockIdx.x * HC;
  const uint16_t *aw[NA], *bx[NB];
  for (int i = 0; i < NA; ++i) {
    const int32_t c = min(c0 + i % (NA / 2) * 16 + (l & 15), a.cols - 1);
    aw[i] = static_cast<const uint16_t*>(a.a) + (int64_t)(i < NA / 2 ? c : a.cols + c) * a.lda;
  }
  for (int j = 0; j < NB; ++j)
    bx[j] = static_cast<const uint16_t*>(a.b) +
            min((int64_t)(j * 16 + (l & 15)), a.rows - 1) * a.ldb;
  lf4 acc[NA][NB];
  for (int i = 0; i < NA; ++i)
    for (int j = 0; j < NB; ++j) acc[i][j] = lf4{0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t step = kFewWaves * 64;
  for (int64_t k0 = wave * 64; k0 < a.k; k0 += step * U) {
    lu4 fa[U][NA][2], fb[U][NB][2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t k = k0 + u * step + h * 32 + (l >> 4) * 8;
#pragma unroll
        for (int i = 0; i < NA; ++i) fa[u][i][h] = load_k(aw[i], k, a.k);
#pragma unroll
        for (int j = 0; j < NB; ++j) fb[u][j][h] = load_k(bx[j], k, a.k);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int i = 0; i < NA; ++i)
            acc[i][j] = mfma(fa[u][i][h], fb[u][j][h], acc[i][j], (const T*)nullptr);
  }
  for (int j = 0; j < NB; ++j)
    for (int i = 0; i < NA; ++i) lds[wave][j][i][l] = acc[i][j];
  __syncthreads();
  // wave j finishes rows 16j .. 16j+15: NA lanes to a row, eight columns each
  if (wave >= NB || l >= 16 * NA) return;
  const int row = l / NA, cc = l % NA * 8;
  const int64_t r = wave * 16 + row;
  const int32_t c = c0 + cc;
  float v[2][8] = {}, bp[8], bu[8];
  load_bias(a, c, bp, bu);
  for (int w = 0; w < kFewWaves; ++w)
    for (int g = 0; g < 2; ++g)
      for (int h = 0; h < 2; ++h) {
        const lf4 x = lds[w][wave][g * (NA / 2) + cc / 16][((cc % 16) / 4 + h) * 16 + row];
        for (int j = 0; j < 4; ++j) v[g][4 * h + j] += x[j];
      }
  finish_forward<T>(a, r, c, bp, bu, v[0], v[1]);
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
constexpr int kSplitBelow = kCUs / 2, kSplitLeast = 4;

int64_t tiles_of(GatedKind kind, int64_t rows, int32_t cols, int32_t tile) {
  const int32_t wide = kind == GatedKind::kForward ? tile / 2 : tile;
  return (int64_t)((cols + wide - 1) / wide) * ((rows + tile - 1) / tile);
}

// Whether a product of few tiles of 128 x 128 is cut into tiles of 64 x 64.  In us,
// 128 and 64: 515 x 777 -> 2 x 1001 (80 tiles) 21.3 and 14.3, 256 x 1600 -> 2 x 6400
// (200) 35.3 and 25.6; but 2048 x 1024 -> 2 x 2048 (512 tiles) 24.2 and 32.9; the hidden
// gradient of 1500 x 1600 -> 3200 (300 tiles) 45.0 and 35.2, of 4096 x 1024 -> 2048
// (512) 38.4 and 42.1.
bool small(GatedKind kind, int64_t rows, int32_t cols) {
  return tiles_of(kind, rows, cols, 128) <=
         (kind == GatedKind::kForward ? kCUs : kCUs + kCUs / 2);
}

Tiles choose(GatedKind kind, int64_t rows, int32_t cols, int64_t k) {
  const int32_t tile = small(kind, rows, cols) ? 64 : 128;
  const int32_t wide = kind == GatedKind::kForward ? tile / 2 : tile;
  Tiles t;
  t.ta = (cols + wide - 1) / wide;
  t.tb = (int32_t)((rows + tile - 1) / tile);
  const int64_t all = (int64_t)t.ta * t.tb, steps = (k + kBK - 1) / kBK;
  int64_t splits = 1;
  if (all > 0 && all <= kSplitBelow)
    splits = std::max<int64_t>(1, std::min<int64_t>({2 * kCUs / all, steps / kSplitLeast,
                                                     (int64_t)kMaxSplits}));
  t.ksteps = (int32_t)std::max<int64_t>(1, (steps + splits - 1) / splits);
  t.splits = (int32_t)std::max<int64_t>(1, (steps + t.ksteps - 1) / t.ksteps);
  return t;
}

// Whether the tiles of 256 x 256 are taken: sums of the two whole steps that are
// loaded ahead, and rounds of one tile to a CU that leave few CUs without one.  In
// us, 128 x 128 and 256 x 256: 4096 x 1024 -> 2 x 4096 (2 full rounds) 80 and 68, 6000
// x 1000 -> 2 x 4300 (4 rounds, 80 % full) 149 and 133, 2600 x 300 -> 2 x 2600 (1
// round, 90 %) 26.5 and 22.6, 3000 x 2000 -> 2 x 1500 (1 round, 56 %) 62 and 50; but
// 4096 x 1024 -> 2 x 3000 (2 rounds, 75 %) 60 and 66, 4096 x 1024 -> 2 x 1024 (1, 50
// %) 24 and 28; the hidden gradient of 4096 x 1024 -> 3000 (1 round, 75 %) 58 and 49,
// of 4096 x 4000 -> 2300 (1, 56 %) 124 and 130.
bool wide(GatedKind kind, int64_t rows, int32_t cols, int64_t k) {
  if (k < 2 * kBK) return false;
  const int64_t t = tiles_of(kind, rows, cols, kWideTile), rounds = (t + kCUs - 1) / kCUs;
  if (rounds > 1) return t * 100 >= rounds * kCUs * 77;
  return t >= kCUs * 3 / 4 || (kind == GatedKind::kForward && t > kCUs / 2 && k >= 1536);
}

// Whether the few-rows kernel takes a forward product: one launch and no
// workspace, but every block walks all of k and reads all of x.  Against the split
// tiles, us a call: 1 x 1600 -> 2 x 6400 10.7 and 15.8, 1 x 16384 -> 2 x 1024 34.9
// and 37.7, 16 x 4096 -> 2 x 1024 14.2 and 17.6, 64 x 1024 -> 2 x 4096 9.7 and 14.6,
// 64 x 1600 -> 2 x 6400 17.5 and 18.7; but 64 x 2048 -> 2 x 6400 22.4 and 21.0, 8 x
// 16384 -> 2 x 1024 40.2 and 38.5, 32 x 4096 -> 2 x 6400 40.5 and 30.3.
bool few(GatedKind kind, int64_t rows, int64_t k) {
  return kind == GatedKind::kForward && rows <= 64 && rows * k <= 102400;
}
// Whether its blocks take 32 columns where they could take 16: half as many, and x
// read half as often.  16 and 32 columns, us: 16 x 1600 -> 2 x 6400 12.7 and 11.8,
// 64 rows 22.7 and 17.5; but 1 row 10.7 and 10.9, 64 x 1024 -> 2 x 4096 9.7 and 11.7.
bool few_wide(const Gated& a) { return a.qp || a.q || (a.rows > 4 && a.cols >= 6144); }

template <typename T, int NB>
void product_few(const Gated& a, hipStream_t st) {
  const dim3 block(kFewWaves * 64);
  if (few_wide(a))
    hipLaunchKernelGGL(HIP_KERNEL_NAME(k_gated_few<T, NB, 4>), dim3((a.cols + 31) / 32), block, 0,
                       st, a);
  else
    hipLaunchKernelGGL(HIP_KERNEL_NAME(k_gated_few<T, NB, 2>), dim3((a.cols + 15) / 16), block, 0,
                       st, a);
}

template <typename T, GatedKind KIND>
void product(const Gated& a, hipStream_t st) {
  if (few(KIND, a.rows, a.k)) {
    if (a.rows <= 16) product_few<T, 1>(a, st);
    else if (a.rows <= 32) product_few<T, 2>(a, st);
    else product_few<T, 4>(a, st);
    return;
  }
  if (wide(KIND, a.rows, a.cols, a.k)) {
    constexpr int32_t c = KIND == GatedKind::kForward ? kWideTile / 2 : kWideTile;
    const Tiles t{(a.cols + c - 1) / c, (int32_t)((a.rows + kWideTile - 1) / kWideTile), 1, 0};
    auto launch = [&](auto gate) {
      hipLaunchKernelGGL(HIP_KERNEL_NAME(k_gated_wide<T, KIND, gate.value>), dim3(kCUs),
                         dim3(kWideThreads), 0, st, a, t);
    };
    if (a.gate == kGateSilu) launch(std::integral_constant<int, kGateSilu>{});
    else if (a.gate == kGateSigmoid) launch(std::integral_constant<int, kGateSigmoid>{});
    else if (a.gate == kActGelu) launch(std::integral_constant<int, kActGelu>{});
    else if (a.gate == kActGeluTanh) launch(std::integral_constant<int, kActGeluTanh>{});
    else launch(std::integral_constant<int, kActNone>{});
    return;
  }
  const Tiles t = choose(KIND, a.rows, a.cols, a.k);
  const uint32_t grid = (uint32_t)gated_blocks(KIND, a.rows, a.cols, a.k);
  if (small(KIND, a.rows, a.cols)) {
    constexpr int WA = KIND == GatedKind::kForward ? 1 : 2;
    hipLaunchKernelGGL(HIP_KERNEL_NAME(k_gated<T, KIND, 64, 64, WA, 4 / WA, 3>), dim3(grid),
                       dim3(256), 0, st, a, t);
  } else {
    hipLaunchKernelGGL(HIP_KERNEL_NAME(k_gated<T, KIND, 128, 128, 2, 2, 1>), dim3(grid), dim3(256),
                       0, st, a, t);
  }
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
  if (few(kind, rows, k) || wide(kind, rows, cols, k)) return 1;
  return choose(kind, rows, cols, k).splits;
}

int64_t gated_blocks(GatedKind kind, int64_t rows, int32_t cols, int64_t k) {
  if (few(kind, rows, k)) return (cols + 15) / 16;
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
