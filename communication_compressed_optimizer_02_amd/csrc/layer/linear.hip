// linear.hip -- the matrix products of a linear layer on the matrix cores
// (gfx950), with everything that touches their result in the epilogue.
//
//   forward       y[t][f]  = act(sum_k x[t][k] w[f][k] + bias[f]) + residual[t][f]
//   input grad    dx[t][i] = (sum_o dy[t][o] w[o][i]) act'(p[t][i]) + add[t][i]
//   weight grad   dw[o][i] = sum_t dy[t][o] x[t][i], db[o] = sum_t dy[t][o]
//                 (one product per worker, x and p kept in 8 bits)
//
// All three are C[r][c] = sum_k B(r, k) A(c, k), on the operands' paths and
// layouts of tile.hpp.  A lane's four results are four consecutive columns of
// one row: one 16-byte write to the rows of LDS that the epilogue takes back
// eight columns a lane, a group of 32 columns for the 8-bit form in four lanes.
// Sums are binary32 in the accumulators, in increasing k; a product of few
// tiles is split over k, its binary32 sums joined in split order.
//
// One 128 x 128 tile serves all three: a step of 64 along k is 32 KB, loaded
// straight to LDS (no registers, no LDS writes by the waves), so that three
// blocks of four waves fit a CU and one's products hide the others' loads and
// epilogues.  At 16384 x 1024 -> 4096 in bfloat16 (137 GFLOP; us in a steady
// run, and a median of 12 calls under the profiler, whose clocks are lower):
// 147 (158) bare, 167 with GELU, 189-196 (201-229) with GELU and the
// pre-activation kept, 148 the input gradient, 190-204 (199-220) with GELU's
// derivative from 8 bits, 171-176 (177-189) the weight gradients of 8 workers
// from 8 bits; the library's bare product takes 108.  A 256 x 256 tile of eight
// waves with two halves of LDS took 152 bare, but 208 with its epilogue, which
// nothing hides; 128 x 256 took 140, 168 and 197, and 216 for the input gradient
// with GELU's derivative.  What bounds it, by the counters: waiting.  The matrix
// cores are busy for 42 % of a bare product at K = 1024 and 55 % at K = 4096
// (1.13 PFLOP/s; the library 1.55), fragment reads keep LDS busy for 26 and 29 %,
// and the waves wait for 46 and 50 % of their time: a step's loads are all waited
// for before its products start, so only the other blocks of the CU cover them.
// With GELU and the kept form a result takes 30 vector instructions instead of 8,
// and the matrix cores are busy for 34 %.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "layer.hpp"
#include "layer_kernels.hpp"
#include "tile.hpp"

namespace oba {

namespace {

// ---- epilogues ---------------------------------------------------------------------
// What the epilogue reads for eight results, loaded ahead of their use (a
// load behind each use left the epilogue waiting: 107 of 255 us at 16384 x
// 1024 -> 4096 for the bias alone).
struct Extra {
  lu2 u;        // kept pre-activation of the derivative
  uint32_t e;
  lu4 add;      // residual
};

template <LinearKind KIND>
__device__ __forceinline__ void load_extra(const Linear& a, int64_t r, int32_t c, Extra& x) {
  if (r >= a.rows || c >= a.cols) return;
  if constexpr (KIND == LinearKind::kInputGrad) {
    if (a.act != kActNone) {
      const int64_t g = r * ((a.cols + kAct8Group - 1) / kAct8Group) + c / kAct8Group;
      x.u = *reinterpret_cast<const lu2*>(a.pq + g * kAct8Group + c % kAct8Group);
      x.e = a.pe[g];
    }
  }
  if (a.add)
    x.add = *reinterpret_cast<const lu4*>(static_cast<const uint16_t*>(a.add) + r * a.ldadd + c);
}

__device__ __forceinline__ void load_bias(const Linear& a, int32_t c, float (&b)[8]) {
  for (int j = 0; j < 8; ++j) b[j] = a.bias && c + j < a.cols ? a.bias[c + j] : 0.0f;
}

// The forward result from the product, the input gradient from the product:
// bias, 8-bit pre-activation kept or used, activation or its derivative,
// residual, one rounding.  Four neighbouring lanes hold a group of 32 columns.
template <typename T, LinearKind KIND>
__device__ __forceinline__ void finish(const Linear& a, int64_t r, int32_t c, const float (&b)[8],
                                       const Extra& x, float (&v)[8]) {
  const int n = a.cols - c;
  const bool in_rows = r < a.rows;
  if constexpr (KIND == LinearKind::kForward) {
    if (a.bias)
      for (int j = 0; j < 8; ++j) v[j] += b[j];
    if (a.q) {
      const int32_t groups = (a.cols + kAct8Group - 1) / kAct8Group;
      if (n < 8) {  // columns past the last are kept as 0
        for (int j = 0; j < 8; ++j) v[j] = j < n ? v[j] : 0.0f;
      }
      const uint32_t top = max_lanes<4>(magnitude8(v));
      const uint32_t ex = group_exp(top);
      const float inv = inv_step_of(ex), step = step_of(ex);
      if (in_rows && c / kAct8Group < groups) {
        const int64_t g = r * groups + c / kAct8Group;
        *reinterpret_cast<lu2*>(a.q + g * kAct8Group + c % kAct8Group) =
            lu2{quant4(v, inv, step, ex != 255u), quant4(v + 4, inv, step, ex != 255u)};
        if (c % kAct8Group == 0) a.e[g] = (uint8_t)ex;
      }
    }
  }
  if (!in_rows || n <= 0) return;
  if constexpr (KIND == LinearKind::kForward) {
    activate(v, a.act);
  } else if (a.act != kActNone) {
    const float s = step_of(x.e);
    float d[8];
    for (int j = 0; j < 8; ++j) d[j] = dequant(x.u[j / 4], j % 4, s);
    activate_grad(d, a.act);
    for (int j = 0; j < 8; ++j) v[j] *= d[j];
  }
  if (a.add) {
    float w[8];
    unpack(x.add, w, (const T*)nullptr);
    for (int j = 0; j < 8; ++j) v[j] += w[j];
  }
  store8(static_cast<T*>(a.c) + r * a.ldc + c, n, v);
}

// The weight gradient's rows lie where their tensor lies in the flat gradient
// row, at any alignment: vectors where that allows them.
__device__ __forceinline__ bool grad_vec(const Linear& a) {
  return ((uintptr_t)a.c & 15) == 0 && a.cols % 8 == 0 && a.ldg % 8 == 0;
}

__device__ __forceinline__ void store_grad(const Linear& a, bool vec, int32_t worker, int64_t r,
                                           int32_t c, const float (&v)[8]) {
  const int64_t at = (int64_t)worker * a.ldg + r * a.cols + c;
  const int n = a.cols - c;
  if (a.g_dtype == kGradF32) {
    float* p = static_cast<float*>(a.c) + at;
    if (vec) {
      reinterpret_cast<lf4*>(p)[0] = lf4{v[0], v[1], v[2], v[3]};
      reinterpret_cast<lf4*>(p)[1] = lf4{v[4], v[5], v[6], v[7]};
    } else {
      for (int j = 0; j < 8; ++j)
        if (j < n) p[j] = v[j];
    }
  } else if (a.g_dtype == kGradF16) {
    store8(static_cast<_Float16*>(a.c) + at, vec ? 8 : min(n, 7), v);
    if (!vec && n >= 8) static_cast<_Float16*>(a.c)[at + 7] = (_Float16)v[7];
  } else {
    store8(static_cast<__bf16*>(a.c) + at, vec ? 8 : min(n, 7), v);
    if (!vec && n >= 8) static_cast<__bf16*>(a.c)[at + 7] = (__bf16)v[7];
  }
}

__device__ __forceinline__ void store_bias_grad(const Linear& a, int32_t worker, int64_t r,
                                                float v) {
  const int64_t at = (int64_t)worker * a.ldg + r;
  if (a.g_dtype == kGradF32) static_cast<float*>(a.db)[at] = v;
  else if (a.g_dtype == kGradF16) static_cast<_Float16*>(a.db)[at] = (_Float16)v;
  else static_cast<__bf16*>(a.db)[at] = (__bf16)v;
}

// Partial sums of a split product: [split][worker][rows][cols8], then the
// bias gradient's [split][worker][rows].
__device__ __forceinline__ int64_t part_cols(const Linear& a) { return (a.cols + 7) / 8 * 8; }

// ---- the product --------------------------------------------------------------------
struct Tiles {
  int32_t ta, tb;    // tiles along the result's columns and rows
  int32_t splits;
  int32_t ksteps;    // steps of kBK of one split
};

template <typename T, LinearKind KIND, int BA, int BB, int WA, int WB>
__global__ __launch_bounds__(WA* WB * 64, 3) void k_linear(Linear a, Tiles t) {
  constexpr int NT = WA * WB * 64;
  constexpr int ASRC = KIND == LinearKind::kForward ? kKRow
                       : KIND == LinearKind::kInputGrad ? kKCol : kKept;
  constexpr int BSRC = KIND == LinearKind::kWeightGrad ? kKCol : kKRow;
  constexpr int TA = BA / WA / 16, TB = BB / WB / 16;
  constexpr int kA = BA * kBK * 2, kStageBytes = kA + BB * kBK * 2;  // of a step in LDS
  __shared__ __align__(1024) char lds[kStageBytes];

  const int64_t work = xcd_order(blockIdx.x, gridDim.x);
  const int32_t tiles = t.ta * t.tb;
  const int32_t tile = (int32_t)(work % tiles);
  const int32_t rest = (int32_t)(work / tiles);
  const int32_t split = rest % t.splits, worker = rest / t.splits;
  // four rows of tiles together, along the columns: the tiles that run at one
  // time share operands of both sides
  const int32_t super = tile / (4 * t.ta), in = tile - super * 4 * t.ta;
  const int32_t high = min(4, t.tb - super * 4);
  const int32_t r0 = (super * 4 + in % high) * BB, c0 = in / high * BA;

  const int64_t kbeg = (int64_t)split * t.ksteps * kBK;
  const int64_t kend = min(a.k, kbeg + (int64_t)t.ksteps * kBK);
  const uint32_t eld = (uint32_t)((a.cols + kAct8Group - 1) / kAct8Group);
  const char* ap;
  const uint8_t* ae = nullptr;
  int64_t astep, bstep;  // bytes of one step along k
  if constexpr (ASRC == kKRow) {
    ap = static_cast<const char*>(a.a) + ((int64_t)c0 * a.lda + kbeg) * 2;
    astep = kBK * 2;
  } else {
    constexpr int S = ASRC == kKept ? 1 : 2;
    const int64_t k0 = (KIND == LinearKind::kWeightGrad ? worker * a.k : 0) + kbeg;
    ap = static_cast<const char*>(a.a) + (k0 * a.lda + c0) * S;
    astep = kBK * a.lda * S;
    if constexpr (ASRC == kKept) ae = a.ae + k0 * eld + c0 / kAct8Group;
  }
  const char* bp;
  if constexpr (BSRC == kKRow) {
    bp = static_cast<const char*>(a.b) + ((int64_t)r0 * a.ldb + kbeg) * 2;
    bstep = kBK * 2;
  } else {
    bp = static_cast<const char*>(a.b) + (((int64_t)worker * a.k + kbeg) * a.ldb + r0) * 2;
    bstep = kBK * a.ldb * 2;
  }

  Stage<T, ASRC, BA, NT> sa;
  Stage<T, BSRC, BB, NT> sb;
  sa.init(c0, a.cols, (uint32_t)a.lda, eld);
  sb.init(r0, (int32_t)min(a.rows, (int64_t)0x7FFFFFFF), (uint32_t)a.ldb, 0);

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // uniform
  const int wa = wave % WA, wb = wave / WA;
  lf4 acc[TA][TB];
#pragma unroll
  for (int i = 0; i < TA; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j) acc[i][j] = lf4{0.0f, 0.0f, 0.0f, 0.0f};
  // the bias gradient: the product with a row of ones, by the waves that hold
  // the result's first columns
  const bool ones = KIND == LinearKind::kWeightGrad && a.db && c0 == 0 && wa == 0;
  lf4 accb[KIND == LinearKind::kWeightGrad ? TB : 1];
  for (auto& v : accb) v = lf4{0.0f, 0.0f, 0.0f, 0.0f};
  const uint32_t one2 = pack2(1.0f, 1.0f, (const T*)nullptr);
  const lu4 one8 = {one2, one2, one2, one2};

  // the direct loads of a wave have landed in LDS (a barrier alone does not
  // wait for them)
  auto landed = [] { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); };
  auto direct = [&](char* l) __attribute__((always_inline)) {
    if constexpr (ASRC != kKept) {
      sa.direct(ap, l);
      ap += astep;
    }
    sb.direct(bp, l + kA);
    bp += bstep;
  };
  // the kept operand's step to registers: a whole one, or the sum's last
  auto load_full = [&]() __attribute__((always_inline)) {
    if constexpr (ASRC == kKept) {
      sa.template load<false>(ap, ae, kBK);
      ap += astep;
      ae += (int64_t)kBK * eld;
    }
  };
  auto load_tail = [&](int32_t left) __attribute__((always_inline)) {
    if constexpr (ASRC == kKept) sa.template load<true>(ap, ae, left);
  };
  auto products = [&](const lu4 (&fa)[TA], const lu4 (&fb)[TB]) {
#pragma unroll
    for (int j = 0; j < TB; ++j)
#pragma unroll
      for (int i = 0; i < TA; ++i) acc[i][j] = mfma(fa[i], fb[j], acc[i][j], (const T*)nullptr);
    if constexpr (KIND == LinearKind::kWeightGrad) {
      if (ones) {
#pragma unroll
        for (int j = 0; j < TB; ++j) accb[j] = mfma(one8, fb[j], accb[j], (const T*)nullptr);
      }
    }
  };
  auto fragments = [&](const char* la, const char* lb, int ks, lu4 (&fa)[TA], lu4 (&fb)[TB]) {
#pragma unroll
    for (int i = 0; i < TA; ++i) fa[i] = fragment<ASRC, BA>(la, (wa * TA + i) * 16, ks);
#pragma unroll
    for (int j = 0; j < TB; ++j) fb[j] = fragment<BSRC, BB>(lb, (wb * TB + j) * 16, ks);
  };

  auto compute = [&](const char* l) __attribute__((always_inline)) {
#pragma unroll
    for (int ks = 0; ks < kBK / 32; ++ks) {
      lu4 fa[TA], fb[TB];
      fragments(l, l + kA, ks, fa, fb);
      products(fa, fb);
    }
  };
  const int32_t full = (int32_t)((kend - kbeg) / kBK), rest_k = (int32_t)((kend - kbeg) % kBK);
  auto load_rest = [&]() __attribute__((always_inline)) {
    if (rest_k > 0) load_tail(rest_k);
  };
  if (full > 0) load_full();
  else load_rest();
  for (int32_t s = 0; s < full; ++s) {
    if (s > 0) __syncthreads();  // every wave is done with the last step's tile
    direct(lds);
    if constexpr (ASRC == kKept) sa.store(lds);
    if (s + 1 < full) load_full();
    else load_rest();
    landed();
    __syncthreads();
    compute(lds);
  }
  if (rest_k > 0) {
    if (full > 0) __syncthreads();
    if constexpr (ASRC == kKept) sa.store(lds);
    else sa.tail(ap, lds, rest_k);
    sb.tail(bp, lds + kA, rest_k);
    __syncthreads();
    compute(lds);
  }

  // The results go through LDS, 16 rows of a wave at a time and within the
  // wave alone: lane l holds row l % 16 and four columns of each tile, and
  // takes back eight consecutive columns, so that a row's stores and operands
  // are whole lines.
  constexpr int kRow = TA * 16 + 4;  // floats of a row in LDS, off the bank period
  constexpr int kLanes = TA * 2;     // lanes of a row
  static_assert(WA * WB * 16 * kRow * 4 <= kStageBytes, "epilogue rows fit the tile");
  const int l = threadIdx.x & 63;
  float* rows = reinterpret_cast<float*>(lds) + wave * 16 * kRow;
  const bool vec = KIND == LinearKind::kWeightGrad && grad_vec(a);
  const int64_t pc = part_cols(a), wrow = ((int64_t)split * a.n + worker) * a.rows;
  __syncthreads();  // every wave has read its last fragments
  constexpr int kIter = 16 * kLanes / 64;
  const int rr = l / kLanes, cc = l % kLanes * 8;  // the lane's first row, and its columns
  const int32_t c = c0 + wa * TA * 16 + cc;
  float bias[8];
  if constexpr (KIND == LinearKind::kForward) load_bias(a, c, bias);
#pragma unroll 1
  for (int j = 0; j < TB; ++j) {
    const int64_t rj = r0 + (wb * TB + j) * 16;
    Extra extra[kIter];
    if constexpr (KIND != LinearKind::kWeightGrad) {
      if (t.splits == 1) {
#pragma unroll
        for (int i = 0; i < kIter; ++i)
          load_extra<KIND>(a, rj + rr + i * (64 / kLanes), c, extra[i]);
      }
    }
#pragma unroll
    for (int jj = 0; jj < TB; ++jj) {
      if (jj != j) continue;  // a constant index into the accumulators
#pragma unroll
      for (int i = 0; i < TA; ++i)
        *reinterpret_cast<lf4*>(rows + (l & 15) * kRow + i * 16 + (l >> 4) * 4) = acc[i][jj];
      if constexpr (KIND == LinearKind::kWeightGrad) {
        if (ones && l < 16 && rj + l < a.rows) {
          if (t.splits > 1)
            a.part[(int64_t)t.splits * a.n * a.rows * pc + wrow + rj + l] = accb[jj][0];
          else
            store_bias_grad(a, worker, rj + l, accb[jj][0]);
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int ri = rr + i * (64 / kLanes);
      const int64_t r = rj + ri;
      const lf4 x = *reinterpret_cast<const lf4*>(rows + ri * kRow + cc);
      const lf4 y = *reinterpret_cast<const lf4*>(rows + ri * kRow + cc + 4);
      float v[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
      if (t.splits > 1) {
        if (r < a.rows && c < a.cols) {
          lf4* p = reinterpret_cast<lf4*>(a.part + (wrow + r) * pc + c);
          p[0] = x;
          p[1] = y;
        }
      } else if constexpr (KIND == LinearKind::kWeightGrad) {
        if (r < a.rows && c < a.cols) store_grad(a, vec, worker, r, c, v);
      } else {
        finish<T, KIND>(a, r, c, bias, extra[i], v);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

// ---- the forward product of few rows ----------------------------------------------
// Up to 64 rows cost what reading w costs.  A block owns 32 columns (a group
// of the 8-bit form); its 8 waves share k in lines of 64, each wave's
// fragments straight from memory (a line of w is used by one wave, once), all
// of a batch's loads before its products.  The waves' sums meet in LDS, added
// in wave order.  1 x 1600 -> 6400 (20 MB of w): 7.4 us, 2.8 TB/s.  All of this k
// is one batch a wave (2048 to a batch of up to 32 rows), so each load's latency
// is paid once; 200 blocks leave 56 of the 256 CUs idle, and of the 25 lines one
// wave has four and the others three.  Split tiles and their join took 9.0 + 5.0.
constexpr int kFewWaves = 8, kFewCols = 32;

template <typename T, int NB>
__global__ __launch_bounds__(kFewWaves * 64, 2) void k_linear_few(Linear a) {
  constexpr int U = NB <= 2 ? 4 : 2;  // lines of a batch
  __shared__ lf4 lds[kFewWaves][NB][2][64];
  const int l = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t c0 = blockIdx.x * kFewCols;
  const uint16_t *aw[2], *bx[NB];
  for (int i = 0; i < 2; ++i)
    aw[i] = static_cast<const uint16_t*>(a.a) +
            (int64_t)min(c0 + i * 16 + (l & 15), a.cols - 1) * a.lda;
  for (int j = 0; j < NB; ++j)
    bx[j] = static_cast<const uint16_t*>(a.b) +
            min((int64_t)(j * 16 + (l & 15)), a.rows - 1) * a.ldb;
  lf4 acc[2][NB];
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < NB; ++j) acc[i][j] = lf4{0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t step = kFewWaves * 64;
  for (int64_t k0 = wave * 64; k0 < a.k; k0 += step * U) {
    lu4 fa[U][2][2], fb[U][NB][2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t k = k0 + u * step + h * 32 + (l >> 4) * 8;
#pragma unroll
        for (int i = 0; i < 2; ++i) fa[u][i][h] = load_k(aw[i], k, a.k);
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
          for (int i = 0; i < 2; ++i)
            acc[i][j] = mfma(fa[u][i][h], fb[u][j][h], acc[i][j], (const T*)nullptr);
  }
  for (int j = 0; j < NB; ++j)
    for (int i = 0; i < 2; ++i) lds[wave][j][i][l] = acc[i][j];
  __syncthreads();
  if (wave >= NB) return;
  // wave j finishes rows 16j .. 16j+15: four lanes to a row, eight columns each
  const int row = l >> 2, cc = (l & 3) * 8;
  const int64_t r = wave * 16 + row;
  const int32_t c = c0 + cc;
  float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f}, b[8];
  Extra x;
  load_bias(a, c, b);
  load_extra<LinearKind::kForward>(a, r, c, x);
  for (int w = 0; w < kFewWaves; ++w)
    for (int h = 0; h < 2; ++h) {
      const lf4 p = lds[w][wave][cc / 16][((cc % 16) / 4 + h) * 16 + row];
      for (int j = 0; j < 4; ++j) v[4 * h + j] += p[j];
    }
  finish<T, LinearKind::kForward>(a, r, c, b, x, v);
}

constexpr int kMaxSplits = 8;

// ---- joining a split product ------------------------------------------------------
// A thread adds eight columns' sums in split order and finishes them as above;
// four lanes hold a group of 32 columns.
template <typename T, LinearKind KIND>
__global__ __launch_bounds__(256) void k_linear_join(Linear a, int32_t splits) {
  const int32_t per_row = (a.cols + kAct8Group - 1) / kAct8Group * 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t wr = i / per_row;  // worker * rows + row
  const int32_t c = (int32_t)(i - wr * per_row) * 8;
  const int64_t pc = part_cols(a), all = a.n * a.rows;
  if (wr >= all) return;  // whole groups of lanes
  float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (c < a.cols) {
    lf4 x[kMaxSplits], y[kMaxSplits];
#pragma unroll
    for (int s = 0; s < kMaxSplits; ++s)  // all loads before the first sum
      if (s < splits) {
        const lf4* p = reinterpret_cast<const lf4*>(a.part + ((int64_t)s * all + wr) * pc + c);
        x[s] = p[0];
        y[s] = p[1];
      }
#pragma unroll
    for (int s = 0; s < kMaxSplits; ++s)
      if (s < splits)
        for (int j = 0; j < 4; ++j) {
          v[j] += x[s][j];
          v[4 + j] += y[s][j];
        }
  }
  if constexpr (KIND == LinearKind::kWeightGrad) {
    const int32_t worker = (int32_t)(wr / a.rows);
    const int64_t r = wr - worker * a.rows;
    if (c < a.cols) store_grad(a, grad_vec(a), worker, r, c, v);
    if (c == 0 && a.db) {
      float s = 0.0f;
      for (int32_t p = 0; p < splits; ++p)
        s += a.part[(int64_t)splits * all * pc + (int64_t)p * all + wr];
      store_bias_grad(a, worker, r, s);
    }
  } else {
    float b[8];
    Extra x;
    if constexpr (KIND == LinearKind::kForward) load_bias(a, c, b);
    load_extra<KIND>(a, wr, c, x);
    finish<T, KIND>(a, wr, c, b, x, v);
  }
}

// ---- host side ----------------------------------------------------------------------
constexpr int kCUs = 256;
constexpr int kTile = 128;

Tiles choose(int32_t n, int64_t rows, int32_t cols, int64_t k) {
  Tiles t;
  t.ta = (int32_t)((cols + kTile - 1) / kTile);
  t.tb = (int32_t)((rows + kTile - 1) / kTile);
  const int64_t all = (int64_t)t.ta * t.tb * n, steps = (k + kBK - 1) / kBK;
  int64_t splits = 1;
  // A product of few tiles: up to two blocks to a CU, at most kMaxSplits sums
  // to join, and at least four steps each, ten where the tiles alone give half
  // the CUs a block: the join moves each sum twice.  In us, with 5 of the
  // timing events: 256 x 4096 -> 1024 16 splits 26.4, 8 splits 21.3; 515 x 1000
  // -> 776 4 splits 17.7, 2 splits 20.5, none 28.3; 256 x 512 -> 512 2 splits
  // 12.6, none 15.2; 1024 x 1024 -> 3200 2 splits 32.9, none 25.2; 640 x 2048
  // -> 4096 2 splits 34.2, none 41.5.
  if (all > 0 && all <= kCUs) {
    const int64_t least = all <= kCUs / 2 ? 4 : 10;
    splits = std::max<int64_t>(
        1, std::min<int64_t>({2 * kCUs / all, steps / least, (int64_t)kMaxSplits}));
  }
  t.ksteps = (int32_t)std::max<int64_t>(1, (steps + splits - 1) / splits);
  t.splits = (int32_t)std::max<int64_t>(1, (steps + t.ksteps - 1) / t.ksteps);
  return t;
}

// Whether the few-rows kernel takes a forward product: one launch and no
// workspace, but cols / 32 blocks that each walk all of k, a batch of lines at
// a time.  Against the split tiles (us, with the 5 us of the timing events):
// 16 x 1600 -> 6400 10.4 and 16.4, 64 x 1600 -> 6400 15.8 and 18.9, 1 x 4096
// -> 1024 13.2 and 16.3; but 64 x 4096 -> 1024 27.8 and 18.5, 1 x 16384 -> 1024
// 40.6 and 33.2.  With a block for every CU a long k does no harm.
bool few(LinearKind kind, int64_t rows, int32_t cols, int64_t k) {
  if (kind != LinearKind::kForward || rows > 64) return false;
  return (k <= 4096 && rows * k <= 131072) || cols >= kCUs * kFewCols;
}

template <typename T>
void product_few(const Linear& a, hipStream_t st) {
  const dim3 grid((a.cols + kFewCols - 1) / kFewCols), block(kFewWaves * 64);
  if (a.rows <= 16) hipLaunchKernelGGL(HIP_KERNEL_NAME(k_linear_few<T, 1>), grid, block, 0, st, a);
  else if (a.rows <= 32)
    hipLaunchKernelGGL(HIP_KERNEL_NAME(k_linear_few<T, 2>), grid, block, 0, st, a);
  else hipLaunchKernelGGL(HIP_KERNEL_NAME(k_linear_few<T, 4>), grid, block, 0, st, a);
}

template <typename T, LinearKind KIND>
void product(const Linear& a, hipStream_t st) {
  const Tiles t = choose(a.n, a.rows, a.cols, a.k);
  const uint32_t grid = (uint32_t)linear_blocks(KIND, a.n, a.rows, a.cols, a.k);
  hipLaunchKernelGGL(HIP_KERNEL_NAME(k_linear<T, KIND, kTile, kTile, 2, 2>), dim3(grid), dim3(256),
                     0, st, a, t);
}

template <typename T, LinearKind KIND>
void join(const Linear& a, hipStream_t st) {
  const Tiles t = choose(a.n, a.rows, a.cols, a.k);
  const int64_t lanes = (int64_t)a.n * a.rows * ((a.cols + kAct8Group - 1) / kAct8Group) * 4;
  hipLaunchKernelGGL(HIP_KERNEL_NAME(k_linear_join<T, KIND>), dim3((uint32_t)((lanes + 255) / 256)),
                     dim3(256), 0, st, a, t.splits);
}

template <typename T>
void product(LinearKind kind, const Linear& a, hipStream_t st) {
  if (few(kind, a.rows, a.cols, a.k)) product_few<T>(a, st);
  else if (kind == LinearKind::kForward) product<T, LinearKind::kForward>(a, st);
  else if (kind == LinearKind::kInputGrad) product<T, LinearKind::kInputGrad>(a, st);
  else product<T, LinearKind::kWeightGrad>(a, st);
}

template <typename T>
void join(LinearKind kind, const Linear& a, hipStream_t st) {
  if (kind == LinearKind::kForward) join<T, LinearKind::kForward>(a, st);
  else if (kind == LinearKind::kInputGrad) join<T, LinearKind::kInputGrad>(a, st);
  else join<T, LinearKind::kWeightGrad>(a, st);
}

}  // namespace

int32_t linear_splits(LinearKind kind, int32_t n, int64_t rows, int32_t cols, int64_t k) {
  if (few(kind, rows, cols, k)) return 1;
  return choose(n, rows, cols, k).splits;
}

int64_t linear_blocks(LinearKind kind, int32_t n, int64_t rows, int32_t cols, int64_t k) {
  if (few(kind, rows, cols, k)) return (cols + kFewCols - 1) / kFewCols;
  const Tiles t = choose(n, rows, cols, k);
  return (int64_t)t.ta * t.tb * t.splits * n;
}

size_t linear_workspace(LinearKind kind, int32_t n, int64_t rows, int32_t cols, int64_t k) {
  const int32_t s = linear_splits(kind, n, rows, cols, k);
  if (s <= 1) return 0;
  const size_t pc = (size_t)(cols + 7) / 8 * 8;
  return (size_t)s * n * rows * (pc + (kind == LinearKind::kWeightGrad ? 1 : 0)) * 4;
}

void launch_linear(LinearKind kind, const Linear& a, hipStream_t st) {
  if (a.dtype == kGradF16) product<_Float16>(kind, a, st);
  else product<__bf16>(kind, a, st);
}

void launch_linear_join(LinearKind kind, const Linear& a, hipStream_t st) {
  if (a.dtype == kGradF16) join<_Float16>(kind, a, st);
  else join<__bf16>(kind, a, st);
}

}  // namespace oba
