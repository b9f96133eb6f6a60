// sublayer_kernels.hpp -- launch interface between the C ABI and the kernels of
// a gated feed-forward sub-layer: dropout, the join between two blocks, and the
// gated products.
#pragma once
#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "layer_kernels.hpp"

namespace oba {

// ---- dropout -------------------------------------------------------------------
struct Dropout {
  const uint64_t* rng;  // on the device: seed, step; not read for a threshold of 0
  uint32_t site;
  uint32_t threshold;   // of 65536; 0: nothing is dropped
  float scale;          // 65536 / (65536 - threshold)
};
// Blocks of a launch: 1024 pieces of 16 bytes of x each.
int64_t dropout_blocks(int64_t rows, int64_t cols, int dtype);
void launch_dropout(int64_t rows, int32_t cols, const void* x, int64_t ldx, int dtype,
                    const Dropout& d, const void* add, int64_t ldadd, void* y, int64_t ldy,
                    hipStream_t st);

// ---- the join between two blocks ----------------------------------------------
constexpr int kNormLayer = 0, kNormRms = 1;

struct JoinFwd {
  int64_t rows;
  int32_t cols;
  int dtype, kind;
  const void* x;
  int64_t ldx;
  float alpha;
  const void* b;       // the block's output, or null
  int64_t ldb;
  const float *gamma_b, *beta_b;  // the norm behind the block, or null
  const float* gate;   // or null
  Dropout drop;
  float eta;
  void* r;             // or null
  int64_t ldr;
  const float *gamma, *beta;      // the norm before the next block, or null
  void* z;
  int64_t ldz;
  float *rstd_b, *rstd;
  int8_t* qb;          // the branch kept: its normalised rows, or b; or null
  uint8_t* eb;
  int8_t* q;           // the normalised rows of r kept, or null
  uint8_t* e;
};
void launch_join(const JoinFwd& a, hipStream_t st);

struct JoinBwd {
  int32_t n;
  int64_t rows;        // per worker
  int32_t cols;
  int dtype, kind;
  const void* dz;      // with gamma, rstd, q, e; or null
  int64_t lddz;
  const void* dr;      // or null
  int64_t lddr;
  float alpha;
  const int8_t* q;
  const uint8_t* e;
  const float *rstd, *gamma;
  const int8_t* qb;    // or null
  const uint8_t* eb;
  const float *rstd_b, *gamma_b, *beta_b, *gate;
  Dropout drop;
  void* dx;
  int64_t lddx;
  void* db;            // or null
  int64_t lddb;
  // worker i's at + i * ldg elements, or null
  void *dgamma, *dbeta, *dgate, *dgamma_b, *dbeta_b;
  int g_dtype;
  int64_t ldg;
  float* part;         // [n][blocks][4][cols]: sums of dz * xhat, dz, e * bhat, e
};
// Blocks of the backward pass per worker.
int32_t join_bwd_blocks(int32_t n, int64_t rows, int32_t cols);
// columns of a partial sum: whole 16 bytes
__host__ __device__ inline int64_t join_part_cols(int64_t cols) { return (cols + 3) / 4 * 4; }
void launch_join_backward(const JoinBwd& a, hipStream_t st);
void launch_join_weight_grad(const JoinBwd& a, hipStream_t st);

// ---- gated products ---------------------------------------------------------------
// Forward: p = b wg^T + bias, u = b wu^T + bias, c = f(p) * u, both weights in
// `a` [2 * cols][k].  Hidden gradient: d = b a, a [k][cols]; c [rows][2 * cols] =
// [d * u * f'(p), d * f(p)].
struct Gated {
  int64_t rows;
  int32_t cols;         // hidden columns
  int64_t k;            // length of the sums
  const void* a;
  int64_t lda;
  const void* b;
  int64_t ldb;
  int dtype, gate;
  const float* bias;    // [2 * cols] or null
  int8_t *qp, *qu;      // pre-activations in 8 bits: kept (or null), or read
  uint8_t *ep, *eu;
  void* c;
  int64_t ldc;
  int8_t* q;            // the result in 8 bits, or null
  uint8_t* e;
  float* part;          // binary32 sums of a split product
};
enum class GatedKind { kForward, kHiddenGrad };
int32_t gated_splits(GatedKind kind, int64_t rows, int32_t cols, int64_t k);
size_t gated_workspace(GatedKind kind, int64_t rows, int32_t cols, int64_t k);
// Blocks of the product, were all of its tiles a block (what the limits are on).
int64_t gated_blocks(GatedKind kind, int64_t rows, int32_t cols, int64_t k);
void launch_gated(GatedKind kind, const Gated& a, hipStream_t st);
// Joins a split product's sums (launched after it when gated_splits > 1).
void launch_gated_join(GatedKind kind, const Gated& a, hipStream_t st);

}  // namespace oba
