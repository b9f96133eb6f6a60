// layer_kernels.hpp -- launch interface between the C ABI and the layer
// operators' kernels, and the host-side choices (grids, splits, workspaces)
// that both share.
#pragma once
#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "kernels.hpp"

namespace oba {

constexpr int kAct8Group = 32;  // columns that share a step (OBA_ACT8_GROUP)

// Limits of the entry points: sizes stay in 32 bits, products of two in 64.
constexpr int64_t kMaxCols = 1 << 20;       // columns of a kept or linear matrix
constexpr int64_t kMaxNormCols = 16384;     // columns of a layer norm (a row stays in registers)
constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr int64_t kMaxLd = 1 << 22;         // a tile's element offsets stay in 32 bits
// HIP takes fewer than 2^32 threads in a launch: blocks of 256 of the kernels
// that have one for each part of their result (the norms' grids do not grow
// with the rows)
constexpr int64_t kMaxLaunch = ((int64_t)1 << 24) - 1;

// Blocks of an encode or decode: 1024 pieces of 16 bytes of x each.
int64_t act8_blocks(int64_t rows, int64_t cols, int dtype);
void launch_act8_encode(int64_t rows, int32_t cols, const void* x, int64_t ldx, int dtype,
                        int8_t* q, uint8_t* e, hipStream_t st);
void launch_act8_decode(int64_t rows, int32_t cols, const int8_t* q, const uint8_t* e, void* x,
                        int64_t ldx, int dtype, hipStream_t st);

// ---- layer norm --------------------------------------------------------------
struct NormFwd {
  int64_t rows;
  int32_t cols;
  const void* x;
  int64_t ldx;
  int dtype;
  const float *gamma, *beta;
  float eta;
  void* y;
  int64_t ldy;
  float *mean, *rstd;
  int8_t* q;   // kept normalised rows, or null
  uint8_t* e;
};
void launch_layer_norm(const NormFwd& a, hipStream_t st);

struct NormBwd {
  int32_t n;
  int64_t rows;  // per worker
  int32_t cols;
  const void* dy;
  int64_t lddy;
  int dtype;
  const void* x;  // the rows (with mean), or null: q, e
  int64_t ldx;
  const float* mean;
  const int8_t* q;
  const uint8_t* e;
  const float *rstd, *gamma;
  const void* add;  // or null
  int64_t ldadd;
  void* dx;
  int64_t lddx;
  void *dgamma, *dbeta;  // worker i's at + i * ldg elements
  int g_dtype;
  int64_t ldg;
  float* part;  // [n][blocks][2][cols]
};
// Blocks of the backward pass per worker.
int32_t norm_bwd_blocks(int32_t n, int64_t rows, int32_t cols);
void launch_layer_norm_backward(const NormBwd& a, hipStream_t st);
void launch_layer_norm_weight_grad(const NormBwd& a, hipStream_t st);

// ---- linear layers -------------------------------------------------------------
struct Linear {
  int32_t n;        // products in the call (workers; 1 but for the weight gradient)
  int64_t rows;     // rows of the result of one product
  int32_t cols;     // columns of the result
  int64_t k;        // length of the sums
  const void* a;    // the operand that the result's columns come from
  int64_t lda;
  const uint8_t* ae;  // its exponents, where it is kept in 8 bits
  const void* b;    // the operand that the result's rows come from
  int64_t ldb;
  int dtype;
  const float* bias;   // [cols] or null
  int act;
  const int8_t* pq;    // pre-activation of the derivative, or null
  const uint8_t* pe;
  const void* add;     // residual, or null
  int64_t ldadd;
  void* c;
  int64_t ldc;
  int8_t* q;           // kept pre-activation, or null
  uint8_t* e;
  int g_dtype;         // the weight gradient's type
  int64_t ldg;         // and the stride of the workers' gradient rows
  void* db;            // bias gradient, or null
  float* part;         // binary32 sums of a split product
};
enum class LinearKind { kForward, kInputGrad, kWeightGrad };
size_t linear_workspace(LinearKind kind, int32_t n, int64_t rows, int32_t cols, int64_t k);
// Blocks of the product.
int64_t linear_blocks(LinearKind kind, int32_t n, int64_t rows, int32_t cols, int64_t k);
void launch_linear(LinearKind kind, const Linear& a, hipStream_t st);
// Joins a split product's sums (launched after it when linear_splits > 1).
int32_t linear_splits(LinearKind kind, int32_t n, int64_t rows, int32_t cols, int64_t k);
void launch_linear_join(LinearKind kind, const Linear& a, hipStream_t st);

}  // namespace oba
