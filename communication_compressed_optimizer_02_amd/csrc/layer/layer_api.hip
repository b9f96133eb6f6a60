// layer_api.hip -- the layer operators of include/oba.h: argument checks on
// the host and the launches.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "abi.hpp"
#include "layer_kernels.hpp"
#include "oba.h"

static_assert(OBA_ACT8_GROUP == oba::kAct8Group, "group size");

namespace {

using oba::LinearKind;

template <class F>
int launch(const char* name, hipStream_t st, F&& fn) {
  return oba::abi_launch(name, st, [](void* f) { (*static_cast<F*>(f))(); }, &fn);
}

bool is_type(int t) { return t == OBA_F32 || t == OBA_F16 || t == OBA_BF16; }
int size_of(int t) { return t == OBA_F32 ? 4 : 2; }

int check_ptr(const void* p, uintptr_t align) {
  if (!p) return OBA_EINVAL;
  return ((uintptr_t)p & (align - 1)) ? OBA_EALIGN : OBA_OK;
}

bool sizes_ok(int64_t rows, int64_t cols, int64_t most_cols) {
  return rows >= 0 && rows <= oba::kMaxRows && cols >= 1 && cols <= most_cols;
}
bool ld_ok(int64_t ld, int64_t cols) {
  return ld >= cols && ld % 8 == 0 && ld <= oba::kMaxLd;
}
// n workers of `rows` rows
bool workers_ok(int32_t n, int64_t rows) {
  return n >= 1 && n <= 4096 && rows >= 0 && rows <= oba::kMaxRows / n;
}
int check_kept(const int8_t* q, const uint8_t* e) {
  if (!q || !e) return OBA_EINVAL;
  return check_ptr(q, 16);
}
bool act_ok(int act) { return act >= OBA_ACT_NONE && act <= OBA_ACT_GELU_TANH; }

#define OBA_TRY(expr)              \
  do {                             \
    int rc_ = (expr);              \
    if (rc_ != OBA_OK) return rc_; \
  } while (0)

size_t norm_ws(int32_t n, int64_t rows, int64_t cols) {
  return (size_t)n * oba::norm_bwd_blocks(n, rows, (int32_t)cols) * 2 * cols * sizeof(float);
}

// Whether one launch walks the product's tiles.
bool blocks_ok(LinearKind kind, int32_t n, int64_t rows, int64_t cols, int64_t k) {
  return oba::linear_blocks(kind, n, rows, (int32_t)cols, k) <= oba::kMaxLaunch;
}

// The product, and the join of its sums where it was split.
int run_linear(const char* name, LinearKind kind, const oba::Linear& a, hipStream_t stream) {
  return launch(name, stream, [&] {
    oba::launch_linear(kind, a, stream);
    if (oba::linear_splits(kind, a.n, a.rows, a.cols, a.k) > 1)
      oba::launch_linear_join(kind, a, stream);
  });
}

int check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return OBA_OK;
  OBA_TRY(check_ptr(ws, 16));
  return have < need ? OBA_EWORKSPACE : OBA_OK;
}

}  // namespace

extern "C" {

int oba_act8_encode(int64_t rows, int64_t cols, const void* x, int64_t ldx, int dtype, int8_t* q,
                    uint8_t* e, hipStream_t stream) {
  if (!is_type(dtype) || !sizes_ok(rows, cols, oba::kMaxCols) || !ld_ok(ldx, cols) ||
      oba::act8_blocks(rows, cols, dtype) > oba::kMaxLaunch)
    return OBA_EINVAL;
  if (rows == 0) return OBA_OK;
  OBA_TRY(check_ptr(x, 16));
  OBA_TRY(check_kept(q, e));
  return launch("act8_encode", stream, [&] {
    oba::launch_act8_encode(rows, (int32_t)cols, x, ldx, dtype, q, e, stream);
  });
}

int oba_act8_decode(int64_t rows, int64_t cols, const int8_t* q, const uint8_t* e, void* x,
                    int64_t ldx, int dtype, hipStream_t stream) {
  if (!is_type(dtype) || !sizes_ok(rows, cols, oba::kMaxCols) || !ld_ok(ldx, cols) ||
      oba::act8_blocks(rows, cols, dtype) > oba::kMaxLaunch)
    return OBA_EINVAL;
  if (rows == 0) return OBA_OK;
  OBA_TRY(check_kept(q, e));
  OBA_TRY(check_ptr(x, 16));
  return launch("act8_decode", stream, [&] {
    oba::launch_act8_decode(rows, (int32_t)cols, q, e, x, ldx, dtype, stream);
  });
}

int oba_layer_norm(int64_t rows, int64_t cols, const void* x, int64_t ldx, int dtype,
                   const float* gamma, const float* beta, double eta, void* y, int64_t ldy,
                   float* mean, float* rstd, int8_t* q, uint8_t* e, hipStream_t stream) {
  if (!is_type(dtype) || !sizes_ok(rows, cols, oba::kMaxNormCols) || !ld_ok(ldx, cols) ||
      !ld_ok(ldy, cols) || !std::isfinite(eta) || eta < 0.0)
    return OBA_EINVAL;
  if (rows == 0) return OBA_OK;
  OBA_TRY(check_ptr(x, 16));
  OBA_TRY(check_ptr(gamma, 4));
  OBA_TRY(check_ptr(beta, 4));
  OBA_TRY(check_ptr(y, 16));
  OBA_TRY(check_ptr(mean, 4));
  OBA_TRY(check_ptr(rstd, 4));
  if (q || e) OBA_TRY(check_kept(q, e));
  const oba::NormFwd a{rows, (int32_t)cols, x, ldx, dtype, gamma, beta, (float)eta,
                       y, ldy, mean, rstd, q, e};
  return launch("layer_norm", stream, [&] { oba::launch_layer_norm(a, stream); });
}

size_t oba_layer_norm_backward_workspace_bytes(int32_t n, int64_t rows, int64_t cols) {
  if (!workers_ok(n, rows) || cols < 1 || cols > oba::kMaxNormCols) return 0;
  return norm_ws(n, rows, cols);
}

int oba_layer_norm_backward(int32_t n, int64_t rows, int64_t cols, const void* dy, int64_t lddy,
                            int dtype, const void* x, int64_t ldx, const float* mean,
                            const int8_t* q, const uint8_t* e, const float* rstd,
                            const float* gamma, const void* add, int64_t ldadd, void* dx,
                            int64_t lddx, void* dgamma, void* dbeta, int g_dtype, int64_t ldg,
                            void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!is_type(dtype) || !is_type(g_dtype) || !workers_ok(n, rows) ||
      !sizes_ok(n * rows, cols, oba::kMaxNormCols))
    return OBA_EINVAL;
  const bool kept = !x;
  // the rows with their means, or the kept normalised rows
  if (rows > 0 && (kept != !mean || kept == !q || kept == !e)) return OBA_EINVAL;
  if (!ld_ok(lddy, cols) || !ld_ok(lddx, cols) || (!kept && !ld_ok(ldx, cols)) ||
      (add && !ld_ok(ldadd, cols)) || (n > 1 && ldg < cols))
    return OBA_EINVAL;
  OBA_TRY(check_ptr(dgamma, size_of(g_dtype)));
  OBA_TRY(check_ptr(dbeta, size_of(g_dtype)));
  if (rows > 0) {
    OBA_TRY(check_ptr(dy, 16));
    if (kept) {
      OBA_TRY(check_kept(q, e));
    } else {
      OBA_TRY(check_ptr(x, 16));
      OBA_TRY(check_ptr(mean, 4));
    }
    OBA_TRY(check_ptr(rstd, 4));
    OBA_TRY(check_ptr(gamma, 4));
    if (add) OBA_TRY(check_ptr(add, 16));
    OBA_TRY(check_ptr(dx, 16));
    OBA_TRY(check_ws(ws, ws_bytes, norm_ws(n, rows, cols)));
  }
  const oba::NormBwd a{n, rows, (int32_t)cols, dy, lddy, dtype, x, ldx, mean, q, e, rstd, gamma,
                       add, ldadd, dx, lddx, dgamma, dbeta, g_dtype, ldg,
                       static_cast<float*>(ws)};
  return launch("layer_norm_backward", stream, [&] {
    if (rows > 0) oba::launch_layer_norm_backward(a, stream);
    oba::launch_layer_norm_weight_grad(a, stream);  // zeros for no rows
  });
}

size_t oba_linear_workspace_bytes(int64_t rows, int64_t in, int64_t out) {
  if (!sizes_ok(rows, in, oba::kMaxCols) || !sizes_ok(rows, out, oba::kMaxCols)) return 0;
  const size_t f = oba::linear_workspace(LinearKind::kForward, 1, rows, (int32_t)out, in);
  const size_t g = oba::linear_workspace(LinearKind::kInputGrad, 1, rows, (int32_t)in, out);
  return f > g ? f : g;
}

int oba_linear(int64_t rows, int64_t in, int64_t out, const void* x, int64_t ldx, const void* w,
               int64_t ldw, int dtype, const float* bias, int act, const void* residual,
               int64_t ldr, void* y, int64_t ldy, int8_t* q, uint8_t* e, void* ws,
               size_t ws_bytes, hipStream_t stream) {
  if ((dtype != OBA_F16 && dtype != OBA_BF16) || !act_ok(act) ||
      !sizes_ok(rows, in, oba::kMaxCols) || !sizes_ok(rows, out, oba::kMaxCols) ||
      !blocks_ok(LinearKind::kForward, 1, rows, out, in) || !ld_ok(ldx, in) || !ld_ok(ldw, in) ||
      !ld_ok(ldy, out) || (residual && !ld_ok(ldr, out)))
    return OBA_EINVAL;
  if (rows == 0) return OBA_OK;
  OBA_TRY(check_ptr(x, 16));
  OBA_TRY(check_ptr(w, 16));
  if (bias) OBA_TRY(check_ptr(bias, 4));
  if (residual) OBA_TRY(check_ptr(residual, 16));
  OBA_TRY(check_ptr(y, 16));
  if (q || e) OBA_TRY(check_kept(q, e));
  OBA_TRY(check_ws(ws, ws_bytes,
                   oba::linear_workspace(LinearKind::kForward, 1, rows, (int32_t)out, in)));
  oba::Linear a{};
  a.n = 1;
  a.rows = rows;
  a.cols = (int32_t)out;
  a.k = in;
  a.a = w;
  a.lda = ldw;
  a.b = x;
  a.ldb = ldx;
  a.dtype = dtype;
  a.bias = bias;
  a.act = act;
  a.add = residual;
  a.ldadd = ldr;
  a.c = y;
  a.ldc = ldy;
  a.q = q;
  a.e = e;
  a.part = static_cast<float*>(ws);
  return run_linear("linear", LinearKind::kForward, a, stream);
}

int oba_linear_input_grad(int64_t rows, int64_t in, int64_t out, const void* dy, int64_t lddy,
                          const void* w, int64_t ldw, int dtype, int act, const int8_t* q,
                          const uint8_t* e, const void* add, int64_t ldadd, void* dx,
                          int64_t lddx, void* ws, size_t ws_bytes, hipStream_t stream) {
  if ((dtype != OBA_F16 && dtype != OBA_BF16) || !act_ok(act) ||
      !sizes_ok(rows, in, oba::kMaxCols) || !sizes_ok(rows, out, oba::kMaxCols) ||
      !blocks_ok(LinearKind::kInputGrad, 1, rows, in, out) || !ld_ok(lddy, out) ||
      !ld_ok(ldw, in) || !ld_ok(lddx, in) || (add && !ld_ok(ldadd, in)))
    return OBA_EINVAL;
  if (rows == 0) return OBA_OK;
  // a derivative needs the kept pre-activation, and none is read without one
  if ((act == OBA_ACT_NONE) != !q || (act == OBA_ACT_NONE) != !e) return OBA_EINVAL;
  OBA_TRY(check_ptr(dy, 16));
  OBA_TRY(check_ptr(w, 16));
  if (q) OBA_TRY(check_kept(q, e));
  if (add) OBA_TRY(check_ptr(add, 16));
  OBA_TRY(check_ptr(dx, 16));
  OBA_TRY(check_ws(ws, ws_bytes,
                   oba::linear_workspace(LinearKind::kInputGrad, 1, rows, (int32_t)in, out)));
  oba::Linear a{};
  a.n = 1;
  a.rows = rows;
  a.cols = (int32_t)in;
  a.k = out;
  a.a = w;
  a.lda = ldw;
  a.b = dy;
  a.ldb = lddy;
  a.dtype = dtype;
  a.act = act;
  a.pq = q;
  a.pe = e;
  a.add = add;
  a.ldadd = ldadd;
  a.c = dx;
  a.ldc = lddx;
  a.part = static_cast<float*>(ws);
  return run_linear("linear_input_grad", LinearKind::kInputGrad, a, stream);
}

size_t oba_linear_weight_grad_workspace_bytes(int32_t n, int64_t rows, int64_t in, int64_t out) {
  if (!workers_ok(n, rows) || !sizes_ok(n * rows, in, oba::kMaxCols) ||
      !sizes_ok(n * rows, out, oba::kMaxCols) || !sizes_ok(out * (int64_t)n, in, oba::kMaxCols))
    return 0;
  return oba::linear_workspace(LinearKind::kWeightGrad, n, out, (int32_t)in, rows);
}

int oba_linear_weight_grad(int32_t n, int64_t rows, int64_t in, int64_t out, const void* dy,
                           int64_t lddy, int dtype, const int8_t* q, const uint8_t* e, void* dw,
                           void* db, int g_dtype, int64_t ldg, void* ws, size_t ws_bytes,
                           hipStream_t stream) {
  if ((dtype != OBA_F16 && dtype != OBA_BF16) || !is_type(g_dtype) || !workers_ok(n, rows) ||
      !sizes_ok(n * rows, in, oba::kMaxCols) || !sizes_ok(n * rows, out, oba::kMaxCols) ||
      !sizes_ok(out * (int64_t)n, in, oba::kMaxCols) ||
      !blocks_ok(LinearKind::kWeightGrad, n, out, in, rows) || !ld_ok(lddy, out) ||
      (n > 1 && ldg < in * out))
    return OBA_EINVAL;
  OBA_TRY(check_ptr(dw, size_of(g_dtype)));
  if (db) OBA_TRY(check_ptr(db, size_of(g_dtype)));
  if (rows > 0) {
    OBA_TRY(check_ptr(dy, 16));
    OBA_TRY(check_kept(q, e));
  }
  const size_t need = oba::linear_workspace(LinearKind::kWeightGrad, n, out, (int32_t)in, rows);
  OBA_TRY(check_ws(ws, ws_bytes, need));
  const int64_t groups = (in + OBA_ACT8_GROUP - 1) / OBA_ACT8_GROUP;
  oba::Linear a{};
  a.n = n;
  a.rows = out;
  a.cols = (int32_t)in;
  a.k = rows;
  a.a = q;
  a.lda = groups * OBA_ACT8_GROUP;
  a.ae = e;
  a.b = dy;
  a.ldb = lddy;
  a.dtype = dtype;
  a.c = dw;
  a.g_dtype = g_dtype;
  a.ldg = ldg;
  a.db = db;
  a.part = static_cast<float*>(ws);
  return run_linear("linear_weight_grad", LinearKind::kWeightGrad, a, stream);
}

}  // extern "C"
