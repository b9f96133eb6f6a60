// sublayer_api.hip -- the operators of a gated feed-forward sub-layer of
// include/oba.h: argument checks on the host and the launches.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "checks.hpp"
#include "oba.h"
#include "sublayer_kernels.hpp"

static_assert(OBA_NORM_LAYER == oba::kNormLayer && OBA_NORM_RMS == oba::kNormRms, "norm kinds");

namespace {

using oba::GatedKind;

// The dropout of a call; whether its arguments are good.
bool make_dropout(double rate, const uint64_t* rng, uint32_t site, oba::Dropout& d) {
  if (!(rate >= 0.0 && rate < 1.0)) return false;
  const uint32_t t = (uint32_t)std::floor(rate * 65536.0 + 0.5);
  if (t >= 65536u) return false;
  d = oba::Dropout{rng, site, t, (float)(65536.0 / (65536.0 - t))};
  return true;
}
int check_rng(const oba::Dropout& d) { return d.threshold ? check_ptr(d.rng, 8) : OBA_OK; }

bool kind_ok(int kind) { return kind == OBA_NORM_LAYER || kind == OBA_NORM_RMS; }
// a pointer that may be null
int check_opt(const void* p, uintptr_t align) { return p ? check_ptr(p, align) : OBA_OK; }

size_t join_ws(int32_t n, int64_t rows, int64_t cols) {
  return (size_t)n * oba::join_bwd_blocks(n, rows, (int32_t)cols) * 4 * oba::join_part_cols(cols) *
         sizeof(float);
}

bool gated_ok(GatedKind kind, int dtype, int gate, int64_t rows, int64_t hidden, int64_t k) {
  return (dtype == OBA_F16 || dtype == OBA_BF16) && gate >= OBA_GATE_NONE &&
         gate <= OBA_GATE_SIGMOID && sizes_ok(rows, hidden, oba::kMaxCols / 2) &&
         sizes_ok(rows, k, oba::kMaxCols) &&
         oba::gated_blocks(kind, rows, (int32_t)hidden, k) <= oba::kMaxLaunch;
}

int run_gated(const char* name, GatedKind kind, const oba::Gated& a, hipStream_t stream) {
  return launch(name, stream, [&] {
    oba::launch_gated(kind, a, stream);
    if (oba::gated_splits(kind, a.rows, a.cols, a.k) > 1) oba::launch_gated_join(kind, a, stream);
  });
}

}  // namespace

extern "C" {

int oba_dropout(int64_t rows, int64_t cols, const void* x, int64_t ldx, int dtype, double rate,
                const uint64_t* rng, uint32_t site, const void* add, int64_t ldadd, void* y,
                int64_t ldy, hipStream_t stream) {
  oba::Dropout d;
  if (!is_type(dtype) || !sizes_ok(rows, cols, oba::kMaxCols) || !ld_ok(ldx, cols) ||
      !ld_ok(ldy, cols) || (add && !ld_ok(ldadd, cols)) || !make_dropout(rate, rng, site, d) ||
      oba::dropout_blocks(rows, cols, dtype) > oba::kMaxLaunch)
    return OBA_EINVAL;
  if (rows == 0) return OBA_OK;
  OBA_TRY(check_ptr(x, 16));
  OBA_TRY(check_opt(add, 16));
  OBA_TRY(check_ptr(y, 16));
  OBA_TRY(check_rng(d));
  return launch("dropout", stream, [&] {
    oba::launch_dropout(rows, (int32_t)cols, x, ldx, dtype, d, add, ldadd, y, ldy, stream);
  });
}

int oba_residual_norm(int64_t rows, int64_t cols, int dtype, int kind, double eta, const void* x,
                      int64_t ldx, double alpha, const void* b, int64_t ldb, const float* gamma_b,
                      const float* beta_b, const float* gate, double rate, const uint64_t* rng,
                      uint32_t site, float* rstd_b, int8_t* qb, uint8_t* eb, void* r, int64_t ldr,
                      const float* gamma, const float* beta, void* z, int64_t ldz, float* rstd,
                      int8_t* q, uint8_t* e, hipStream_t stream) {
  oba::Dropout d;
  if (!is_type(dtype) || !kind_ok(kind) || !sizes_ok(rows, cols, oba::kMaxNormCols) ||
      !std::isfinite((float)eta) || eta < 0.0 || !std::isfinite((float)alpha) ||
      !ld_ok(ldx, cols) ||
      (b && !ld_ok(ldb, cols)) || (r && !ld_ok(ldr, cols)) || (gamma && !ld_ok(ldz, cols)) ||
      !make_dropout(rate, rng, site, d))
    return OBA_EINVAL;
  if (rows == 0) return OBA_OK;
  // what belongs to the branch needs one; what belongs to a norm needs its gamma
  if (!b && (gamma_b || beta_b || gate || rstd_b || qb || eb || d.threshold)) return OBA_EINVAL;
  if ((!gamma_b && (beta_b || rstd_b)) || (!gamma && (beta || z || rstd || q || e)) ||
      (!gamma && !r))
    return OBA_EINVAL;
  OBA_TRY(check_ptr(x, 16));
  OBA_TRY(check_opt(b, 16));
  OBA_TRY(check_opt(gate, 4));
  if (gamma_b) {
    OBA_TRY(check_ptr(gamma_b, 4));
    OBA_TRY(check_opt(beta_b, 4));
    OBA_TRY(check_ptr(rstd_b, 4));
  }
  if (qb || eb) OBA_TRY(check_kept(qb, eb));
  OBA_TRY(check_rng(d));
  OBA_TRY(check_opt(r, 16));
  if (gamma) {
    OBA_TRY(check_ptr(gamma, 4));
    OBA_TRY(check_opt(beta, 4));
    OBA_TRY(check_ptr(z, 16));
    OBA_TRY(check_ptr(rstd, 4));
  }
  if (q || e) OBA_TRY(check_kept(q, e));
  const oba::JoinFwd a{rows, (int32_t)cols, dtype, kind, x, ldx, (float)alpha, b, ldb,
                       gamma_b, beta_b, gate, d, (float)eta, r, ldr, gamma, beta,
                       z, ldz, rstd_b, rstd, qb, eb, q, e};
  return launch("residual_norm", stream, [&] { oba::launch_join(a, stream); });
}

size_t oba_residual_norm_backward_workspace_bytes(int32_t n, int64_t rows, int64_t cols) {
  if (!workers_ok(n, rows) || cols < 1 || cols > oba::kMaxNormCols) return 0;
  return join_ws(n, rows, cols);
}

int oba_residual_norm_backward(int32_t n, int64_t rows, int64_t cols, int dtype, int kind,
                               const void* dz, int64_t lddz, const int8_t* q, const uint8_t* e,
                               const float* rstd, const float* gamma, const void* dr,
                               int64_t lddr, double alpha, void* dx, int64_t lddx,
                               const int8_t* qb, const uint8_t* eb, const float* rstd_b,
                               const float* gamma_b, const float* beta_b, const float* gate,
                               double rate, const uint64_t* rng, uint32_t site, void* db,
                               int64_t lddb, void* dgamma, void* dbeta, void* dgamma_b,
                               void* dbeta_b, void* dgate, int g_dtype, int64_t ldg, void* ws,
                               size_t ws_bytes, hipStream_t stream) {
  oba::Dropout d;
  if (!is_type(dtype) || !is_type(g_dtype) || !kind_ok(kind) || !workers_ok(n, rows) ||
      !sizes_ok(n * rows, cols, oba::kMaxNormCols) || !std::isfinite((float)alpha) ||
      !ld_ok(lddx, cols) || (gamma && !ld_ok(lddz, cols)) || (dr && !ld_ok(lddr, cols)) ||
      (db && !ld_ok(lddb, cols)) || !make_dropout(rate, rng, site, d))
    return OBA_EINVAL;
  void* const grads[] = {dgamma, dbeta, dgamma_b, dbeta_b, dgate};
  bool any = false;
  for (void* g : grads) any = any || g;
  if (any && n > 1 && ldg < cols) return OBA_EINVAL;
  // what belongs to a norm needs its gamma, the gate's gradient the gate
  if ((!gamma && (dgamma || dbeta)) || (!gamma_b && (beta_b || dgamma_b || dbeta_b)) ||
      (!gate && dgate))
    return OBA_EINVAL;
  for (void* g : grads) OBA_TRY(check_opt(g, size_of(g_dtype)));
  // read for the parameters' gradients also where there are no rows
  OBA_TRY(check_opt(gamma_b, 4));
  OBA_TRY(check_opt(beta_b, 4));
  OBA_TRY(check_opt(gate, 4));
  if (rows > 0) {
    if ((!gamma && (dz || q || e || rstd)) || (!gamma_b && rstd_b) || (!gamma && !dr))
      return OBA_EINVAL;
    // the branch as kept: for its norm's gradient and its parameters'
    if ((gamma_b || dgate) && !qb) return OBA_EINVAL;
    if (gamma) {
      OBA_TRY(check_ptr(gamma, 4));
      OBA_TRY(check_ptr(dz, 16));
      OBA_TRY(check_kept(q, e));
      OBA_TRY(check_ptr(rstd, 4));
    }
    OBA_TRY(check_opt(dr, 16));
    OBA_TRY(check_ptr(dx, 16));
    if (qb || eb) OBA_TRY(check_kept(qb, eb));
    if (gamma_b) OBA_TRY(check_ptr(rstd_b, 4));
    OBA_TRY(check_rng(d));
    OBA_TRY(check_opt(db, 16));
    if (any) OBA_TRY(check_ws(ws, ws_bytes, join_ws(n, rows, cols)));
  }
  const oba::JoinBwd a{n, rows, (int32_t)cols, dtype, kind, dz, lddz, dr, lddr, (float)alpha,
                       q, e, rstd, gamma, qb, eb, rstd_b, gamma_b, beta_b, gate, d, dx, lddx, db,
                       lddb, dgamma, dbeta, dgate, dgamma_b, dbeta_b, g_dtype, ldg,
                       any ? static_cast<float*>(ws) : nullptr};
  if (rows == 0 && !any) return OBA_OK;
  return launch("residual_norm_backward", stream, [&] {
    if (rows > 0) oba::launch_join_backward(a, stream);
    if (any) oba::launch_join_weight_grad(a, stream);  // zeros for no rows
  });
}

size_t oba_gated_linear_workspace_bytes(int64_t rows, int64_t in, int64_t hidden) {
  if (!sizes_ok(rows, in, oba::kMaxCols) || !sizes_ok(rows, hidden, oba::kMaxCols / 2)) return 0;
  return oba::gated_workspace(GatedKind::kForward, rows, (int32_t)hidden, in);
}

int oba_gated_linear(int64_t rows, int64_t in, int64_t hidden, const void* x, int64_t ldx,
                     const void* w, int64_t ldw, int dtype, const float* bias, int gate, void* y,
                     int64_t ldy, int8_t* qp, uint8_t* ep, int8_t* qu, uint8_t* eu, int8_t* q,
                     uint8_t* e, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!gated_ok(GatedKind::kForward, dtype, gate, rows, hidden, in) || !ld_ok(ldx, in) ||
      !ld_ok(ldw, in) || !ld_ok(ldy, hidden))
    return OBA_EINVAL;
  if (rows == 0) return OBA_OK;
  OBA_TRY(check_ptr(x, 16));
  OBA_TRY(check_ptr(w, 16));
  OBA_TRY(check_opt(bias, 4));
  OBA_TRY(check_ptr(y, 16));
  if (qp || ep || qu || eu) {  // both pre-activations or neither
    OBA_TRY(check_kept(qp, ep));
    OBA_TRY(check_kept(qu, eu));
  }
  if (q || e) OBA_TRY(check_kept(q, e));
  OBA_TRY(check_ws(ws, ws_bytes, oba_gated_linear_workspace_bytes(rows, in, hidden)));
  oba::Gated a{};
  a.rows = rows;
  a.cols = (int32_t)hidden;
  a.k = in;
  a.a = w;
  a.lda = ldw;
  a.b = x;
  a.ldb = ldx;
  a.dtype = dtype;
  a.gate = gate;
  a.bias = bias;
  a.qp = qp;
  a.ep = ep;
  a.qu = qu;
  a.eu = eu;
  a.c = y;
  a.ldc = ldy;
  a.q = q;
  a.e = e;
  a.part = static_cast<float*>(ws);
  return run_gated("gated_linear", GatedKind::kForward, a, stream);
}

size_t oba_gated_hidden_grad_workspace_bytes(int64_t rows, int64_t hidden, int64_t out) {
  if (!sizes_ok(rows, out, oba::kMaxCols) || !sizes_ok(rows, hidden, oba::kMaxCols / 2)) return 0;
  return oba::gated_workspace(GatedKind::kHiddenGrad, rows, (int32_t)hidden, out);
}

int oba_gated_hidden_grad(int64_t rows, int64_t hidden, int64_t out, const void* dy, int64_t lddy,
                          const void* w, int64_t ldw, int dtype, int gate, const int8_t* qp,
                          const uint8_t* ep, const int8_t* qu, const uint8_t* eu, void* dpu,
                          int64_t lddpu, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!gated_ok(GatedKind::kHiddenGrad, dtype, gate, rows, hidden, out) || !ld_ok(lddy, out) ||
      !ld_ok(ldw, hidden) || !ld_ok(lddpu, 2 * hidden))
    return OBA_EINVAL;
  if (rows == 0) return OBA_OK;
  OBA_TRY(check_ptr(dy, 16));
  OBA_TRY(check_ptr(w, 16));
  OBA_TRY(check_kept(qp, ep));
  OBA_TRY(check_kept(qu, eu));
  OBA_TRY(check_ptr(dpu, 16));
  OBA_TRY(check_ws(ws, ws_bytes, oba_gated_hidden_grad_workspace_bytes(rows, hidden, out)));
  oba::Gated a{};
  a.rows = rows;
  a.cols = (int32_t)hidden;
  a.k = out;
  a.a = w;
  a.lda = ldw;
  a.b = dy;
  a.ldb = lddy;
  a.dtype = dtype;
  a.gate = gate;
  a.qp = const_cast<int8_t*>(qp);
  a.ep = const_cast<uint8_t*>(ep);
  a.qu = const_cast<int8_t*>(qu);
  a.eu = const_cast<uint8_t*>(eu);
  a.c = dpu;
  a.ldc = lddpu;
  a.part = static_cast<float*>(ws);
  return run_gated("gated_hidden_grad", GatedKind::kHiddenGrad, a, stream);
}

}  // extern "C"
