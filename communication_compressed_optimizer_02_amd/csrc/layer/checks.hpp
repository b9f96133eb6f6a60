// checks.hpp -- argument checks and launches that the layer operators' entry
// points share (layer_api.hip, sublayer_api.hip).
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "abi.hpp"
#include "layer_kernels.hpp"
#include "oba.h"

namespace {

template <class F>
int launch(const char* name, hipStream_t st, F&& fn) {
  return oba::abi_launch(name, st, [](void* f) { (*static_cast<F*>(f))(); }, &fn);
}

inline bool is_type(int t) { return t == OBA_F32 || t == OBA_F16 || t == OBA_BF16; }
inline int size_of(int t) { return t == OBA_F32 ? 4 : 2; }

inline int check_ptr(const void* p, uintptr_t align) {
  if (!p) return OBA_EINVAL;
  return ((uintptr_t)p & (align - 1)) ? OBA_EALIGN : OBA_OK;
}

inline bool sizes_ok(int64_t rows, int64_t cols, int64_t most_cols) {
  return rows >= 0 && rows <= oba::kMaxRows && cols >= 1 && cols <= most_cols;
}
inline bool ld_ok(int64_t ld, int64_t cols) {
  return ld >= cols && ld % 8 == 0 && ld <= oba::kMaxLd;
}
// n workers of `rows` rows
inline bool workers_ok(int32_t n, int64_t rows) {
  return n >= 1 && n <= 4096 && rows >= 0 && rows <= oba::kMaxRows / n;
}
inline int check_kept(const int8_t* q, const uint8_t* e) {
  if (!q || !e) return OBA_EINVAL;
  return check_ptr(q, 16);
}
inline bool act_ok(int act) { return act >= OBA_ACT_NONE && act <= OBA_ACT_GELU_TANH; }

#define OBA_TRY(expr)              \
  do {                             \
    int rc_ = (expr);              \
    if (rc_ != OBA_OK) return rc_; \
  } while (0)

inline int check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return OBA_OK;
  OBA_TRY(check_ptr(ws, 16));
  return have < need ? OBA_EWORKSPACE : OBA_OK;
}

}  // namespace
