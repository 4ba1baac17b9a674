// qmv_checks.h -- argument checks that the many-row calls of the C ABI share.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/qmv.h"
#include "qmv_internal.h"

namespace qmv {

inline bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

template <typename... P>
bool any_null(const P*... p) {
  return ((p == nullptr) || ...);
}
template <typename... P>
bool any_misaligned(const P*... p) {
  return (misaligned(p) || ...);
}

inline int launched(cudaError_t e, const char* name) {
  if (e == cudaSuccess) return record_error(QMV_OK, "%s", "");
  cudaGetLastError();   // clear a non-sticky error so later calls start clean
  return record_error(QMV_ECUDA, "%s: %s failed: %s (%s)", name, g_launch_stage, cudaGetErrorName(e),
                      cudaGetErrorString(e));
}
inline int done() { return record_error(QMV_OK, "%s", ""); }

inline int check_type(int type, const char* name) {
  if (type < QMV_BF16 || type > QMV_F32) return record_error(QMV_EINVAL, "%s: unknown element type %d", name, type);
  return QMV_OK;
}

inline int check_width(int K, bool groups, const char* name, int most = QMV_MAX_K) {
  if (K < 1 || K > most) return record_error(QMV_ESHAPE, "%s: %d columns outside [1, %d]", name, K, most);
  if (groups && K % 32) return record_error(QMV_ESHAPE, "%s: %d columns are not a multiple of 32", name, K);
  return QMV_OK;
}

inline int check_ld(int64_t ld, int K, const char* name) {
  if (ld < K || ld > (int64_t)1 << 40)
    return record_error(QMV_ESHAPE, "%s: row stride %lld for %d columns", name, (long long)ld, K);
  return QMV_OK;
}

inline int check_rows(int nrows, const char* name) {
  if (nrows < 0 || nrows > QMV_MAX_ROWS)
    return record_error(QMV_EINVAL, "%s: %d rows outside [0, %d]", name, nrows, QMV_MAX_ROWS);
  return QMV_OK;
}

inline int check_slots(int ntok, int top_k, const char* name) {
  if (top_k < 1 || top_k > QMV_MAX_TOPK)
    return record_error(QMV_EINVAL, "%s: top_k=%d outside [1, %d]", name, top_k, QMV_MAX_TOPK);
  if (ntok < 0 || (int64_t)ntok * top_k > QMV_MAX_ROWS)
    return record_error(QMV_EINVAL, "%s: ntok=%d with top_k=%d: at most %d slots", name, ntok, top_k, QMV_MAX_ROWS);
  return QMV_OK;
}

#define QMV_TRY(call)             \
  do {                            \
    const int rc_ = (call);       \
    if (rc_ != QMV_OK) return rc_; \
  } while (0)

inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace qmv
