// qmv_train_api.cpp -- the C ABI (include/qmv.h) of the router with its balance
// loss, and of the products with a scale for each block of 128, with their
// gradients: argument checks and dispatch to the launchers. Nothing here reads
// device memory or synchronizes. Without rows (an empty tensor's address is
// NULL) only what does not depend on them has to be there.
#include <cmath>
#include <cstring>

#include "qmv_checks.h"
#include "qmv_layout.h"

namespace qmv {
namespace {

int check_router(int type, int64_t ldl, int ntok, int n_experts, int top_k, int score, const char* name) {
  QMV_TRY(check_type(type, name));
  QMV_TRY(check_slots(ntok, top_k, name));
  if (n_experts < 1 || n_experts > QMV_MAX_SORT_EXPERTS)
    return record_error(QMV_EINVAL, "%s: n_experts=%d outside [1, %d]", name, n_experts, QMV_MAX_SORT_EXPERTS);
  if (top_k > n_experts) return record_error(QMV_EINVAL, "%s: top_k=%d of %d experts", name, top_k, n_experts);
  if (score != QMV_SCORE_SOFTMAX && score != QMV_SCORE_SIGMOID)
    return record_error(QMV_EINVAL, "%s: unknown score %d", name, score);
  return check_ld(ldl, n_experts, name);
}

int check_scale(float scale, const char* name) {
  if (std::isnan(scale) || std::isinf(scale)) return record_error(QMV_EINVAL, "%s: scale=%g", name, (double)scale);
  return QMV_OK;
}

// Parts of the balance loss's workspace.
struct BalanceSpace {
  int parts;
  size_t sums, counts, total;
};
BalanceSpace balance_space(int ntok, int n_experts) {
  BalanceSpace s;
  s.parts = balance_parts(ntok);
  s.sums = 0;
  s.counts = up256((size_t)s.parts * n_experts * 4);
  s.total = s.counts + up256((size_t)s.parts * (n_experts + 1) * 4);
  return s;
}

// N and K of a matrix in blocks of 128.
int check_matrix(int n_experts, int N, int K, const int32_t* offsets, const char* name) {
  if (n_experts < 1 || n_experts > QMV_MAX_SORT_EXPERTS)
    return record_error(QMV_EINVAL, "%s: n_experts=%d outside [1, %d]", name, n_experts, QMV_MAX_SORT_EXPERTS);
  if (N < 1 || N > QMV_MAX_N) return record_error(QMV_ESHAPE, "%s: N=%d outside [1, %d]", name, N, QMV_MAX_N);
  QMV_TRY(check_width(K, false, name));
  if (K % 16) return record_error(QMV_ESHAPE, "%s: K=%d is not a multiple of 16", name, K);
  if (offsets == nullptr && n_experts != 1)
    return record_error(QMV_EINVAL, "%s: rows of %d experts need offsets", name, n_experts);
  return QMV_OK;
}

// Checks of the products of a quantized buffer of D columns; fills `g`.
int product_args(const void* w, const float* w_scales, int n_experts, int N, int K, const void* xq, size_t xq_bytes, int D,
                 int nrows, const int32_t* offsets, int out_type, const void* y, void* stream, const char* name,
                 B128GemmArgs& g) {
  QMV_TRY(check_matrix(n_experts, N, K, offsets, name));
  QMV_TRY(check_type(out_type, name));
  QMV_TRY(check_rows(nrows, name));
  if (any_null(w, w_scales) || (nrows > 0 && any_null(xq, y))) return record_error(QMV_EINVAL, "%s: NULL pointer", name);
  if (any_misaligned(w, w_scales, xq, y, offsets))
    return record_error(QMV_EALIGN, "%s: pointers must be 16-byte aligned", name);
  const size_t need = b128_act_bytes(nrows, D);
  if (xq_bytes < need) return record_error(QMV_ESIZE, "%s: rows %zu bytes < %zu", name, xq_bytes, need);
  g = B128GemmArgs();
  g.n_experts = n_experts;
  g.N = N;
  g.K = K;
  g.w = w;
  g.w_scales = w_scales;
  g.xq = xq;
  g.nrows = nrows;
  g.offsets = offsets;
  g.out_type = out_type;
  g.y = const_cast<void*>(y);
  g.stream = static_cast<cudaStream_t>(stream);
  return QMV_OK;
}

bool act_shape(int64_t nrows, int K) { return nrows >= 0 && nrows <= QMV_MAX_ROWS && K >= 1 && K <= QMV_MAX_N; }

}  // namespace
}  // namespace qmv

using namespace qmv;

extern "C" {

int qmv_moe_router(int32_t type, const void* logits, int64_t ldl, const uint8_t* live, int32_t ntok, int32_t n_experts,
                   int32_t top_k, int32_t score, int32_t renorm, float scale, int32_t* ids, float* weights, void* stream) {
  const char* name = "qmv_moe_router";
  QMV_TRY(check_router(type, ldl, ntok, n_experts, top_k, score, name));
  QMV_TRY(check_scale(scale, name));
  if (ntok > 0 && any_null(logits, ids, weights)) return record_error(QMV_EINVAL, "%s: NULL pointer", name);
  if (any_misaligned(logits, live, ids, weights))
    return record_error(QMV_EALIGN, "%s: pointers must be 16-byte aligned", name);
  if (ntok == 0) return done();
  RouterArgs a;
  a.type = type;
  a.score = score;
  a.logits = logits;
  a.ldl = ldl;
  a.live = live;
  a.ntok = ntok;
  a.n_experts = n_experts;
  a.top_k = top_k;
  a.renorm = renorm != 0;
  a.scale = scale;
  a.ids = ids;
  a.weights = weights;
  a.stream = static_cast<cudaStream_t>(stream);
  g_launch_stage = "launch";
  return launched(launch_router(a), name);
}

size_t qmv_moe_balance_workspace_bytes(int32_t ntok, int32_t n_experts) {
  if (ntok < 0 || ntok > QMV_MAX_ROWS || n_experts < 1 || n_experts > QMV_MAX_SORT_EXPERTS) return 0;
  return balance_space(ntok, n_experts).total;
}

int qmv_moe_balance(int32_t type, const void* logits, int64_t ldl, const uint8_t* live, const int32_t* ids, int32_t ntok,
                    int32_t n_experts, int32_t top_k, int32_t score, int32_t* counts, float* means, float* loss,
                    void* workspace, size_t workspace_bytes, void* stream) {
  const char* name = "qmv_moe_balance";
  QMV_TRY(check_router(type, ldl, ntok, n_experts, top_k, score, name));
  if (any_null(counts, means, loss, workspace) || (ntok > 0 && any_null(logits, ids)))
    return record_error(QMV_EINVAL, "%s: NULL pointer", name);
  if (any_misaligned(logits, live, ids, counts, means, loss, workspace))
    return record_error(QMV_EALIGN, "%s: pointers must be 16-byte aligned", name);
  const BalanceSpace s = balance_space(ntok, n_experts);
  if (workspace_bytes < s.total) return record_error(QMV_ESIZE, "%s: workspace %zu bytes < %zu", name, workspace_bytes, s.total);
  BalanceArgs a;
  a.type = type;
  a.score = score;
  a.logits = logits;
  a.ldl = ldl;
  a.live = live;
  a.ids = ids;
  a.ntok = ntok;
  a.n_experts = n_experts;
  a.top_k = top_k;
  a.counts = counts;
  a.means = means;
  a.loss = loss;
  a.parts = s.parts;
  a.part_sums = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + s.sums);
  a.part_counts = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + s.counts);
  a.stream = static_cast<cudaStream_t>(stream);
  g_launch_stage = "launch";
  return launched(launch_balance(a), name);
}

int qmv_moe_router_grad(int32_t type, const void* logits, int64_t ldl, const uint8_t* live, const int32_t* ids,
                        const float* dweights, const int32_t* counts, const float* dloss, int32_t ntok, int32_t n_experts,
                        int32_t top_k, int32_t score, int32_t renorm, float scale, void* dlogits, int64_t ldd, void* stream) {
  const char* name = "qmv_moe_router_grad";
  QMV_TRY(check_router(type, ldl, ntok, n_experts, top_k, score, name));
  QMV_TRY(check_ld(ldd, n_experts, name));
  QMV_TRY(check_scale(scale, name));
  if ((ntok > 0 && (any_null(logits, dlogits) || (dweights != nullptr && ids == nullptr))) || (counts == nullptr) != (dloss == nullptr))
    return record_error(QMV_EINVAL, "%s: NULL pointer", name);
  if (any_misaligned(logits, live, ids, dweights, counts, dloss, dlogits))
    return record_error(QMV_EALIGN, "%s: pointers must be 16-byte aligned", name);
  if (ntok == 0) return done();
  RouterGradArgs a;
  a.type = type;
  a.score = score;
  a.logits = logits;
  a.ldl = ldl;
  a.live = live;
  a.ids = ids;
  a.dweights = dweights;
  a.counts = counts;
  a.dloss = dloss;
  a.ntok = ntok;
  a.n_experts = n_experts;
  a.top_k = top_k;
  a.renorm = renorm != 0;
  a.scale = scale;
  a.dlogits = dlogits;
  a.ldd = ldd;
  a.stream = static_cast<cudaStream_t>(stream);
  g_launch_stage = "launch";
  return launched(launch_router_grad(a), name);
}

size_t qmv_act_b128_bytes(int32_t nrows, int32_t K) { return act_shape(nrows, K) ? (size_t)b128_act_bytes(nrows, K) : 0; }

size_t qmv_act_b128_scale_offset(int32_t nrows, int32_t K) {
  return act_shape(nrows, K) ? (size_t)b128_scale_offset(nrows, K) : 0;
}

int qmv_act_b128_unpack(const void* xq, int32_t nrows, int32_t K, uint8_t* codes, float* scales) {
  const char* name = "qmv_act_b128_unpack";
  if (!act_shape(nrows, K)) return record_error(QMV_ESHAPE, "%s: %d rows, K=%d", name, nrows, K);
  if (nrows > 0 && any_null(xq, codes, scales)) return record_error(QMV_EINVAL, "%s: NULL pointer", name);
  const uint8_t* src = static_cast<const uint8_t*>(xq);
  const uint8_t* words = src + b128_scale_offset(nrows, K);
  const size_t blocks = (size_t)b128_blocks(K);
  for (size_t r = 0; r < (size_t)nrows; ++r) {
    std::memcpy(codes + r * K, src + r * b128_row_bytes(K), (size_t)K);
    for (size_t b = 0; b < blocks; ++b) std::memcpy(scales + r * blocks + b, words + (r * (size_t)b128_scale_row(K) + b) * 4, 4);
  }
  return done();
}

int qmv_quantize_act_b128(int32_t type, const void* x, int64_t ldx, int32_t nrows, int32_t K, void* xq, size_t xq_bytes,
                          void* stream) {
  const char* name = "qmv_quantize_act_b128";
  QMV_TRY(check_type(type, name));
  QMV_TRY(check_rows(nrows, name));
  QMV_TRY(check_width(K, false, name, QMV_MAX_N));
  QMV_TRY(check_ld(ldx, K, name));
  if (nrows > 0 && any_null(x, xq)) return record_error(QMV_EINVAL, "%s: NULL pointer", name);
  if (any_misaligned(x, xq)) return record_error(QMV_EALIGN, "%s: pointers must be 16-byte aligned", name);
  const size_t need = b128_act_bytes(nrows, K);
  if (xq_bytes < need) return record_error(QMV_ESIZE, "%s: output %zu bytes < %zu", name, xq_bytes, need);
  if (nrows == 0) return done();
  B128QuantArgs q;
  q.type = type;
  q.x = x;
  q.ldx = ldx;
  q.nrows = nrows;
  q.K = K;
  q.xq = xq;
  q.stream = static_cast<cudaStream_t>(stream);
  g_launch_stage = "launch";
  return launched(launch_quantize_b128(q), name);
}

int qmv_quantize_weights_b128(int32_t type, const void* w, int32_t n_experts, int32_t N, int32_t K, void* codes, float* scales,
                              void* stream) {
  const char* name = "qmv_quantize_weights_b128";
  static const int32_t grouped = 0;   // offsets play no part here
  QMV_TRY(check_type(type, name));
  QMV_TRY(check_matrix(n_experts, N, K, &grouped, name));
  if ((int64_t)n_experts * b128_blocks(N) * b128_blocks(K) > INT32_MAX)
    return record_error(QMV_ESHAPE, "%s: more than 2^31 - 1 blocks", name);
  if (any_null(w, codes, scales)) return record_error(QMV_EINVAL, "%s: NULL pointer", name);
  if (any_misaligned(w, codes, scales)) return record_error(QMV_EALIGN, "%s: pointers must be 16-byte aligned", name);
  g_launch_stage = "launch";
  return launched(launch_quantize_weights_b128(type, w, n_experts, N, K, codes, scales, static_cast<cudaStream_t>(stream)), name);
}

int qmv_b128_product(const void* w, const float* w_scales, int32_t n_experts, int32_t N, int32_t K, const void* xq,
                     size_t xq_bytes, int32_t nrows, const int32_t* offsets, int32_t out_type, void* y, void* stream) {
  const char* name = "qmv_b128_product";
  B128GemmArgs g;
  QMV_TRY(product_args(w, w_scales, n_experts, N, K, xq, xq_bytes, K, nrows, offsets, out_type, y, stream, name, g));
  if (nrows == 0) return done();
  g_launch_stage = "launch";
  return launched(launch_b128_product(g), name);
}

size_t qmv_b128_linear_workspace_bytes(int32_t nrows, int32_t K) { return qmv_act_b128_bytes(nrows, K); }

int qmv_b128_linear(const void* w, const float* w_scales, int32_t n_experts, int32_t N, int32_t K, int32_t type, const void* x,
                    int64_t ldx, int32_t nrows, const int32_t* offsets, void* workspace, size_t workspace_bytes, void* y,
                    void* stream) {
  const char* name = "qmv_b128_linear";
  B128GemmArgs g;
  QMV_TRY(product_args(w, w_scales, n_experts, N, K, workspace, workspace_bytes, K, nrows, offsets, type, y, stream, name, g));
  QMV_TRY(check_ld(ldx, K, name));
  if (nrows > 0 && any_null(x)) return record_error(QMV_EINVAL, "%s: NULL pointer", name);
  if (any_misaligned(x)) return record_error(QMV_EALIGN, "%s: pointers must be 16-byte aligned", name);
  if (nrows == 0) return done();
  g.x = x;
  g.ldx = ldx;
  g.x_type = type;
  g_launch_stage = "launch";
  return launched(launch_b128_linear(g), name);
}

int qmv_b128_grad_x(const void* w, const float* w_scales, int32_t n_experts, int32_t N, int32_t K, const void* dyq,
                    size_t dyq_bytes, int32_t nrows, const int32_t* offsets, int32_t out_type, void* dx, void* stream) {
  const char* name = "qmv_b128_grad_x";
  B128GemmArgs g;
  QMV_TRY(product_args(w, w_scales, n_experts, N, K, dyq, dyq_bytes, N, nrows, offsets, out_type, dx, stream, name, g));
  if (nrows == 0) return done();
  g_launch_stage = "launch";
  return launched(launch_b128_grad_x(g), name);
}

int qmv_b128_grad_w(int32_t type, const void* dy, int64_t ld_dy, const void* x, int64_t ldx, int32_t n_experts, int32_t N,
                    int32_t K, int32_t nrows, const int32_t* offsets, int32_t out_type, void* dw, void* stream) {
  const char* name = "qmv_b128_grad_w";
  if (type != QMV_BF16 && type != QMV_F16) return record_error(QMV_EINVAL, "%s: bf16 or fp16 only (type %d)", name, type);
  QMV_TRY(check_matrix(n_experts, N, K, offsets, name));
  QMV_TRY(check_type(out_type, name));
  QMV_TRY(check_rows(nrows, name));
  QMV_TRY(check_ld(ld_dy, N, name));
  QMV_TRY(check_ld(ldx, K, name));
  if (ld_dy % 8 || ldx % 8) return record_error(QMV_ESHAPE, "%s: row strides must be multiples of 8", name);
  if (any_null(dw) || (nrows > 0 && any_null(dy, x))) return record_error(QMV_EINVAL, "%s: NULL pointer", name);
  if (any_misaligned(dy, x, offsets, dw)) return record_error(QMV_EALIGN, "%s: pointers must be 16-byte aligned", name);
  if (nrows == 0) {   // the sum over no rows
    g_launch_stage = "cudaMemsetAsync";
    return launched(cudaMemsetAsync(dw, 0, (size_t)n_experts * N * K * (out_type == QMV_F32 ? 4 : 2),
                                    static_cast<cudaStream_t>(stream)), name);
  }
  B128GradWArgs g;
  g.type = type;
  g.dy = dy;
  g.ld_dy = ld_dy;
  g.x = x;
  g.ldx = ldx;
  g.n_experts = n_experts;
  g.N = N;
  g.K = K;
  g.nrows = nrows;
  g.offsets = offsets;
  g.out_type = out_type;
  g.dw = dw;
  g.stream = static_cast<cudaStream_t>(stream);
  g_launch_stage = "launch";
  return launched(launch_b128_grad_w(g), name);
}

}  // extern "C"
