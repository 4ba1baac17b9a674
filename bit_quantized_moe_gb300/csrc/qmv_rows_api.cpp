// qmv_rows_api.cpp -- the many-row part of the C ABI (include/qmv.h): argument
// checks and dispatch to the launchers. Nothing here reads device memory or
// synchronizes. Without rows (an empty tensor's address is NULL) only what does
// not depend on them has to be there.
#include <cmath>
#include <cstring>

#include "../../include/qmv.h"
#include "qmv_checks.h"
#include "qmv_internal.h"
#include "qmv_layout.h"

namespace qmv {
namespace {

bool mx_shape(int fmt, int64_t nrows, int K) {
  return (fmt == QMV_MXFP4 || fmt == QMV_MXFP8) && nrows >= 0 && nrows <= QMV_MAX_ROWS && K >= 32 && K <= QMV_MAX_K &&
         K % 32 == 0;
}

// Common checks of the two products; fills `g`.
int product_args(const qmv_wdesc* desc, const void* w, const void* xq, size_t xq_bytes, int nrows, const int32_t* offsets,
                 const void* y, void* stream, const char* name, MxGemmArgs& g) {
  QMV_TRY(check_weight_desc(desc));
  if (!fmt_is_mx(desc->fmt)) return record_error(QMV_EINVAL, "%s: MX formats only (got format %d)", name, desc->fmt);
  QMV_TRY(check_rows(nrows, name));
  if (offsets == nullptr && desc->n_experts != 1)
    return record_error(QMV_EINVAL, "%s: a dense product needs n_experts == 1 (got %d)", name, desc->n_experts);
  if (desc->n_experts > QMV_MAX_SORT_EXPERTS)
    return record_error(QMV_EINVAL, "%s: %d experts > %d", name, desc->n_experts, QMV_MAX_SORT_EXPERTS);
  if (any_null(w) || (nrows > 0 && any_null(xq, y))) return record_error(QMV_EINVAL, "%s: NULL pointer", name);
  if (any_misaligned(w, xq, y, offsets)) return record_error(QMV_EALIGN, "%s: pointers must be 16-byte aligned", name);
  const size_t need = mx_act_bytes(desc->fmt, nrows, desc->K);
  if (xq_bytes < need) return record_error(QMV_ESIZE, "%s: activations %zu bytes < %zu", name, xq_bytes, need);
  g = MxGemmArgs();
  g.fmt = desc->fmt;
  g.N = desc->N;
  g.K = desc->K;
  g.n_experts = desc->n_experts;
  g.w = w;
  g.xq = xq;
  g.nrows = nrows;
  g.offsets = offsets;
  g.out_n = desc->N;
  g.y = const_cast<void*>(y);
  g.stream = static_cast<cudaStream_t>(stream);
  return QMV_OK;
}

int mx_product(const qmv_wdesc* desc, const void* w, const void* xq, size_t xq_bytes, int nrows, const int32_t* offsets,
               int out_type, float* wide, void* y, void* stream, const char* name) {
  MxGemmArgs g;
  QMV_TRY(check_type(out_type, name));
  QMV_TRY(product_args(desc, w, xq, xq_bytes, nrows, offsets, y, stream, name, g));
  if (nrows == 0) return done();
  g.out_type = out_type;
  g.wide = wide;
  return launched(launch_mx_gemm(g), name);
}

// most: columns that a row may have: QMV_MAX_K of a product's input, QMV_MAX_N of its output.
int route_args(int type, int ntok, int top_k, int K, int most, const int32_t* row_of_slot, void* stream, const char* name,
               RouteArgs& r) {
  QMV_TRY(check_type(type, name));
  QMV_TRY(check_slots(ntok, top_k, name));
  QMV_TRY(check_width(K, false, name, most));
  if (ntok > 0 && row_of_slot == nullptr) return record_error(QMV_EINVAL, "%s: NULL pointer", name);
  if (misaligned(row_of_slot)) return record_error(QMV_EALIGN, "%s: pointers must be 16-byte aligned", name);
  r = RouteArgs();
  r.type = type;
  r.ntok = ntok;
  r.top_k = top_k;
  r.K = K;
  r.row_of_slot = row_of_slot;
  r.stream = static_cast<cudaStream_t>(stream);
  return QMV_OK;
}

int return_rows(int type, const void* ys, bool ys_f32, const float* wide, const float* weights, int ntok, int top_k, int N,
                const int32_t* row_of_slot, void* y, int64_t ldy, void* stream, const char* name) {
  RouteArgs r;
  QMV_TRY(route_args(type, ntok, top_k, N, QMV_MAX_N, row_of_slot, stream, name, r));
  QMV_TRY(check_ld(ldy, N, name));
  if (ntok > 0 && any_null(ys, weights, y)) return record_error(QMV_EINVAL, "%s: NULL pointer", name);
  if (any_misaligned(ys, weights, y)) return record_error(QMV_EALIGN, "%s: pointers must be 16-byte aligned", name);
  if (ntok == 0) return done();
  r.rows = ys;
  r.rows_f32 = ys_f32 && type != QMV_F32;
  r.wide = wide;
  r.weights = weights;
  r.out_tok = y;
  r.ld_out = ldy;
  g_launch_stage = "launch";
  return launched(launch_return(r), name);
}

// The experts' rows between the down product and the weighted sum are kept in
// fp32 where that is at most this many bytes, so that the layer's output is
// rounded once: they stay in L2 then, and cost about nothing. Larger calls
// keep them in the output's 16 bits, which doubles the rounding error's square
// and halves 2 x 189 MB of traffic for 4096 tokens x 4 slots of 2880 columns.
// A sum past fp16's 65,504 may come back into its range with its weight: large
// fp16 calls keep such sums in fp32 beside the rows, where the weighted sum
// looks for what it reads as infinity.
constexpr size_t kExactRowsBytes = 32u << 20;
bool rows_in_f32(int64_t slots, int N) { return (size_t)slots * N * 4 <= kExactRowsBytes; }

// Parts of the layer's workspace.
struct LayerSpace {
  size_t offsets, row_of_slot, slot_of_row, xq, hq, ys, wide, total;
};

LayerSpace layer_space(const qmv_wdesc* gu, const qmv_wdesc* down, int64_t slots) {
  LayerSpace s;
  size_t at = 0;
  const auto take = [&at](size_t bytes) {
    const size_t here = at;
    at += up256(bytes);
    return here;
  };
  s.offsets = take(((size_t)gu->n_experts + 1) * 4);
  s.row_of_slot = take((size_t)slots * 4);
  s.slot_of_row = take((size_t)slots * 4);
  s.xq = take(mx_act_bytes(gu->fmt, slots, gu->K));
  s.hq = take(mx_act_bytes(down->fmt, slots, gu->N));
  const size_t outputs = (size_t)slots * down->N;
  s.ys = take(outputs * (rows_in_f32(slots, down->N) ? 4 : 2));
  s.wide = take(rows_in_f32(slots, down->N) ? 0 : outputs * 4);
  s.total = at;
  return s;
}

int check_layer(const qmv_wdesc* gu, const qmv_wdesc* down, int ntok, int top_k, const char* name) {
  QMV_TRY(check_weight_desc(gu));
  QMV_TRY(check_weight_desc(down));
  if (!fmt_is_mx(gu->fmt) || !fmt_is_mx(down->fmt))
    return record_error(QMV_EINVAL, "%s: gate/up and down must both be MX formats", name);
  if (gu->N > QMV_MAX_N / 2) return record_error(QMV_ESHAPE, "%s: N=%d too large for gate/up fusion", name, gu->N);
  if (down->K != gu->N) return record_error(QMV_ESHAPE, "%s: down K=%d must equal gate/up N=%d", name, down->K, gu->N);
  if (down->n_experts != gu->n_experts || gu->n_experts > QMV_MAX_SORT_EXPERTS)
    return record_error(QMV_EINVAL, "%s: expert counts %d and %d (equal, at most %d)", name, gu->n_experts,
                        down->n_experts, QMV_MAX_SORT_EXPERTS);
  return check_slots(ntok, top_k, name);
}

}  // namespace
}  // namespace qmv

using namespace qmv;

extern "C" {

size_t qmv_act_mx_bytes(int32_t fmt, int32_t nrows, int32_t K) {
  return mx_shape(fmt, nrows, K) ? (size_t)mx_act_bytes(fmt, nrows, K) : 0;
}

size_t qmv_act_mx_scale_offset(int32_t fmt, int32_t nrows, int32_t K) {
  return mx_shape(fmt, nrows, K) ? (size_t)mx_scale_offset(fmt, nrows, K) : 0;
}

int qmv_act_mx_unpack(int32_t fmt, const void* xq, int32_t nrows, int32_t K, uint8_t* codes, uint8_t* scales) {
  const char* name = "qmv_act_mx_unpack";
  if (!mx_shape(fmt, nrows, K)) return record_error(QMV_ESHAPE, "%s: format %d, %d rows, K=%d", name, fmt, nrows, K);
  if (nrows == 0) return done();
  if (any_null(xq, codes, scales)) return record_error(QMV_EINVAL, "%s: NULL pointer", name);
  const uint8_t* src = static_cast<const uint8_t*>(xq);
  std::memcpy(codes, src, (size_t)nrows * mx_row_bytes(fmt, K));
  const uint8_t* words = src + mx_scale_offset(fmt, nrows, K);
  const size_t groups = (size_t)K / 32;
  for (int64_t r = 0; r < nrows; ++r) {
    for (size_t i = 0; i < groups; ++i) scales[r * groups + i] = words[((i / 4) * (size_t)nrows + r) * 4 + i % 4];
  }
  return done();
}

int qmv_quantize_act_mx(int32_t fmt, int32_t type, const void* x, int64_t ldx, int32_t nrows, int32_t K, void* xq,
                        size_t xq_bytes, void* stream) {
  const char* name = "qmv_quantize_act_mx";
  if (fmt != QMV_MXFP4 && fmt != QMV_MXFP8) return record_error(QMV_EINVAL, "%s: not an MX format: %d", name, fmt);
  QMV_TRY(check_type(type, name));
  QMV_TRY(check_rows(nrows, name));
  QMV_TRY(check_width(K, true, name));
  QMV_TRY(check_ld(ldx, K, name));
  if (nrows > 0 && any_null(x, xq)) return record_error(QMV_EINVAL, "%s: NULL pointer", name);
  if (any_misaligned(x, xq)) return record_error(QMV_EALIGN, "%s: pointers must be 16-byte aligned", name);
  const size_t need = mx_act_bytes(fmt, nrows, K);
  if (xq_bytes < need) return record_error(QMV_ESIZE, "%s: output %zu bytes < %zu", name, xq_bytes, need);
  if (nrows == 0) return done();
  QuantArgs q;
  q.fmt = fmt;
  q.type = type;
  q.x = x;
  q.ldx = ldx;
  q.ntok = nrows;
  q.K = K;
  q.xq = xq;
  q.nrows = nrows;
  q.scale_offset = mx_scale_offset(fmt, nrows, K);
  q.stream = static_cast<cudaStream_t>(stream);
  g_launch_stage = "launch";
  return launched(launch_quantize_mx(q), name);
}

int qmv_rms_norm(int32_t type, const void* x, int64_t ldx, const void* res, int64_t ldr, const void* gain,
                 int32_t nrows, int32_t K, float eps, void* sum, int32_t out, void* y, size_t y_bytes, void* stream) {
  const char* name = "qmv_rms_norm";
  QMV_TRY(check_type(type, name));
  if (out < QMV_NORM_PLAIN || out > QMV_NORM_Q8) return record_error(QMV_EINVAL, "%s: unknown output %d", name, out);
  QMV_TRY(check_rows(nrows, name));
  QMV_TRY(check_width(K, out != QMV_NORM_PLAIN, name));
  QMV_TRY(check_ld(ldx, K, name));
  if (res != nullptr || sum != nullptr) QMV_TRY(check_ld(ldr, K, name));
  if (!(eps >= 0.0f) || std::isinf(eps)) return record_error(QMV_EINVAL, "%s: eps=%g", name, (double)eps);
  if (any_null(gain) || (nrows > 0 && any_null(x, y))) return record_error(QMV_EINVAL, "%s: NULL pointer", name);
  if (any_misaligned(x, res, gain, sum, y)) return record_error(QMV_EALIGN, "%s: pointers must be 16-byte aligned", name);
  size_t need = (size_t)nrows * K * (type == QMV_F32 ? 4 : 2);
  if (out == QMV_NORM_MXFP8 || out == QMV_NORM_MXFP4) {
    need = mx_act_bytes(out == QMV_NORM_MXFP8 ? MXFP8 : MXFP4, nrows, K);
  } else if (out == QMV_NORM_Q8) {
    need = (size_t)nrows * q8_vec_bytes(K);
  }
  if (y_bytes < need) return record_error(QMV_ESIZE, "%s: output %zu bytes < %zu", name, y_bytes, need);
  if (nrows == 0) return done();
  NormArgs a;
  a.type = type;
  a.x = x;
  a.ldx = ldx;
  a.res = res;
  a.ldr = ldr;
  a.gain = gain;
  a.nrows = nrows;
  a.K = K;
  a.eps = eps;
  a.sum = sum;
  a.out = out;
  a.y = y;
  if (out == QMV_NORM_MXFP8) a.scale_offset = mx_scale_offset(MXFP8, nrows, K);
  if (out == QMV_NORM_MXFP4) a.scale_offset = mx_scale_offset(MXFP4, nrows, K);
  a.stream = static_cast<cudaStream_t>(stream);
  g_launch_stage = "launch";
  return launched(launch_rms_norm(a), name);
}

int qmv_mx_product(const qmv_wdesc* desc, const void* w, const void* xq, size_t xq_bytes, int32_t nrows,
                   const int32_t* offsets, int32_t out_type, void* y, void* stream) {
  return mx_product(desc, w, xq, xq_bytes, nrows, offsets, out_type, nullptr, y, stream, "qmv_mx_product");
}

int qmv_mx_gate_up_swiglu(const qmv_wdesc* desc, const void* w, const void* xq, size_t xq_bytes, int32_t nrows,
                          const int32_t* offsets, int32_t h_fmt, void* hq, size_t hq_bytes, void* stream) {
  const char* name = "qmv_mx_gate_up_swiglu";
  MxGemmArgs g;
  QMV_TRY(product_args(desc, w, xq, xq_bytes, nrows, offsets, hq, stream, name, g));
  if (h_fmt != QMV_MXFP4 && h_fmt != QMV_MXFP8) return record_error(QMV_EINVAL, "%s: not an MX format: %d", name, h_fmt);
  if (desc->N > QMV_MAX_N / 2) return record_error(QMV_ESHAPE, "%s: N=%d too large for gate/up fusion", name, desc->N);
  QMV_TRY(check_width(desc->N, true, name));
  const size_t need = mx_act_bytes(h_fmt, nrows, desc->N);
  if (hq_bytes < need) return record_error(QMV_ESIZE, "%s: output %zu bytes < %zu", name, hq_bytes, need);
  if (nrows == 0) return done();
  g.N = gate_up_rows(desc->N);
  g.glu = true;
  g.h_fmt = h_fmt;
  return launched(launch_mx_gemm(g), name);
}

size_t qmv_moe_sort_workspace_bytes(int32_t, int32_t, int32_t) { return 0; }

int qmv_moe_sort(const int32_t* ids, int32_t ntok, int32_t top_k, int32_t n_experts, int32_t* offsets,
                 int32_t* row_of_slot, int32_t* slot_of_row, void* workspace, size_t workspace_bytes, void* stream) {
  const char* name = "qmv_moe_sort";
  QMV_TRY(check_slots(ntok, top_k, name));
  if (n_experts < 1 || n_experts > QMV_MAX_SORT_EXPERTS)
    return record_error(QMV_EINVAL, "%s: n_experts=%d outside [1, %d]", name, n_experts, QMV_MAX_SORT_EXPERTS);
  if (any_null(offsets) || (ntok > 0 && any_null(ids, row_of_slot, slot_of_row))) return record_error(QMV_EINVAL, "%s: NULL pointer", name);
  if (any_misaligned(ids, offsets, row_of_slot, slot_of_row, workspace))
    return record_error(QMV_EALIGN, "%s: pointers must be 16-byte aligned", name);
  const size_t need = qmv_moe_sort_workspace_bytes(ntok, top_k, n_experts);
  if (workspace_bytes < need) return record_error(QMV_ESIZE, "%s: workspace %zu bytes < %zu", name, workspace_bytes, need);
  SortArgs s;
  s.ids = ids;
  s.nslots = (int64_t)ntok * top_k;
  s.n_experts = n_experts;
  s.offsets = offsets;
  s.row_of_slot = row_of_slot;
  s.slot_of_row = slot_of_row;
  s.stream = static_cast<cudaStream_t>(stream);
  g_launch_stage = "launch";
  return launched(launch_moe_sort(s), name);
}

int qmv_moe_dispatch(int32_t type, const void* x, int64_t ldx, int32_t ntok, int32_t top_k, int32_t K,
                     const int32_t* row_of_slot, void* xs, void* stream) {
  const char* name = "qmv_moe_dispatch";
  RouteArgs r;
  QMV_TRY(route_args(type, ntok, top_k, K, QMV_MAX_K, row_of_slot, stream, name, r));
  QMV_TRY(check_ld(ldx, K, name));
  if (ntok > 0 && any_null(x, xs)) return record_error(QMV_EINVAL, "%s: NULL pointer", name);
  if (any_misaligned(x, xs)) return record_error(QMV_EALIGN, "%s: pointers must be 16-byte aligned", name);
  if (ntok == 0) return done();
  r.tok = x;
  r.ld_tok = ldx;
  r.out_rows = xs;
  g_launch_stage = "launch";
  return launched(launch_dispatch(r), name);
}

int qmv_moe_dispatch_mx(int32_t fmt, int32_t type, const void* x, int64_t ldx, int32_t ntok, int32_t top_k, int32_t K,
                        const int32_t* row_of_slot, void* xq, size_t xq_bytes, void* stream) {
  const char* name = "qmv_moe_dispatch_mx";
  RouteArgs r;
  if (fmt != QMV_MXFP4 && fmt != QMV_MXFP8) return record_error(QMV_EINVAL, "%s: not an MX format: %d", name, fmt);
  QMV_TRY(route_args(type, ntok, top_k, K, QMV_MAX_K, row_of_slot, stream, name, r));
  QMV_TRY(check_width(K, true, name));
  QMV_TRY(check_ld(ldx, K, name));
  if (ntok > 0 && any_null(x, xq)) return record_error(QMV_EINVAL, "%s: NULL pointer", name);
  if (any_misaligned(x, xq)) return record_error(QMV_EALIGN, "%s: pointers must be 16-byte aligned", name);
  const int64_t slots = (int64_t)ntok * top_k;
  const size_t need = mx_act_bytes(fmt, slots, K);
  if (xq_bytes < need) return record_error(QMV_ESIZE, "%s: output %zu bytes < %zu", name, xq_bytes, need);
  if (ntok == 0) return done();
  QuantArgs q;
  q.fmt = fmt;
  q.type = type;
  q.x = x;
  q.ldx = ldx;
  q.ntok = ntok;
  q.top_k = top_k;
  q.K = K;
  q.row_of_slot = row_of_slot;
  q.xq = xq;
  q.nrows = slots;
  q.scale_offset = mx_scale_offset(fmt, slots, K);
  q.stream = r.stream;
  g_launch_stage = "launch";
  return launched(launch_quantize_mx(q), name);
}

int qmv_moe_dispatch_grad(int32_t type, const void* dxs, int32_t ntok, int32_t top_k, int32_t K,
                          const int32_t* row_of_slot, void* dx, int64_t ldx, void* stream) {
  const char* name = "qmv_moe_dispatch_grad";
  RouteArgs r;
  QMV_TRY(route_args(type, ntok, top_k, K, QMV_MAX_K, row_of_slot, stream, name, r));
  QMV_TRY(check_ld(ldx, K, name));
  if (ntok > 0 && any_null(dxs, dx)) return record_error(QMV_EINVAL, "%s: NULL pointer", name);
  if (any_misaligned(dxs, dx)) return record_error(QMV_EALIGN, "%s: pointers must be 16-byte aligned", name);
  if (ntok == 0) return done();
  r.rows = dxs;
  r.out_tok = dx;
  r.ld_out = ldx;
  g_launch_stage = "launch";
  return launched(launch_return(r), name);
}

int qmv_moe_return(int32_t type, const void* ys, const float* weights, int32_t ntok, int32_t top_k, int32_t N,
                   const int32_t* row_of_slot, void* y, int64_t ldy, void* stream) {
  return return_rows(type, ys, false, nullptr, weights, ntok, top_k, N, row_of_slot, y, ldy, stream, "qmv_moe_return");
}

int qmv_moe_return_grad(int32_t type, const void* dy, int64_t ld_dy, const void* ys, const float* weights,
                        int32_t ntok, int32_t top_k, int32_t N, const int32_t* row_of_slot, void* dys, float* dweights,
                        void* stream) {
  const char* name = "qmv_moe_return_grad";
  RouteArgs r;
  QMV_TRY(route_args(type, ntok, top_k, N, QMV_MAX_N, row_of_slot, stream, name, r));
  QMV_TRY(check_ld(ld_dy, N, name));
  if (ntok > 0 && any_null(dy, ys, weights, dys, dweights)) return record_error(QMV_EINVAL, "%s: NULL pointer", name);
  if (any_misaligned(dy, ys, weights, dys, dweights))
    return record_error(QMV_EALIGN, "%s: pointers must be 16-byte aligned", name);
  if (ntok == 0) return done();
  r.tok = dy;
  r.ld_tok = ld_dy;
  r.rows = ys;
  r.weights = weights;
  r.out_rows = dys;
  r.dweights = dweights;
  g_launch_stage = "launch";
  return launched(launch_return_grad(r), name);
}

size_t qmv_moe_prefill_layer_workspace_bytes(const qmv_wdesc* gu, const qmv_wdesc* down, int32_t ntok, int32_t top_k) {
  if (check_layer(gu, down, ntok, top_k, "qmv_moe_prefill_layer")) return 0;
  return layer_space(gu, down, (int64_t)ntok * top_k).total;
}

int qmv_moe_prefill_layer(const qmv_wdesc* gu, const void* w_gu, const qmv_wdesc* down, const void* w_down,
                          int32_t type, const void* x, int64_t ldx, const int32_t* ids, const float* weights,
                          int32_t ntok, int32_t top_k, void* ws, size_t ws_bytes, void* y, void* stream) {
  const char* name = "qmv_moe_prefill_layer";
  QMV_TRY(check_layer(gu, down, ntok, top_k, name));
  if (type != QMV_BF16 && type != QMV_F16) return record_error(QMV_EINVAL, "%s: bf16 or fp16 only (type %d)", name, type);
  QMV_TRY(check_ld(ldx, gu->K, name));
  if (any_null(w_gu, w_down, ws) || (ntok > 0 && any_null(x, ids, weights, y))) return record_error(QMV_EINVAL, "%s: NULL pointer", name);
  if (any_misaligned(w_gu, w_down, x, ids, weights, ws, y))
    return record_error(QMV_EALIGN, "%s: pointers must be 16-byte aligned", name);
  const int64_t slots = (int64_t)ntok * top_k;
  const LayerSpace s = layer_space(gu, down, slots);
  if (ws_bytes < s.total) return record_error(QMV_ESIZE, "%s: workspace %zu bytes < %zu", name, ws_bytes, s.total);
  if (ntok == 0) return done();
  uint8_t* base = static_cast<uint8_t*>(ws);
  int32_t* offsets = reinterpret_cast<int32_t*>(base + s.offsets);
  int32_t* row_of_slot = reinterpret_cast<int32_t*>(base + s.row_of_slot);
  int32_t* slot_of_row = reinterpret_cast<int32_t*>(base + s.slot_of_row);
  QMV_TRY(qmv_moe_sort(ids, ntok, top_k, gu->n_experts, offsets, row_of_slot, slot_of_row, nullptr, 0, stream));
  QMV_TRY(qmv_moe_dispatch_mx(gu->fmt, type, x, ldx, ntok, top_k, gu->K, row_of_slot, base + s.xq,
                              mx_act_bytes(gu->fmt, slots, gu->K), stream));
  QMV_TRY(qmv_mx_gate_up_swiglu(gu, w_gu, base + s.xq, mx_act_bytes(gu->fmt, slots, gu->K), (int32_t)slots, offsets,
                                down->fmt, base + s.hq, mx_act_bytes(down->fmt, slots, gu->N), stream));
  const bool exact = rows_in_f32(slots, down->N);
  float* wide = !exact && type == QMV_F16 ? reinterpret_cast<float*>(base + s.wide) : nullptr;
  QMV_TRY(mx_product(down, w_down, base + s.hq, mx_act_bytes(down->fmt, slots, gu->N), (int32_t)slots, offsets,
                     exact ? QMV_F32 : type, wide, base + s.ys, stream, name));
  return return_rows(type, base + s.ys, exact, wide, weights, ntok, top_k, down->N, row_of_slot, y, down->N, stream, name);
}

}  // extern "C"
