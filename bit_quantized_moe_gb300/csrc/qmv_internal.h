// qmv_internal.h -- host-side interface between the C ABI and the kernel launchers.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/qmv.h"
#include "qmv_layout.h"

namespace qmv {

// Everything a matvec launch needs; filled and validated by the C ABI layer.
struct MatvecArgs {
  int fmt = 0;
  int N = 0, K = 0, n_experts = 1;
  const void* w = nullptr;        // GPU weight layout, expert 0
  uint64_t expert_stride = 0;     // bytes between experts
  const void* x = nullptr;        // bf16 vectors (MXFP4) or q8_1 vectors
  int nvec = 0;                   // activation vectors in x
  int per_slot = 0;
  const int32_t* ids = nullptr;   // null: dense
  int ntok = 1, top_k = 1;
  void* y = nullptr;
  int32_t* dbg = nullptr;         // integer block sums (CB formats) or null
  uint32_t lut[4] = {0, 0, 0, 0}; // 16 int8 codebook bytes
  bool prefetch = false;          // QMV_FLAG_PREFETCH_INPUTS
  bool x_f32 = false;             // QMV_FLAG_X_F32: fp32 x, quantized to q8_1 in the kernel
  bool x_f16 = false;             // QMV_FLAG_X_F16: MX formats, fp16 x and y
  bool glu = false;               // gate/up-interleaved matrix, store silu(gate) * up
  int out_n = 0;                  // output rows per slot (0: N)
  int path = 0;                   // 0: cost model, 1: tensor cores where possible, 2: CUDA cores
  cudaStream_t stream = nullptr;
};

// Name of the CUDA call a launcher made last on this thread (for error messages).
extern thread_local const char* g_launch_stage;

// Dynamic shared memory a launch of `a` needs (0 if it exceeds the device limit).
size_t matvec_smem_bytes(const MatvecArgs& a);

// Launch plan of `a` for an explicit device shape (qmv_debug_plan).
void debug_plan(const MatvecArgs& a, int sm_count, int ctas_per_sm, size_t smem_per_sm, int64_t out[12]);

cudaError_t launch_matvec_mxfp4(const MatvecArgs& a);
cudaError_t launch_matvec_cb2(const MatvecArgs& a);
cudaError_t launch_matvec_cb3(const MatvecArgs& a);
cudaError_t launch_matvec_cb4(const MatvecArgs& a);
cudaError_t launch_matvec_mxfp8(const MatvecArgs& a);

// Compute-rate probe of the chunk routine (qmv_debug_chunk_rate).
cudaError_t launch_chunk_rate_mxfp4(int nv, int ctas_per_sm, int iters, float* sink, int64_t* weights,
                                    int64_t* threads, cudaStream_t s);
cudaError_t launch_chunk_rate_mxfp8(int nv, int ctas_per_sm, int iters, float* sink, int64_t* weights,
                                    int64_t* threads, cudaStream_t s);
cudaError_t launch_chunk_rate_cb2(int nv, int ctas_per_sm, int iters, float* sink, int64_t* weights,
                                  int64_t* threads, cudaStream_t s);
cudaError_t launch_chunk_rate_cb3(int nv, int ctas_per_sm, int iters, float* sink, int64_t* weights,
                                  int64_t* threads, cudaStream_t s);
cudaError_t launch_chunk_rate_cb4(int nv, int ctas_per_sm, int iters, float* sink, int64_t* weights,
                                  int64_t* threads, cudaStream_t s);

// Dense verify batches of the MX formats (5..16 bf16 tokens) on the tensor
// cores: whether a call takes that path, and its launcher.
bool verify_supported(const MatvecArgs& a);
cudaError_t launch_verify(const MatvecArgs& a);

cudaError_t launch_quantize_q8(const float* x, int nvec, int K, void* xq, cudaStream_t s);
cudaError_t launch_swiglu_bf16(const void* g, const void* u, void* h, int64_t n, cudaStream_t s);
// Output types of the combine.
enum : int { kOutBF16 = 0, kOutF16 = 1, kOutF32 = 2 };
cudaError_t launch_combine(int dtype, const void* ys, const float* w, const int32_t* ids, int ntok, int top_k,
                           int n_experts, int N, void* y, cudaStream_t s);
cudaError_t launch_dequant(int fmt, int N, int K, const void* w, const uint32_t lut[4], float* out,
                           cudaStream_t s);

// Output kinds of the norm (qmv_norm_out).
enum : int { kNormPlain = 0, kNormMxfp8 = 1, kNormMxfp4 = 2, kNormQ8 = 3 };

struct NormArgs {
  int type = 0;                 // qmv_type of x, res, gain, sum and a plain y
  const void* x = nullptr;
  int64_t ldx = 0;              // elements between rows of x
  const void* res = nullptr;    // null: no residual
  int64_t ldr = 0;              // elements between rows of res and of sum
  const void* gain = nullptr;
  int64_t nrows = 0;
  int K = 0;
  float eps = 0.0f;
  void* sum = nullptr;          // null: the sum is not stored
  int out = 0;                  // kNorm*
  void* y = nullptr;
  uint64_t scale_offset = 0;    // MX outputs
  cudaStream_t stream = nullptr;
};
cudaError_t launch_rms_norm(const NormArgs& a);

struct QuantArgs {
  int fmt = 0, type = 0;
  const void* x = nullptr;
  int64_t ldx = 0;
  int64_t ntok = 0;             // rows of x
  int top_k = 1;
  int K = 0;
  const int32_t* row_of_slot = nullptr;   // null: row t of x is row t of xq
  void* xq = nullptr;
  int64_t nrows = 0;            // rows of xq
  uint64_t scale_offset = 0;
  cudaStream_t stream = nullptr;
};
cudaError_t launch_quantize_mx(const QuantArgs& a);

struct SortArgs {
  const int32_t* ids = nullptr;
  int64_t nslots = 0;
  int n_experts = 0;
  int32_t *offsets = nullptr, *row_of_slot = nullptr, *slot_of_row = nullptr;
  cudaStream_t stream = nullptr;
};
cudaError_t launch_moe_sort(const SortArgs& a);

// Rows between the tokens' and the experts' order (qmv_route.cu).
struct RouteArgs {
  int type = 0;
  int64_t ntok = 0;
  int top_k = 1;
  int K = 0;                    // columns
  const int32_t* row_of_slot = nullptr;
  const void* tok = nullptr;    // token-major rows read (x, dy)
  int64_t ld_tok = 0;
  const void* rows = nullptr;   // expert-major rows read (ys, dxs)
  bool rows_f32 = false;        // launch_return: rows are fp32 whatever `type`
  const float* wide = nullptr;  // launch_return, fp16 rows: the values of the infinite ones; null: infinity
  const float* weights = nullptr;   // null: every weight is 1
  void* out_tok = nullptr;      // token-major rows written (y, dx)
  int64_t ld_out = 0;
  void* out_rows = nullptr;     // expert-major rows written (xs, dys)
  float* dweights = nullptr;
  cudaStream_t stream = nullptr;
};
cudaError_t launch_dispatch(const RouteArgs& a);      // out_rows[row] = tok[t]
cudaError_t launch_return(const RouteArgs& a);        // out_tok[t] = sum_j weights * rows[row]
cudaError_t launch_return_grad(const RouteArgs& a);   // out_rows[row] = weights * tok[t]; dweights = <rows[row], tok[t]>

// Product of microscaled activations and weights on the tensor cores.
struct MxGemmArgs {
  int fmt = 0;
  int N = 0, K = 0;             // of the packed matrix (gate/up interleaved: both projections' rows)
  int n_experts = 1;
  const void* w = nullptr;
  const void* xq = nullptr;     // mx_act buffer of nrows rows
  int64_t nrows = 0;
  const int32_t* offsets = nullptr;   // [n_experts + 1] first row of each expert; null: every row, expert 0
  int out_n = 0;                // output columns
  int out_type = 0;             // qmv_type (plain outputs)
  float* wide = nullptr;        // out_type fp16: [nrows][out_n], the sums that fp16 stores as infinity; null: none kept
  void* y = nullptr;            // [nrows][out_n], or the mx_act buffer of h (glu)
  bool glu = false;             // store silu(gate) * up, quantized to h_fmt
  int h_fmt = 0;
  cudaStream_t stream = nullptr;
};
cudaError_t launch_mx_gemm(const MxGemmArgs& a);
uint32_t status_mx_gemm(int clear);

// A number (0 or more) that is asked of each device once, by the first call
// that needs it there; host threads may ask at the same time.
class PerDevice {
 public:
  // ask(int*) -> cudaError_t: the current device's number. An error is not kept.
  template <typename F>
  cudaError_t get(int* value, F&& ask) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    const int known = known_[dev].load(std::memory_order_relaxed);
    if (known != 0) {
      *value = known - 1;
      return cudaSuccess;
    }
    e = ask(value);
    if (e == cudaSuccess) known_[dev].store(*value + 1, std::memory_order_relaxed);
    return e;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<int> known_[kDevices] = {};   // the number + 1; 0: not asked yet
};

// Launch with programmatic stream serialization (the kernel begins with
// griddepcontrol.wait); the legacy default stream has no such edges.
template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = s != nullptr ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

cudaError_t launch_wait_probe(unsigned long long limit_ns, cudaStream_t s);

// Phase probe (build variant -DQMV_PHASE_PROBE, never the product build):
// lane 0 of every warp records %globaltimer at the phases of a launch into
// g_phase[launch slot][CTA][warp][phase], for the launches made while the
// probe is enabled (qmv_debug_phase_probe), slots dealt in launch order. The
// phases (kPh*) run from kernel start to the warp's end.
enum : int {
  kPhStart = 0,        // kernel entry
  kPhWorkList = 1,     // work list built (first CTA barrier passed)
  kPhEarlyTiles = 2,   // tile copies before griddepcontrol.wait issued
  kPhDepWait = 3,      // griddepcontrol.wait returned
  kPhActLoads = 4,     // first round of activation loads issued
  kPhRingIssued = 5,   // every ring stage's first tile copy issued
  kPhActStaged = 6,    // activations staged (CTA barrier passed)
  kPhTile0Ready = 7,   // first tile landed
  kPhTile0Done = 8,    // first tile computed
  kPhTile1Ready = 9,
  kPhTile2Ready = 10,
  kPhLastDone = 11,    // last tile computed
  kPhEnd = 12,         // warp done (after its stores)
  kPhases = 16
};
constexpr int kProbeSlots = 8, kProbeCtas = 512, kProbeWarps = 16;

// Phase probe (probe build only): launches made while on record their phases.
extern bool g_phase_probe_on;
int phase_mxfp4(unsigned long long* out, size_t n, int clear);
int phase_mxfp8(unsigned long long* out, size_t n, int clear);
int phase_cb2(unsigned long long* out, size_t n, int clear);
int phase_cb3(unsigned long long* out, size_t n, int clear);
int phase_cb4(unsigned long long* out, size_t n, int clear);

uint32_t status_act(int clear);
uint32_t status_mxfp4(int clear);
uint32_t status_cb2(int clear);
uint32_t status_cb3(int clear);
uint32_t status_cb4(int clear);
uint32_t status_mxfp8(int clear);
uint32_t status_verify(int clear);

// Sets the calling thread's qmv_last_error() message and returns `code`.
int record_error(int code, const char* fmt, ...);

// QMV_OK, or the error code of an invalid weight descriptor (message recorded).
int check_weight_desc(const qmv_wdesc* d);

// Per-device cached properties.
int device_sm_count();
size_t device_max_smem_optin();
size_t device_smem_per_sm();

}  // namespace qmv
