// qmv_b128_gemm.cu -- products of E4M3 operands with fp32 scales of 128 columns
// (rows) and blocks of 128 x 128 (weights), and their gradients:
//
//   y[r][n]     = sum_b sx[r][b] sw[n / 128][b] sum_{k in b} q[r][k] w[n][k]
//   dx[r][k]    = sum_b sd[r][b] sw[b][k / 128] sum_{n in b} d[r][n] w[n][k]
//   dW[e][n][k] = sum over e's rows r of dy[r][n] x[r][k]
//
// One CTA an output tile of 64 x 64, its operands decoded to fp32 in shared
// memory, a thread 4 x 4 outputs.
#include "qmv_internal.h"
#include "qmv_rows.cuh"

namespace qmv {

constexpr int kTile = 64, kDepth = 16;

__device__ __forceinline__ float e4m3_to_f32(uint8_t c) {
  uint32_t h[2];
  e4m3x4_to_f16x2(c, h);
  return __half2float(__ushort_as_half((unsigned short)(h[0] & 0xffffu)));
}

template <typename T>
__device__ __forceinline__ void store_one(void* y, int64_t at, float v) {
  static_cast<T*>(y)[at] = from_f32<T>(v);
}
__device__ __forceinline__ void store_as(int type, void* y, int64_t at, float v) {
  if (type == QMV_BF16) store_one<__nv_bfloat16>(y, at, v);
  else if (type == QMV_F16) store_one<__half>(y, at, v);
  else store_one<float>(y, at, v);
}

// Rows of expert e of the call; an offset below an earlier one counts as it.
__device__ __forceinline__ void expert_rows(const int32_t* offsets, int nrows, int e, int& lo, int& hi) {
  if (offsets == nullptr) {
    lo = 0;
    hi = nrows;
    return;
  }
  lo = 0;
  for (int i = 0; i <= e; ++i) lo = max(lo, min(offsets[i], nrows));
  hi = max(lo, min(offsets[e + 1], nrows));
}

// A: [M][D] and B: [C][D] as functions of (row, depth); out of (row, column).
template <typename A, typename B, typename O>
__device__ __forceinline__ void tile_product(int m0, int M, int c0, int C, int D, A&& fa, B&& fb, O&& out) {
  __shared__ float sa[kDepth][kTile + 1], sb[kDepth][kTile + 1];
  float acc[4][4] = {};
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  for (int d0 = 0; d0 < D; d0 += kDepth) {
    for (int i = threadIdx.x; i < kTile * kDepth; i += 256) {
      const int d = i % kDepth, r = i / kDepth;
      sa[d][r] = m0 + r < M && d0 + d < D ? fa(m0 + r, d0 + d) : 0.0f;
      sb[d][r] = c0 + r < C && d0 + d < D ? fb(c0 + r, d0 + d) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[d][ty * 4 + i], sb[d][tx * 4 + j], acc[i][j]);
      }
    }
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty * 4 + i, c = c0 + tx * 4 + j;
      if (m < M && c < C) out(m, c, acc[i][j]);
    }
  }
}

template <bool GRAD>
__global__ void __launch_bounds__(256) b128_product_kernel(B128GemmArgs a) {
  pdl_wait();
  const int D = GRAD ? a.N : a.K, C = GRAD ? a.K : a.N;
  const int e = blockIdx.z;
  int lo, hi;
  expert_rows(a.offsets, (int)a.nrows, e, lo, hi);
  const int m0 = blockIdx.y * kTile;
  if (m0 < hi - lo) {
    const uint8_t* q = static_cast<const uint8_t*>(a.xq);
    const float* sx = reinterpret_cast<const float*>(q + b128_scale_offset(a.nrows, D));
    const uint64_t row = b128_row_bytes(D);
    const uint8_t* w = static_cast<const uint8_t*>(a.w) + (int64_t)e * a.N * a.K;
    const int kb = b128_blocks(a.K);
    const float* sw = a.w_scales + (int64_t)e * b128_blocks(a.N) * kb;
    tile_product(
        m0, hi - lo, blockIdx.x * kTile, C, D,
        [&](int r, int d) { return e4m3_to_f32(q[(uint64_t)(lo + r) * row + d]) * sx[(int64_t)(d / kB128) * a.nrows + lo + r]; },
        [&](int c, int d) {
          const int n = GRAD ? d : c, k = GRAD ? c : d;
          return e4m3_to_f32(w[(int64_t)n * a.K + k]) * sw[n / kB128 * kb + k / kB128];
        },
        [&](int r, int c, float v) { store_as(a.out_type, a.y, (int64_t)(lo + r) * C + c, v); });
  }
  pdl_launch_dependents();
}

template <typename T>
__global__ void __launch_bounds__(256) b128_grad_w_kernel(B128GradWArgs a) {
  pdl_wait();
  const int e = blockIdx.z;
  int lo, hi;
  expert_rows(a.offsets, (int)a.nrows, e, lo, hi);
  const T* dy = static_cast<const T*>(a.dy);
  const T* x = static_cast<const T*>(a.x);
  tile_product(
      blockIdx.y * kTile, a.N, blockIdx.x * kTile, a.K, hi - lo,
      [&](int n, int r) { return to_f32(dy[(int64_t)(lo + r) * a.ld_dy + n]); },
      [&](int k, int r) { return to_f32(x[(int64_t)(lo + r) * a.ldx + k]); },
      [&](int n, int k, float v) { store_as(a.out_type, a.dw, ((int64_t)e * a.N + n) * a.K + k, v); });
  pdl_launch_dependents();
}

namespace {

unsigned tiles_of(int64_t n) { return (unsigned)((n + kTile - 1) / kTile); }

}  // namespace

cudaError_t launch_b128_product(const B128GemmArgs& a) {
  return launch_pdl(b128_product_kernel<false>, dim3(tiles_of(a.N), tiles_of(a.nrows), a.n_experts), dim3(256), 0, a.stream, a);
}

cudaError_t launch_b128_grad_x(const B128GemmArgs& a) {
  return launch_pdl(b128_product_kernel<true>, dim3(tiles_of(a.K), tiles_of(a.nrows), a.n_experts), dim3(256), 0, a.stream, a);
}

cudaError_t launch_b128_grad_w(const B128GradWArgs& a) {
  const dim3 grid(tiles_of(a.K), tiles_of(a.N), a.n_experts);
  if (a.type == QMV_BF16) return launch_pdl(b128_grad_w_kernel<__nv_bfloat16>, grid, dim3(256), 0, a.stream, a);
  return launch_pdl(b128_grad_w_kernel<__half>, grid, dim3(256), 0, a.stream, a);
}

}  // namespace qmv
