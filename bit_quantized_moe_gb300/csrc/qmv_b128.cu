// qmv_b128.cu -- quantization to E4M3 with one fp32 scale per 128 columns of a
// row (activations, gradients) or per block of 128 x 128 (weights).
#include "qmv_b128.cuh"
#include "qmv_internal.h"

namespace qmv {

// Rows: four lanes take a block of 128 columns, 32 columns each, whose loads are
// under way together. Bound by memory: 2 bytes in, 1 + 1/32 out (bf16).
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) quantize_b128_kernel(B128QuantArgs a) {
  const int blocks = b128_blocks(a.K);
  const int64_t unit = (int64_t)blockIdx.x * 64 + threadIdx.x / 4;   // a block of 128 columns
  const int64_t r = unit / blocks;
  const int kb = (int)(unit - r * blocks);
  const bool live = r < a.nrows;
  const int c = kb * kB128 + (int)(threadIdx.x & 3) * 32;
  pdl_wait();
  Raw8<T> raw[4];
  const T* row = static_cast<const T*>(a.x) + (live ? r : 0) * a.ldx;
#pragma unroll
  for (int i = 0; i < 4; ++i) load_to<T, VEC>(row, c + 8 * i, live ? a.K : 0, raw[i]);
  uint32_t m = max(max(amax_bits8(raw[0]), amax_bits8(raw[1])), max(amax_bits8(raw[2]), amax_bits8(raw[3])));
#pragma unroll
  for (int o = 2; o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  const BlockScale s = block_scale(m);
  uint4 codes[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint2 lo = codes8<T>(raw[2 * h], s.inverse), hi = codes8<T>(raw[2 * h + 1], s.inverse);
    codes[h] = make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
  // two lanes trade halves, so that each store of a lane pair fills 32 bytes (8192 x 7168: 35 us with a lane's own two)
  const bool odd = (threadIdx.x & 1) != 0;
  uint4 other = odd ? codes[0] : codes[1];
  other.x = __shfl_xor_sync(0xffffffffu, other.x, 1);
  other.y = __shfl_xor_sync(0xffffffffu, other.y, 1);
  other.z = __shfl_xor_sync(0xffffffffu, other.z, 1);
  other.w = __shfl_xor_sync(0xffffffffu, other.w, 1);
  if (odd) codes[0] = other;
  else codes[1] = other;
  if (live) {
    uint8_t* out = static_cast<uint8_t*>(a.xq);
    const int64_t wide = (int64_t)b128_row_bytes(a.K);   // the row's last 16 codes may go past K: they are 0
    const int at = c + (odd ? -16 : 0);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (at + 32 * h < wide) *reinterpret_cast<uint4*>(out + r * wide + at + 32 * h) = codes[h];
    }
    if ((threadIdx.x & 3) == 0) {
      reinterpret_cast<float*>(out + b128_scale_offset(a.nrows, a.K))[r * b128_scale_row(a.K) + kb] = s.scale;
    }
  }
  pdl_launch_dependents();
}

// Weights: a CTA takes a block; 16 threads a row, eight columns each, four rows.
template <typename T>
__global__ void __launch_bounds__(512)
quantize_weights_b128_kernel(const T* w, int N, int K, int n_blocks, int k_blocks, uint8_t* codes, float* scales) {
  constexpr int kEach = 4, kStep = 32;   // rows of a thread, and how far apart
  __shared__ uint32_t part[16];
  const int64_t block = blockIdx.x;
  const int kb = (int)(block % k_blocks);
  const int nb = (int)(block / k_blocks % n_blocks);
  const int64_t e = block / k_blocks / n_blocks;
  const int c = kb * kB128 + (int)(threadIdx.x & 15) * 8;
  const int r0 = nb * kB128 + (int)threadIdx.x / 16;
  const int64_t base = e * N * K;
  pdl_wait();
  Raw8<T> raw[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {   // K is a multiple of 16
    const int r = r0 + kStep * i;
    if (r < N && c < K) load_raw8<T, true>(w + base + (int64_t)r * K + c, raw[i]);
    else clear_raw8(raw[i]);
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) m = max(m, amax_bits8(raw[i]));
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, part[i]);
  const BlockScale s = block_scale(m);
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int r = r0 + kStep * i;
    if (r < N && c < K) *reinterpret_cast<uint2*>(codes + base + (int64_t)r * K + c) = codes8<T>(raw[i], s.inverse);
  }
  if (threadIdx.x == 0) scales[block] = s.scale;
  pdl_launch_dependents();
}

namespace {

template <typename T>
cudaError_t quant_b128(const B128QuantArgs& a) {
  const int64_t units = a.nrows * b128_blocks(a.K);
  const dim3 grid((unsigned)((units + 63) / 64)), block(256);
  const bool vec = a.ldx % (16 / (int)sizeof(T)) == 0;
  return vec ? launch_pdl(quantize_b128_kernel<T, true>, grid, block, 0, a.stream, a)
             : launch_pdl(quantize_b128_kernel<T, false>, grid, block, 0, a.stream, a);
}

template <typename T>
cudaError_t quant_weights(const void* w, int n_experts, int N, int K, void* codes, float* scales, cudaStream_t s) {
  const int nb = b128_blocks(N), kb = b128_blocks(K);
  return launch_pdl(quantize_weights_b128_kernel<T>, dim3((unsigned)((int64_t)n_experts * nb * kb)), dim3(512), 0, s,
                    static_cast<const T*>(w), N, K, nb, kb, static_cast<uint8_t*>(codes), scales);
}

}  // namespace

cudaError_t launch_quantize_b128(const B128QuantArgs& a) {
  switch (a.type) {
    case QMV_BF16: return quant_b128<__nv_bfloat16>(a);
    case QMV_F16: return quant_b128<__half>(a);
    default: return quant_b128<float>(a);
  }
}

cudaError_t launch_quantize_weights_b128(int type, const void* w, int n_experts, int N, int K, void* codes, float* scales,
                                         cudaStream_t s) {
  switch (type) {
    case QMV_BF16: return quant_weights<__nv_bfloat16>(w, n_experts, N, K, codes, scales, s);
    case QMV_F16: return quant_weights<__half>(w, n_experts, N, K, codes, scales, s);
    default: return quant_weights<float>(w, n_experts, N, K, codes, scales, s);
  }
}

}  // namespace qmv
