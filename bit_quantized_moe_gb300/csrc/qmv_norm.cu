// qmv_norm.cu -- root-mean-square norm with the residual's addition and a
// quantized output, and the microscaled quantizer of activation rows.
#include <type_traits>

#include "qmv_internal.h"
#include "qmv_rows.cuh"

namespace qmv {

// ---------------------------------------------------------------------------
// y = s * rsqrt(mean(s^2) + eps) * gain, s = x + r.
//
// One pass: a row's s stays in the registers of its TPR threads (V vectors of
// 8 columns each; past 32,768 columns, with V = 8 and 1024 threads, a part of
// it goes to local memory: 512 x 65536 bf16 to MXFP8 67 us, 0.52 of the copy
// bandwidth, 512 x 32768 27 us, 0.65), its squares are summed in fp32, and the same registers give
// the output. s is rounded only where it is stored: the norm takes the fp32
// sum. Bound by memory: 2 + 2 bytes in, 2 + 1 + 1/32 out per element for bf16
// and MXFP8.
//
// Squares of numbers past 2^64 or far below 1 leave fp32. Where the mean (with
// eps) comes out outside [2^-100, infinity), the row's threads take the squares
// again of numbers scaled by 2^-100 or 2^100.
//
// VEC: every row starts on a 16-byte boundary and the width is a multiple of
// 8. Otherwise (plain output only needs no group of 32) a thread's elements
// are TPR apart, so that a warp still reads consecutive ones.
// ---------------------------------------------------------------------------
constexpr float kMeanLow = 0x1p-100f, kUp = 0x1p100f, kDown = 0x1p-100f;

// Barrier of a row's TPR threads: rows of a CTA may differ in how many they pass.
template <int TPR, int THREADS>
__device__ __forceinline__ void row_barrier() {
  if constexpr (TPR == THREADS) __syncthreads();
  else asm volatile("bar.sync %0, %1;" :: "r"(1 + (int)threadIdx.x / TPR), "n"(TPR) : "memory");
}

template <typename T, int OUT, int TPR, int V, bool VEC>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
rms_norm_kernel(NormArgs a) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int kRowsPerCta = kThreads / TPR;
  constexpr int kWarps = TPR / 32;
  constexpr bool kCols = VEC || OUT != kNormPlain;   // a thread owns 8 consecutive columns
  __shared__ float part[2][kThreads / 32];
  const int tid = threadIdx.x % TPR;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kRowsPerCta + threadIdx.x / TPR;
  const bool live = row < a.nrows;
  const int K = a.K;
  pdl_wait();
  const T* x = static_cast<const T*>(a.x) + (live ? row : 0) * a.ldx;
  const T* res = a.res != nullptr ? static_cast<const T*>(a.res) + (live ? row : 0) * a.ldr : nullptr;
  T* sum = a.sum != nullptr ? static_cast<T*>(a.sum) + (live ? row : 0) * a.ldr : nullptr;
  const T* gain = static_cast<const T*>(a.gain);

  float s[V][8];
  float sq = 0.0f;
  if constexpr (kCols) {
    // every load of the row is under way before the first is used
    Raw8<T> rx[V], rr[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * TPR + tid) * 8;
      if (live && c < K) load_raw8<T, VEC>(x + c, rx[j]);
      else clear_raw8(rx[j]);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * TPR + tid) * 8;
      if (res != nullptr && live && c < K) load_raw8<T, VEC>(res + c, rr[j]);
      else clear_raw8(rr[j]);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[j][i] = to_f32(rx[j].e[i]) + to_f32(rr[j].e[i]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = (j * 8 + i) * TPR + tid;
        s[j][i] = live && c < K ? to_f32(x[c]) : 0.0f;
      }
    }
    if (res != nullptr) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = (j * 8 + i) * TPR + tid;
          if (live && c < K) s[j][i] += to_f32(res[c]);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    float p = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) p = fmaf(s[j][i], s[j][i], p);
    sq += p;
  }
  if (sum != nullptr) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if constexpr (kCols) {
        const int c = (j * TPR + tid) * 8;
        if (live && c < K) store8<T, VEC>(sum + c, s[j]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = (j * 8 + i) * TPR + tid;
          if (live && c < K) sum[c] = from_f32<T>(s[j][i]);
        }
      }
    }
  }
  // the row's sum of its threads' parts, the same in all of them; the first is taken by all rows of the CTA together
  const auto row_sum = [&](float v, auto first) {
    constexpr int use = decltype(first)::value ? 0 : 1;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (kWarps > 1) {
      if (lane == 0) part[use][threadIdx.x / 32] = v;
      if constexpr (use == 0) __syncthreads();
      else row_barrier<TPR, kThreads>();
      const int w0 = (threadIdx.x / TPR) * kWarps;
      v = lane < kWarps ? part[use][w0 + lane] : 0.0f;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;
  };
  const float mean = row_sum(sq, std::true_type()) / (float)K + a.eps;
  float rs = 1.0f / sqrtf(mean);
  // fp16's squares stay in the range
  if (!std::is_same_v<T, __half> && !(mean >= kMeanLow && mean <= 3.402823466e38f)) {   // the same in a row's threads
    const bool small = mean < kMeanLow;
    const float f = small ? kUp : kDown;
    float again = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = s[j][i] * f;
        again = fmaf(v, v, again);
      }
    }
    rs = 1.0f / sqrtf(row_sum(again, std::false_type()) / (float)K + a.eps * f * f);
    // Small numbers take the factor first, exactly. Large rows take it last: s * rs is then at most 2^100 sqrt(K),
    // and the row's small numbers, which the factor would take below the normal ones, keep their places.
    const float first = small ? f : rs;
    rs = small ? rs : f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[j][i] *= first;
    }
  }

#pragma unroll
  for (int j = 0; j < V; ++j) {
    if constexpr (kCols) {
      const int c = (j * TPR + tid) * 8;
      const bool in = live && c < K;
      float y[8];
      if (in) {
        float g[8];
        load8<T, VEC>(gain + c, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = s[j][i] * rs * g[i];
      } else {
#pragma unroll
        for (float& v : y) v = 0.0f;
      }
      if constexpr (OUT == kNormPlain) {
        if (in) store8<T, VEC>(static_cast<T*>(a.y) + row * K + c, y);
      } else {
        uint32_t m = amax_bits8(y);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));   // four lanes: one group of 32
        if constexpr (OUT == kNormQ8) {
          // as quantize_q8_kernel: d = amax / 127, q = x / d rounded half away from zero
          const float amax = __uint_as_float(m);
          const float d = __fdiv_rn(amax, 127.0f);
          const float id = d != 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
          if (in) {
            uint8_t* out = static_cast<uint8_t*>(a.y) + row * q8_vec_bytes(K);
            uint32_t w[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float r = fminf(fmaxf(roundf(__fmul_rn(y[i], id)), -127.0f), 127.0f);
              w[i >> 2] |= (uint32_t)(uint8_t)(int8_t)(int)r << (8 * (i & 3));
            }
            *reinterpret_cast<uint2*>(out + c) = make_uint2(w[0], w[1]);
            if ((tid & 3) == 0) reinterpret_cast<__half*>(out + K)[c / 32] = __float2half_rn(d);
          }
        } else {
          constexpr int FMT = OUT == kNormMxfp8 ? MXFP8 : MXFP4;
          const uint32_t e = group_e8m0<FMT>(m);
          uint32_t w[FMT == MXFP4 ? 1 : 2];
          mx_codes8<FMT>(y, e, w);
          uint8_t* out = static_cast<uint8_t*>(a.y);
          if (in) store_codes8<FMT>(out + row * mx_row_bytes(FMT, K), c, w);
          const uint32_t word = scale_word16(e);
          if ((lane & 15) == 0 && in) {
            reinterpret_cast<uint32_t*>(out + a.scale_offset)[(int64_t)(c / 128) * a.nrows + row] = word;
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = (j * 8 + i) * TPR + tid;
        if (live && c < K) static_cast<T*>(a.y)[row * K + c] = from_f32<T>(s[j][i] * rs * to_f32(gain[c]));
      }
    }
  }
  pdl_launch_dependents();
}

namespace {

template <typename T, int OUT, int TPR, int V, bool VEC>
cudaError_t norm_go(const NormArgs& a) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int kRowsPerCta = kThreads / TPR;
  return launch_pdl(rms_norm_kernel<T, OUT, TPR, V, VEC>, dim3((unsigned)((a.nrows + kRowsPerCta - 1) / kRowsPerCta)),
                    dim3(kThreads), 0, a.stream, a);
}

// Threads of a row, and vectors of 8 columns that each holds: three or four, so
// that a row's loads are under way together and few of the last are empty
// (4096 rows of 2880 to MXFP8: 18.2 us with 256 threads x 2, 15.7 with 128 x
// 3). Rows read element by element want the threads: 513 x 2881 6.5 us with
// 128, 4.6 with 256.
template <typename T, int OUT, bool VEC>
cudaError_t norm_width(const NormArgs& a) {
  if (a.K <= 256) return norm_go<T, OUT, 32, 1, VEC>(a);
  if (a.K <= 1024) return norm_go<T, OUT, 32, 4, VEC>(a);
  if constexpr (VEC) {
    if (a.K <= 2048) return norm_go<T, OUT, 64, 4, VEC>(a);
    if (a.K <= 128 * 3 * 8) return norm_go<T, OUT, 128, 3, VEC>(a);
    if (a.K <= 4096) return norm_go<T, OUT, 128, 4, VEC>(a);
  } else if (a.K <= 4096) {
    return norm_go<T, OUT, 256, 2, VEC>(a);
  }
  if (a.K <= 8192) return norm_go<T, OUT, 256, 4, VEC>(a);
  if (a.K <= 32768) return norm_go<T, OUT, 1024, 4, VEC>(a);
  return norm_go<T, OUT, 1024, 8, VEC>(a);
}

template <typename T, int OUT>
cudaError_t norm_vec(const NormArgs& a) {
  const int64_t unit = 16 / (int)sizeof(T);
  const bool vec = a.K % 8 == 0 && a.ldx % unit == 0 && (a.ldr % unit == 0 || (a.res == nullptr && a.sum == nullptr));
  return vec ? norm_width<T, OUT, true>(a) : norm_width<T, OUT, false>(a);
}

template <typename T>
cudaError_t norm_out(const NormArgs& a) {
  switch (a.out) {
    case kNormMxfp8: return norm_vec<T, kNormMxfp8>(a);
    case kNormMxfp4: return norm_vec<T, kNormMxfp4>(a);
    case kNormQ8: return norm_vec<T, kNormQ8>(a);
    default: return norm_vec<T, kNormPlain>(a);
  }
}

}  // namespace

cudaError_t launch_rms_norm(const NormArgs& a) {
  switch (a.type) {
    case QMV_BF16: return norm_out<__nv_bfloat16>(a);
    case QMV_F16: return norm_out<__half>(a);
    default: return norm_out<float>(a);
  }
}

// ---------------------------------------------------------------------------
// Microscaled quantization of rows (and, with row_of_slot, their dispatch to
// the experts' order). A thread takes a group of 32 columns: 64 bytes in (bf16)
// under way at once, the maximum without another lane, 16 or 32 bytes of codes
// out; four lanes' scale bytes make a word. (Eight columns a thread, with
// shuffles for the maximum, took 29.5 us for 8192 x 7168 to MXFP4.) A routed
// token is read and quantized once and written to its top_k rows; a dropped
// slot's row (~row in row_of_slot) is written as zeros.
// Bound by memory: 2 bytes in, 0.53 (E2M1) or 1.03 (E4M3) out per row.
// ---------------------------------------------------------------------------
template <typename T, int FMT, bool ROUTED, bool VEC>
__global__ void __launch_bounds__(256)
quantize_mx_kernel(QuantArgs a) {
  constexpr int kWords = FMT == MXFP4 ? 4 : 8;   // of a group's codes
  const unsigned words = (unsigned)mx_scale_words(a.K);
  const unsigned unit = blockIdx.x * 64u + threadIdx.x / 4u;   // 128 columns of a row, four lanes
  const unsigned total = (unsigned)a.ntok * words;             // at most 2^22 rows of 2^9 words
  const bool live = unit < total;
  const unsigned t = live ? unit / words : 0u, kb = live ? unit - t * words : 0u;
  const int c = (int)(kb * 128u) + (int)(threadIdx.x & 3u) * 32;
  const bool in = live && c < a.K;
  pdl_wait();
  Raw8<T> raw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (in) load_raw8<T, VEC>(static_cast<const T*>(a.x) + (int64_t)t * a.ldx + c + 8 * i, raw[i]);
    else clear_raw8(raw[i]);
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, amax_bits8(raw[i]));
  const uint32_t e = group_e8m0<FMT>(m);
  uint4 codes[kWords / 4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = to_f32(raw[i].e[k]);
    mx_codes8<FMT>(v, e, *reinterpret_cast<uint32_t(*)[kWords / 4]>(reinterpret_cast<uint32_t*>(codes) + i * (kWords / 4)));
  }
  // E4M3: two lanes trade halves, so that each store of a lane pair fills a group's 32 bytes
  // (8191 tokens to 4 rows of 2880 each: 30.3 us with a lane's own two stores).
  const bool odd = (threadIdx.x & 1u) != 0;
  const int c0 = c - (odd ? 32 : 0);   // the pair's first group
  if constexpr (FMT == MXFP8) {
    uint4 other = odd ? codes[0] : codes[1];
    other.x = __shfl_xor_sync(0xffffffffu, other.x, 1);
    other.y = __shfl_xor_sync(0xffffffffu, other.y, 1);
    other.z = __shfl_xor_sync(0xffffffffu, other.z, 1);
    other.w = __shfl_xor_sync(0xffffffffu, other.w, 1);
    if (odd) codes[0] = other;
    else codes[1] = other;
  }
  // the unit's four scale bytes, in its first lane
  uint32_t word = e | __shfl_down_sync(0xffffffffu, e, 1) << 8;
  word |= __shfl_down_sync(0xffffffffu, word, 2) << 16;
  uint8_t* out = static_cast<uint8_t*>(a.xq);
  const uint64_t row_bytes = mx_row_bytes(FMT, a.K);
  const int at = FMT == MXFP8 ? c0 + (odd ? 16 : 0) : c / 2;
  uint32_t* scales = reinterpret_cast<uint32_t*>(out + a.scale_offset) + (int64_t)kb * a.nrows;
  if (live) {
    constexpr int kGroup = ROUTED ? 4 : 1;   // rows looked up together
    const int copies = ROUTED ? a.top_k : 1;
    for (int j0 = 0; j0 < copies; j0 += kGroup) {
      int r[kGroup];
#pragma unroll
      for (int j = 0; j < kGroup; ++j) {
        r[j] = !ROUTED ? (int)t : (j0 + j < copies ? a.row_of_slot[(int64_t)t * copies + j0 + j] : 0);
      }
#pragma unroll
      for (int j = 0; j < kGroup; ++j) {
        if (j0 + j < copies) {
          const bool keep = r[j] >= 0;
          const int row = keep ? r[j] : ~r[j];
          if (row >= a.nrows) continue;   // no row of this call
#pragma unroll
          for (int i = 0; i < kWords / 4; ++i) {
            if (FMT == MXFP8 ? c0 + 32 * i < a.K : in) {
              *reinterpret_cast<uint4*>(out + (uint64_t)row * row_bytes + at + 32 * i) =
                  keep ? codes[i] : make_uint4(0, 0, 0, 0);
            }
          }
          if ((threadIdx.x & 3u) == 0) scales[row] = keep ? word : 0u;
        }
      }
    }
  }
  pdl_launch_dependents();
}

namespace {

template <typename T, int FMT>
cudaError_t quant_go(const QuantArgs& a) {
  const int64_t units = a.ntok * mx_scale_words(a.K);
  const dim3 grid((unsigned)((units + 63) / 64)), block(256);
  const bool vec = a.ldx % (16 / (int)sizeof(T)) == 0;
  if (a.row_of_slot != nullptr) {
    return vec ? launch_pdl(quantize_mx_kernel<T, FMT, true, true>, grid, block, 0, a.stream, a)
               : launch_pdl(quantize_mx_kernel<T, FMT, true, false>, grid, block, 0, a.stream, a);
  }
  return vec ? launch_pdl(quantize_mx_kernel<T, FMT, false, true>, grid, block, 0, a.stream, a)
             : launch_pdl(quantize_mx_kernel<T, FMT, false, false>, grid, block, 0, a.stream, a);
}

template <typename T>
cudaError_t quant_fmt(const QuantArgs& a) {
  return a.fmt == MXFP4 ? quant_go<T, MXFP4>(a) : quant_go<T, MXFP8>(a);
}

}  // namespace

cudaError_t launch_quantize_mx(const QuantArgs& a) {
  switch (a.type) {
    case QMV_BF16: return quant_fmt<__nv_bfloat16>(a);
    case QMV_F16: return quant_fmt<__half>(a);
    default: return quant_fmt<float>(a);
  }
}

}  // namespace qmv
