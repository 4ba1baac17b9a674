// qmv_rows.cuh -- device helpers of the many-row operators: element types,
// vector access, and the microscaled quantization of a group of 32.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qmv_device.cuh"
#include "qmv_layout.h"

namespace qmv {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Eight consecutive elements as they lie in memory, so that several can be
// asked for before the first is used.
template <typename T>
struct alignas(16) Raw8 {
  T e[8];
};

// VEC: the address is 16-byte aligned. Plain loads here and in the kernels that
// read what another kernel wrote: these kernels start before the one before
// them has ended (griddepcontrol.wait), so what it writes is not constant for
// their lifetime, as the non-coherent loads of __ldg demand.
template <typename T, bool VEC>
__device__ __forceinline__ void load_raw8(const T* p, Raw8<T>& r) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(r) / 16; ++i) {
      reinterpret_cast<uint4*>(r.e)[i] = reinterpret_cast<const uint4*>(p)[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.e[i] = p[i];
  }
}

template <typename T>
__device__ __forceinline__ void clear_raw8(Raw8<T>& r) {
#pragma unroll
  for (T& e : r.e) e = from_f32<T>(0.0f);
}

// Eight consecutive elements as fp32.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  Raw8<T> r;
  load_raw8<T, VEC>(p, r);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = to_f32(r.e[i]);
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  if constexpr (!VEC) {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = from_f32<T>(v[i]);
  } else if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint4 a;
    T* e = reinterpret_cast<T*>(&a);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = from_f32<T>(v[i]);
    *reinterpret_cast<uint4*>(p) = a;
  }
}

// Largest |v| of eight values as fp32 bits. Compared as integers, so that a
// NaN is larger than every number and infinity.
__device__ __forceinline__ uint32_t amax_bits8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return m;
}

// The same of elements as loaded. 16-bit types compare two at a time; the
// NaN-propagating maximum keeps a NaN above everything.
__device__ __forceinline__ uint32_t amax_bits8(const Raw8<float>& r) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(r.e[i]) & 0x7fffffffu);
  return m;
}
template <typename T, typename T2>
__device__ __forceinline__ T2 amax_pair8(const Raw8<T>& r) {
  T2 p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(r.e)[i] & 0x7fff7fffu;
    p[i] = *reinterpret_cast<const T2*>(&w);
  }
  return __hmax2_nan(__hmax2_nan(p[0], p[1]), __hmax2_nan(p[2], p[3]));
}
__device__ __forceinline__ uint32_t amax_bits8(const Raw8<__nv_bfloat16>& r) {
  const __nv_bfloat162 m = amax_pair8<__nv_bfloat16, __nv_bfloat162>(r);
  return __float_as_uint(__bfloat162float(__hmax_nan(m.x, m.y)));
}
__device__ __forceinline__ uint32_t amax_bits8(const Raw8<__half>& r) {
  const __half2 m = amax_pair8<__half, __half2>(r);
  return __float_as_uint(__half2float(__hmax_nan(m.x, m.y)));
}

// E8M0 byte of a group whose largest |v| has these bits: the exponent of the
// largest power of two not above it, less the element type's largest exponent
// (2 for E2M1, 8 for E4M3), so that the largest element needs the element
// type's top binade; 0 at the bottom of the range and for a group of zeros,
// 255 (NaN) for a group with an infinity or a NaN.
template <int FMT>
__device__ __forceinline__ uint32_t group_e8m0(uint32_t amax) {
  constexpr uint32_t emax = FMT == MXFP4 ? 2u : 8u;
  const uint32_t ex = amax >> 23;
  return ex == 255u ? 255u : (ex > emax ? ex - emax : 0u);
}

// 2^(127 - e): the power of two that divides a group by its scale. e is at
// most 254 - 2 here, so it is a normal number. 0 for e = 255 (see mx_codes8).
__device__ __forceinline__ float e8m0_inverse(uint32_t e) { return __uint_as_float(e == 255u ? 0u : (254u - e) << 23); }

// Eight elements' codes, rounded to nearest even and saturating: one word
// (E2M1, element i in nibble i) or two (E4M3, element i in byte i). Elements
// of a group that is NaN get the code 0.
template <int FMT>
__device__ __forceinline__ void mx_codes8(const float (&v)[8], uint32_t e, uint32_t (&w)[FMT == MXFP4 ? 1 : 2]) {
  const float s = e8m0_inverse(e);
  if constexpr (FMT == MXFP4) {
    asm("{\n .reg .b8 a, b, c, d;\n"
        " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        " mov.b32 %0, {a, b, c, d};\n}"
        : "=r"(w[0])
        : "f"(v[0] * s), "f"(v[1] * s), "f"(v[2] * s), "f"(v[3] * s), "f"(v[4] * s), "f"(v[5] * s), "f"(v[6] * s),
          "f"(v[7] * s));
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      asm("{\n .reg .b16 a, b;\n cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n"
          " mov.b32 %0, {a, b};\n}"
          : "=r"(w[h])
          : "f"(v[4 * h] * s), "f"(v[4 * h + 1] * s), "f"(v[4 * h + 2] * s), "f"(v[4 * h + 3] * s));
    }
  }
#pragma unroll
  for (uint32_t& x : w) x = e == 255u ? 0u : x;
}

// Stores eight elements' codes at column c (a multiple of 8) of a row.
template <int FMT>
__device__ __forceinline__ void store_codes8(uint8_t* row, int c, const uint32_t (&w)[FMT == MXFP4 ? 1 : 2]) {
  if constexpr (FMT == MXFP4) {
    *reinterpret_cast<uint32_t*>(row + c / 2) = w[0];
  } else {
    *reinterpret_cast<uint2*>(row + c) = make_uint2(w[0], w[1]);
  }
}

// The four scale bytes of 128 columns from 16 lanes of eight columns each (a
// lane of the 16 holds its group's byte): the word, in the first lane of the 16.
__device__ __forceinline__ uint32_t scale_word16(uint32_t e) {
  const uint32_t two = e | __shfl_down_sync(0xffffffffu, e, 4) << 8;
  return two | __shfl_down_sync(0xffffffffu, two, 8) << 16;
}

}  // namespace qmv
