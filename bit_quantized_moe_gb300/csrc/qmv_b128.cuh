// qmv_b128.cuh -- quantization of a block of 128 columns, or of 128 x 128, to
// E4M3 with one fp32 scale.
#pragma once

#include "qmv_rows.cuh"

namespace qmv {

// ---------------------------------------------------------------------------
//   a = max(largest |x| of the block, 2^-116),  scale = a / 448,
//   code = E4M3(x * (448 / a)),
// both quotients IEEE divisions, the product rounded to fp32 and then to
// nearest even. 2^-116 keeps 448 / a finite and the scale a normal number; a
// block of zeros has codes of 0. A block with an infinity or a NaN has the scale
// NaN and codes of 0, so that it shows in every product it enters.
// ---------------------------------------------------------------------------
constexpr float kB128Floor = 0x1p-116f;

struct BlockScale {
  float scale, inverse;
};
__device__ __forceinline__ BlockScale block_scale(uint32_t amax) {
  const bool bad = amax >= 0x7f800000u;
  const float a = fmaxf(__uint_as_float(bad ? 0u : amax), kB128Floor);
  BlockScale s;
  s.scale = bad ? __uint_as_float(0x7fc00000u) : __fdiv_rn(a, 448.0f);
  s.inverse = bad ? 0.0f : __fdiv_rn(448.0f, a);
  return s;
}

// Codes of four numbers; inverse 0 stands for a block without numbers.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float inverse) {
  uint32_t w;
  const bool none = inverse == 0.0f;
  asm("{\n .reg .b16 a, b;\n cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n"
      " mov.b32 %0, {a, b};\n}"
      : "=r"(w)
      : "f"(none ? 0.0f : __fmul_rn(a, inverse)), "f"(none ? 0.0f : __fmul_rn(b, inverse)),
        "f"(none ? 0.0f : __fmul_rn(c, inverse)), "f"(none ? 0.0f : __fmul_rn(d, inverse)));
  return w;
}
template <typename T>
__device__ __forceinline__ uint2 codes8(const Raw8<T>& r, float inverse) {
  return make_uint2(codes4(to_f32(r.e[0]), to_f32(r.e[1]), to_f32(r.e[2]), to_f32(r.e[3]), inverse),
                    codes4(to_f32(r.e[4]), to_f32(r.e[5]), to_f32(r.e[6]), to_f32(r.e[7]), inverse));
}

// Eight elements from column c on, those past the last as zeros.
template <typename T, bool VEC>
__device__ __forceinline__ void load_to(const T* row, int c, int K, Raw8<T>& r) {
  if (VEC && c + 8 <= K) {
    load_raw8<T, true>(row + c, r);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.e[i] = c + i < K ? row[c + i] : from_f32<T>(0.0f);
  }
}

}  // namespace qmv
