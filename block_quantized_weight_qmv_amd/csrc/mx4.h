// Device helpers of the MXFP4 kernels.
//
// An MXFP4 tensor (include/qmv.h) is a plane of 4-bit float codes, two to a
// byte, and a plane of one scale byte p for every 32 columns: 2^(p - 127), p =
// 255 NaN.  gfx950 converts such codes and multiplies them with their scales in
// its matrix instructions; both take the scale as a power of two.
#pragma once

#include "device_util.h"

namespace qmv {

// 2^(p - 127) as fp32 (p = 0: a subnormal, which the conversions take as such).
__device__ __forceinline__ float mx4_scale(uint32_t p) {
  return __uint_as_float(p == 0 ? 0x00400000u : p == 255 ? 0x7FC00000u : p << 23);
}

// The eight codes of a dword times 2^(p - 127), exact in fp32 (above 2^128:
// infinities).
__device__ __forceinline__ void mx4_decode8(uint32_t q, uint32_t p, float* v) {
  typedef float f2_t __attribute__((ext_vector_type(2)));
  const float s = mx4_scale(p == 255 ? 127 : p), nan = __builtin_nanf("");
  const f2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, 1),
             c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, 3);
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y, v[4] = c.x, v[5] = c.y, v[6] = d.x, v[7] = d.y;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = p == 255 ? nan : v[i];
}

// Two fp32 numbers rounded to bf16 / fp16 (nearest even) in one dword.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 b2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, b2_t{static_cast<__bf16>(a), static_cast<__bf16>(b)});
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  return __builtin_bit_cast(uint32_t, h2_t{static_cast<_Float16>(a), static_cast<_Float16>(b)});
}

}  // namespace qmv
