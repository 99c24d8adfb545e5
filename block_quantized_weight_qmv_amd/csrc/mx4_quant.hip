// Activations to MXFP4 blocks on the device, and back.
//
// A block is 32 consecutive numbers of a row.  With top = max |x|:
//   p = max(0, floor(log2 top) - 2 + 127),   code = nearest(x / 2^(p - 127))
// so the largest lands in [4, 8) and what lies above 6 is held as 6 (OCP
// microscaling, conversion of a vector to an MX block).  Ties go to the even
// code; the conversion instruction rounds so, from subnormals too.  The maximum
// is taken on the bit patterns without their signs, which are ordered as the
// numbers are, infinities and NaN above all: a block that holds one has p = 255
// and zero codes, and reads back as NaN.
//
// Bound: HBM.  A thread takes eight numbers (16 bytes of bf16 or fp16), four
// neighbours a block: their maximum is two quad swaps away, loads are whole
// lines, and a wave's codes are 256 consecutive bytes.  16384 x 3584 in bf16: 31 us
// to blocks (4.8 TB/s, as a copy reaches), 22 us back (6.6 TB/s); 64 rows of fp32
// 2.3 us each way, below what a launch takes.
#include "launch.h"
#include "mx4.h"

namespace qmv {

// Eight numbers from p (16-byte aligned) as fp32.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float* v) {
  uint4 raw[8 * sizeof(T) / 16];
#pragma unroll
  for (int i = 0; i < static_cast<int>(8 * sizeof(T) / 16); ++i) raw[i] = reinterpret_cast<const uint4*>(p)[i];
  x_to_f32<8>(raw, v, static_cast<const T*>(nullptr));
}

template <typename T>
__global__ void __launch_bounds__(256)
mx4_quantize_kernel(const T* x, int64_t x_row, uint32_t chunks, int64_t total, uint8_t* codes, uint8_t* scales) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;  // chunk of eight numbers
  if (i >= total) return;  // (chunks come in fours: a block's threads leave together)
  const int64_t r = i / chunks;
  float v[8];
  load8(x + r * x_row + (i - r * chunks) * 8, v);
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(v[k]) & 0x7FFFFFFFu);
  m = max(m, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(m), 0xB1, 0xF, 0xF, true)));  // quad_perm 1,0,3,2
  m = max(m, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(m), 0x4E, 0xF, 0xF, true)));  // quad_perm 2,3,0,1
  const bool finite = m < 0x7F800000u;
  const int e = static_cast<int>(m >> 23) - 2;
  const uint32_t p = finite ? (e > 0 ? e : 0) : 255;
  const float s = mx4_scale(finite ? p : 127);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], s, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], s, 3);
  reinterpret_cast<uint32_t*>(codes)[i] = finite ? c : 0;
  if ((threadIdx.x & 3) == 0) scales[i >> 2] = static_cast<uint8_t>(p);
}

template <int OUT>
__global__ void __launch_bounds__(256)
mx4_dequant_kernel(const uint8_t* codes, const uint8_t* scales, int64_t total, void* out) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= total) return;
  float v[8];
  mx4_decode8(reinterpret_cast<const uint32_t*>(codes)[i], scales[i >> 2], v);
  if constexpr (OUT == QMV_F32) {
    float4* o = static_cast<float4*>(out) + 2 * i;
    o[0] = make_float4(v[0], v[1], v[2], v[3]);
    o[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    auto two = [&](int k) { return OUT == QMV_F16 ? pack_f16(v[k], v[k + 1]) : pack_bf16(v[k], v[k + 1]); };
    static_cast<uint4*>(out)[i] = make_uint4(two(0), two(2), two(4), two(6));
  }
}

// (A launch's work-items along x are counted in 32 bits: chunks past 2^31 take
// another launch.)
constexpr int64_t kMost = int64_t{1} << 31;

hipError_t mx4_quantize(const qmv_weights& W, const void* x, int x_dtype, int64_t x_row, hipStream_t s) {
  uint8_t* codes = static_cast<uint8_t*>(const_cast<void*>(W.data));
  const uint32_t chunks = static_cast<uint32_t>(W.cols / 8);
  const int64_t most = kMost / chunks < 1 ? 1 : kMost / chunks;  // rows of a launch
  for (int64_t r = 0; r < W.rows; r += most) {
    const int64_t rows = W.rows - r < most ? W.rows - r : most, total = rows * chunks;
    const dim3 grid(static_cast<unsigned>((total + 255) / 256));
    uint8_t* c = codes + r * (W.cols / 2);
    uint8_t* p = codes + W.scales_offset + r * (W.cols / 32);
    switch (x_dtype) {
      case QMV_F32:
        hipLaunchKernelGGL(mx4_quantize_kernel<float>, grid, dim3(256), 0, s, static_cast<const float*>(x) + r * x_row,
                           x_row, chunks, total, c, p);
        break;
      case QMV_F16:
        hipLaunchKernelGGL(mx4_quantize_kernel<_Float16>, grid, dim3(256), 0, s,
                           static_cast<const _Float16*>(x) + r * x_row, x_row, chunks, total, c, p);
        break;
      case QMV_BF16:
        hipLaunchKernelGGL(mx4_quantize_kernel<bf16_t>, grid, dim3(256), 0, s,
                           static_cast<const bf16_t*>(x) + r * x_row, x_row, chunks, total, c, p);
        break;
      default: return hipErrorInvalidValue;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t mx4_dequant(const qmv_weights& W, void* out, int out_dtype, hipStream_t s) {
  const uint8_t* codes = static_cast<const uint8_t*>(W.data);
  const int64_t all = W.rows * (W.cols / 8);
  for (int64_t i = 0; i < all; i += kMost) {
    const int64_t total = all - i < kMost ? all - i : kMost;
    const dim3 grid(static_cast<unsigned>((total + 255) / 256));
    const uint8_t* c = codes + 4 * i;
    const uint8_t* p = codes + W.scales_offset + i / 4;
    uint8_t* o = static_cast<uint8_t*>(out) + i * (out_dtype == QMV_F32 ? 32 : 16);
    switch (out_dtype) {
      case QMV_F32: hipLaunchKernelGGL(mx4_dequant_kernel<QMV_F32>, grid, dim3(256), 0, s, c, p, total, o); break;
      case QMV_F16: hipLaunchKernelGGL(mx4_dequant_kernel<QMV_F16>, grid, dim3(256), 0, s, c, p, total, o); break;
      case QMV_BF16: hipLaunchKernelGGL(mx4_dequant_kernel<QMV_BF16>, grid, dim3(256), 0, s, c, p, total, o); break;
      default: return hipErrorInvalidValue;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace qmv
