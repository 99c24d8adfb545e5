// Dequantization kernels: packed blocks -> dense [rows][cols] fp32 / fp16 / bf16.
//
// VTE (kyuubyn.github.io/VTE), feature list: blocks are decoded byte for byte
// in llama.cpp's reference layout and checked against a NumPy decoder.  Each
// thread decodes four consecutive weights of one row, reading the bytes named
// by the layout tables below one at a time, and stores them as one vector.
//
// Q5_K (hipEngine 0.3.0, "GGUF Support", read as GGUF's published block) is
// decoded the same way.
//
// Exactness: every product here is exact in fp32 (Q8_0 11+7 bits, Q6_K
// 11 + 12 bits, INT4 11+3 bits, Q4_K d*sc*u 21 bits, Q5_K 22 bits, dmin*m
// 17 bits), so the fp32 result is the exact weight, except Q4_K and Q5_K,
// which round once at the subtraction.  fp16 / bf16 outputs are that fp32 value rounded to nearest even.
#include "device_util.h"
#include "launch.h"
#include "mx4.h"
#include "planes.h"

namespace qmv {

__device__ __forceinline__ uint32_t ld_u8(const uint8_t* p) { return *p; }
__device__ __forceinline__ uint32_t ld_le16(const uint8_t* p) { return p[0] | (p[1] << 8); }

// Q8_0: d fp16 | q[32] int8; w = d*q.
__device__ __forceinline__ void dq_q8_0(const uint8_t* row, int k, float* w) {
  const uint8_t* b = row + (k / 32) * 34;
  const float d = f16_to_f32(ld_le16(b));
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int t = (k + e) % 32;
    w[e] = d * static_cast<float>(static_cast<int8_t>(ld_u8(b + 2 + t)));
  }
}

// Six-bit scale and min of sub-block s from the twelve scale bytes of a Q4_K or
// Q5_K block.
__device__ __forceinline__ void k_scale_min(const uint8_t* sc, int s, uint32_t& scale,
                                            uint32_t& mn) {
  if (s < 4) {
    scale = ld_u8(sc + s) & 63;
    mn = ld_u8(sc + s + 4) & 63;
  } else {
    scale = (ld_u8(sc + s + 4) & 15) | ((ld_u8(sc + s - 4) >> 6) << 4);
    mn = (ld_u8(sc + s + 4) >> 4) | ((ld_u8(sc + s) >> 6) << 4);
  }
}

// Q4_K: d | dmin | scales[12] | qs[128]; t = 64c + 32h + l, u = nibble h of qs[32c+l].
__device__ __forceinline__ void dq_q4_k(const uint8_t* row, int k, float* w) {
  const uint8_t* b = row + (k / 256) * 144;
  const float d = f16_to_f32(ld_le16(b));
  const float dmin = f16_to_f32(ld_le16(b + 2));
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int t = (k + e) % 256;
    const int c = t >> 6, h = (t >> 5) & 1, l = t & 31, s = t >> 5;
    uint32_t scale, mn;
    k_scale_min(b + 4, s, scale, mn);
    const uint32_t u = (ld_u8(b + 16 + 32 * c + l) >> (4 * h)) & 15;
    w[e] = (d * static_cast<float>(scale)) * static_cast<float>(u) - dmin * static_cast<float>(mn);
  }
}

// Q4_K in the plane layout (planes.h): the header of block b at 16 b,
// qs[32c + l] at a + 64 b + 16 c + l (l < 16) or 5 a + 64 b + 16 c + l - 16.
// Same decode as dq_q4_k, byte addresses aside.
constexpr int kQ4KPlanes = 0x102;  // kernel template tag, not a public format

__device__ __forceinline__ void dq_q4_k_planes(const uint8_t* w, uint64_t a, int64_t b, int k,
                                               float* out) {
  const uint8_t* h = w + 16 * b;
  const float d = f16_to_f32(ld_le16(h));
  const float dmin = f16_to_f32(ld_le16(h + 2));
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int t = (k + e) % 256;
    const int c = t >> 6, hh = (t >> 5) & 1, l = t & 31, s = t >> 5;
    uint32_t scale, mn;
    k_scale_min(h + 4, s, scale, mn);
    const uint8_t* q = l < 16 ? w + a + 64 * b + 16 * c + l : w + 5 * a + 64 * b + 16 * c + (l - 16);
    const uint32_t u = (ld_u8(q) >> (4 * hh)) & 15;
    out[e] = (d * static_cast<float>(scale)) * static_cast<float>(u) - dmin * static_cast<float>(mn);
  }
}

// Q5_K: d | dmin | scales[12] | qh[32] | qs[128]; t = 64c + 32h + l,
// u = (nibble h of qs[32c+l]) | (bit 2c+h of qh[l]) << 4.
__device__ __forceinline__ void dq_q5_k(const uint8_t* row, int k, float* w) {
  const uint8_t* b = row + (k / 256) * 176;
  const float d = f16_to_f32(ld_le16(b));
  const float dmin = f16_to_f32(ld_le16(b + 2));
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int t = (k + e) % 256;
    const int c = t >> 6, h = (t >> 5) & 1, l = t & 31, s = t >> 5;
    uint32_t scale, mn;
    k_scale_min(b + 4, s, scale, mn);
    const uint32_t lo = (ld_u8(b + 48 + 32 * c + l) >> (4 * h)) & 15;
    const uint32_t hi = (ld_u8(b + 16 + l) >> s) & 1;
    const uint32_t u = lo | (hi << 4);
    w[e] = (d * static_cast<float>(scale)) * static_cast<float>(u) - dmin * static_cast<float>(mn);
  }
}

// Q6_K: ql[128] | qh[64] | sc[16] | d; t = 128h + 32g + l.
__device__ __forceinline__ void dq_q6_k(const uint8_t* row, int k, float* w) {
  const uint8_t* b = row + (k / 256) * 210;
  const float d = f16_to_f32(ld_le16(b + 208));
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int t = (k + e) % 256;
    const int h = t >> 7, g = (t >> 5) & 3, l = t & 31;
    const uint32_t lo = (ld_u8(b + 64 * h + 32 * (g & 1) + l) >> (4 * (g >> 1))) & 15;
    const uint32_t hi = (ld_u8(b + 128 + 32 * h + l) >> (2 * g)) & 3;
    const int q6 = static_cast<int>(lo | (hi << 4)) - 32;
    const int sc = static_cast<int8_t>(ld_u8(b + 192 + t / 16));
    w[e] = (d * static_cast<float>(sc)) * static_cast<float>(q6);
  }
}

// Q6_K in the plane layout (planes.h): ql[64h + 32m + 16i + t] of block b at
// 4 m a + 64 b + 16 (2h + i) + t, qh[32h + 16i + t] at 8 a + 64 b +
// 16 (2h + i) + t, sc[k] at 12 a + 16 b + k, d at 13 a + 2 b.  Same decode as
// dq_q6_k, byte addresses aside.
constexpr int kQ6KPlanes = 0x103;  // kernel template tag, not a public format
constexpr int kQ5KPlanes = 0x105;  // kernel template tag, not a public format

// Q5_K in the plane layout (planes.h): header of block b at 16 b, qh[l] at
// a + 16 b + l (l < 16) or 2 a + 16 b + l - 16, qs[32c + l] at
// 3 a + 64 b + 16 c + l (l < 16) or 7 a + 64 b + 16 c + l - 16.  Same decode
// as dq_q5_k, byte addresses aside.
__device__ __forceinline__ void dq_q5_k_planes(const uint8_t* w, uint64_t a, int64_t b, int k,
                                               float* out) {
  const uint8_t* h = w + 16 * b;
  const float d = f16_to_f32(ld_le16(h));
  const float dmin = f16_to_f32(ld_le16(h + 2));
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int t = (k + e) % 256;
    const int c = t >> 6, hh = (t >> 5) & 1, l = t & 31, s = t >> 5;
    uint32_t scale, mn;
    k_scale_min(h + 4, s, scale, mn);
    const uint8_t* q = l < 16 ? w + 3 * a + 64 * b + 16 * c + l : w + 7 * a + 64 * b + 16 * c + (l - 16);
    const uint8_t* qh = l < 16 ? w + a + 16 * b + l : w + 2 * a + 16 * b + (l - 16);
    const uint32_t lo = (ld_u8(q) >> (4 * hh)) & 15;
    const uint32_t hi = (ld_u8(qh) >> s) & 1;
    const uint32_t u = lo | (hi << 4);
    out[e] = (d * static_cast<float>(scale)) * static_cast<float>(u) - dmin * static_cast<float>(mn);
  }
}

__device__ __forceinline__ void dq_q6_k_planes(const uint8_t* w, uint64_t a, int64_t b, int k,
                                               float* out) {
  const float d = f16_to_f32(ld_le16(w + 13 * a + 2 * b));
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int t = (k + e) % 256;
    const int h = t >> 7, g = (t >> 5) & 3, l = t & 31;
    const int m = g & 1, i = l >> 4, tt = l & 15, p = 2 * h + i;
    const uint32_t lo = (ld_u8(w + 4 * m * a + 64 * b + 16 * p + tt) >> (4 * (g >> 1))) & 15;
    const uint32_t hi = (ld_u8(w + 8 * a + 64 * b + 16 * p + tt) >> (2 * g)) & 3;
    const int q6 = static_cast<int>(lo | (hi << 4)) - 32;
    const int sc = static_cast<int8_t>(ld_u8(w + 12 * a + 16 * b + t / 16));
    out[e] = (d * static_cast<float>(sc)) * static_cast<float>(q6);
  }
}

// INT4_G128: codes plane (u_{2j} low nibble, u_{2j+1} high) then fp16 scales.
__device__ __forceinline__ void dq_int4(const uint8_t* codes_row, const uint8_t* scales_row,
                                        int k, float* w) {
  const float s = f16_to_f32(ld_le16(scales_row + 2 * (k / 128)));
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int t = k + e;
    const int u = (ld_u8(codes_row + t / 2) >> (4 * (t & 1))) & 15;
    w[e] = s * static_cast<float>(u - 8);
  }
}

__device__ __forceinline__ uint32_t f32_to_bf16_rne(float f) {
  const uint32_t u = __float_as_uint(f);
  return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

__device__ __forceinline__ uint32_t f32_to_f16_rne(float f) {
  return __builtin_bit_cast(uint16_t, static_cast<_Float16>(f));
}

// Weights k .. k + 3 of row r.
template <int FMT>
__device__ __forceinline__ void dq_quad(const uint8_t* w, uint64_t scales_offset, int cols, int r, int k, float* v) {
  if (FMT == QMV_Q8_0) {
    dq_q8_0(w + static_cast<size_t>(r) * (cols / 32) * 34, k, v);
  } else if (FMT == QMV_Q4_K) {
    dq_q4_k(w + static_cast<size_t>(r) * (cols / 256) * 144, k, v);
  } else if (FMT == kQ4KPlanes) {
    dq_q4_k_planes(w, scales_offset, static_cast<int64_t>(r) * (cols / 256) + k / 256, k, v);
  } else if (FMT == kQ5KPlanes) {
    dq_q5_k_planes(w, scales_offset, static_cast<int64_t>(r) * (cols / 256) + k / 256, k, v);
  } else if (FMT == kQ6KPlanes) {
    dq_q6_k_planes(w, scales_offset, static_cast<int64_t>(r) * (cols / 256) + k / 256, k, v);
  } else if (FMT == QMV_Q5_K) {
    dq_q5_k(w + static_cast<size_t>(r) * (cols / 256) * 176, k, v);
  } else if (FMT == QMV_Q6_K) {
    dq_q6_k(w + static_cast<size_t>(r) * (cols / 256) * 210, k, v);
  } else {
    dq_int4(w + static_cast<size_t>(r) * (cols / 2), w + scales_offset + static_cast<size_t>(r) * (cols / 128) * 2, k,
            v);
  }
}

template <int FMT, int OUT>
__global__ void __launch_bounds__(256)
dequant_kernel(const uint8_t* __restrict__ w, uint64_t scales_offset, int rows, int cols,
               void* __restrict__ out) {
  const int64_t quads_per_row = cols / 4;
  const int64_t total = static_cast<int64_t>(rows) * quads_per_row;
  for (int64_t idx = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; idx < total;
       idx += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int r = static_cast<int>(idx / quads_per_row);
    const int k = static_cast<int>(idx % quads_per_row) * 4;
    float v[4];
    dq_quad<FMT>(w, scales_offset, cols, r, k, v);
    const size_t o = static_cast<size_t>(r) * cols + k;
    if (OUT == QMV_F32) {
      *reinterpret_cast<float4*>(static_cast<float*>(out) + o) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      uint32_t h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = OUT == QMV_F16 ? f32_to_f16_rne(v[e]) : f32_to_bf16_rne(v[e]);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + o) =
          make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    }
  }
}

template <int FMT>
static hipError_t dequant_fmt(const qmv_weights& W, void* out, int out_dtype, hipStream_t s) {
  const int rows = static_cast<int>(W.rows), cols = static_cast<int>(W.cols);
  const int64_t total = W.rows * (W.cols / 4);
  const int64_t want = (total + 255) / 256;
  const int grid = static_cast<int>(want < 65536 ? want : 65536);
  const uint8_t* w = static_cast<const uint8_t*>(W.data);
  switch (out_dtype) {
    case QMV_F32:
      hipLaunchKernelGGL((dequant_kernel<FMT, QMV_F32>), dim3(grid), dim3(256), 0, s, w,
                         W.scales_offset, rows, cols, out);
      break;
    case QMV_F16:
      hipLaunchKernelGGL((dequant_kernel<FMT, QMV_F16>), dim3(grid), dim3(256), 0, s, w,
                         W.scales_offset, rows, cols, out);
      break;
    case QMV_BF16:
      hipLaunchKernelGGL((dequant_kernel<FMT, QMV_BF16>), dim3(grid), dim3(256), 0, s, w,
                         W.scales_offset, rows, cols, out);
      break;
    default:
      return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

hipError_t dequant(const qmv_weights& W, void* out, int out_dtype, hipStream_t s) {
  if (W.fmt == QMV_MXFP4) return mx4_dequant(W, out, out_dtype, s);
  if (W.layout == QMV_LAYOUT_PLANES) {
    if (W.fmt == QMV_Q4_K) return dequant_fmt<kQ4KPlanes>(W, out, out_dtype, s);
    if (W.fmt == QMV_Q5_K) return dequant_fmt<kQ5KPlanes>(W, out, out_dtype, s);
    if (W.fmt == QMV_Q6_K) return dequant_fmt<kQ6KPlanes>(W, out, out_dtype, s);
    return hipErrorInvalidValue;
  }
  switch (W.fmt) {
    case QMV_Q8_0: return dequant_fmt<QMV_Q8_0>(W, out, out_dtype, s);
    case QMV_Q4_K: return dequant_fmt<QMV_Q4_K>(W, out, out_dtype, s);
    case QMV_Q5_K: return dequant_fmt<QMV_Q5_K>(W, out, out_dtype, s);
    case QMV_Q6_K: return dequant_fmt<QMV_Q6_K>(W, out, out_dtype, s);
    case QMV_INT4_G128: return dequant_fmt<QMV_INT4_G128>(W, out, out_dtype, s);
    default: return hipErrorInvalidValue;
  }
}

// Sixteen consecutive weights k .. k + 15 of row r (k a multiple of 16: half a
// sub-block of 32, with one scale), by 16-byte loads.  Same arithmetic as
// dq_quad.
template <int FMT>
__device__ __forceinline__ void dq_half(const uint8_t* w, uint64_t scales_offset, int cols, int r, int k, float* v) {
  constexpr bool kQ4 = FMT == QMV_Q4_K || FMT == kQ4KPlanes, kQ5 = FMT == QMV_Q5_K || FMT == kQ5KPlanes;
  auto byte = [](const uint4& x, int i) {
    const uint32_t d = i < 4 ? x.x : i < 8 ? x.y : i < 12 ? x.z : x.w;
    return d >> (8 * (i & 3)) & 255;
  };
  if constexpr (FMT == QMV_Q8_0) {
    const uint8_t* b = w + (static_cast<size_t>(r) * (cols / 32) + k / 32) * 34;
    const float d = f16_to_f32(ld_u16(b));
    const uint4 q = ld16_any(b + 2 + k % 32);
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = d * static_cast<float>(static_cast<int8_t>(byte(q, e)));
  } else if constexpr (FMT == QMV_INT4_G128) {
    const float s = f16_to_f32(ld_u16(w + scales_offset + (static_cast<size_t>(r) * (cols / 128) + k / 128) * 2));
    const uint2 q = ld8_any(w + static_cast<size_t>(r) * (cols / 2) + k / 2);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int u = (e < 8 ? q.x : q.y) >> (4 * (e & 7)) & 15;
      v[e] = s * static_cast<float>(u - 8);
    }
  } else if constexpr (FMT == QMV_MXFP4) {
    const uint32_t p = ld_u8(w + scales_offset + static_cast<size_t>(r) * (cols / 32) + k / 32);
    const uint2 q = ld8_any(w + static_cast<size_t>(r) * (cols / 2) + k / 2);
    mx4_decode8(q.x, p, v);
    mx4_decode8(q.y, p, v + 8);
  } else {
    const size_t blk = static_cast<size_t>(r) * (cols / 256) + k / 256;
    const int t = k % 256, l = t & 16;
    const uint64_t a = scales_offset;
    if constexpr (kQ4 || kQ5) {
      const int c = t >> 6, hh = (t >> 5) & 1, s = t >> 5;
      constexpr bool kPlanes = FMT == kQ4KPlanes || FMT == kQ5KPlanes;
      const uint8_t* h = kPlanes ? w + 16 * blk : w + blk * (kQ4 ? 144 : 176);
      // codes of half l of quarter c, and (Q5_K) the high bits' half
      constexpr int kA = kQ4 ? 1 : 3, kB = kQ4 ? 5 : 7;
      const uint8_t* qp = kPlanes ? w + (l ? kB : kA) * a + 64 * blk + 16 * c : h + (kQ4 ? 16 : 48) + 32 * c + l;
      const uint4 head = ld16_any(h), q = ld16_any(qp);
      uint4 qh = make_uint4(0, 0, 0, 0);
      if constexpr (kQ5) qh = ld16_any(kPlanes ? w + (l ? 2 : 1) * a + 16 * blk : h + 16 + l);
      const float d = f16_to_f32(head.x & 0xFFFF), dmin = f16_to_f32(head.x >> 16);
      // scale bytes 0 .. 11 are head.y, head.z, head.w
      const int sh = 8 * (s & 3);
      const uint32_t b0 = head.y >> sh & 255, b1 = head.z >> sh & 255, b2 = head.w >> sh & 255;
      const uint32_t sc = s < 4 ? b0 & 63 : (b2 & 15) | b0 >> 6 << 4, mn = s < 4 ? b1 & 63 : b2 >> 4 | b1 >> 6 << 4;
      const float ds = d * static_cast<float>(sc), dm = dmin * static_cast<float>(mn);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        uint32_t u = byte(q, e) >> (4 * hh) & 15;
        if constexpr (kQ5) u |= (byte(qh, e) >> s & 1) << 4;
        v[e] = ds * static_cast<float>(u) - dm;
      }
    } else {
      constexpr bool kPlanes = FMT == kQ6KPlanes;
      const int h = t >> 7, gq = (t >> 5) & 3, i = l >> 4, p = 2 * h + i;
      const uint8_t* b = w + blk * 210;
      const uint4 ql = ld16_any(kPlanes ? w + 4 * (gq & 1) * a + 64 * blk + 16 * p : b + 64 * h + 32 * (gq & 1) + l);
      const uint4 qh = ld16_any(kPlanes ? w + 8 * a + 64 * blk + 16 * p : b + 128 + 32 * h + l);
      const int sc = static_cast<int8_t>(ld_u8(kPlanes ? w + 12 * a + 16 * blk + t / 16 : b + 192 + t / 16));
      const float ds = f16_to_f32(ld_u16(kPlanes ? w + 13 * a + 2 * blk : b + 208)) * static_cast<float>(sc);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const uint32_t u = (byte(ql, e) >> (4 * (gq >> 1)) & 15) | (byte(qh, e) >> (2 * gq) & 3) << 4;
        v[e] = ds * static_cast<float>(static_cast<int>(u) - 32);
      }
    }
  }
}

// out[i] = scale * W[ids[i]], a thread for 16 consecutive weights: a 256-thread
// workgroup takes a row's pieces of 4096 columns (grid y), or several narrow
// rows.  16384 rows of 3584 Q8_0 weights to bf16 take 42 us (4.2 TB/s read and
// written; with four weights to a thread, decoded from single bytes, 80 us),
// one Q4_K row 2 us, which is the launch.
template <int FMT, int OUT>
__global__ void __launch_bounds__(256)
embed_kernel(const uint8_t* w, uint64_t scales_offset, int rows, int cols, const int32_t* ids, int64_t n, float scale,
             void* out) {
  const int chunks = cols / 16, per = chunks < 256 ? 256 / chunks : 1;  // rows of a workgroup
  const int sub = chunks < 256 ? static_cast<int>(threadIdx.x) / chunks : 0;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * per + sub;
  if (sub >= per || i >= n) return;
  const int r = ids[i];
  for (int c = chunks < 256 ? static_cast<int>(threadIdx.x) - sub * chunks : blockIdx.y * 256 + threadIdx.x; c < chunks;
       c += gridDim.y * 256) {
    float v[16];
    if (r >= 0 && r < rows) {
      dq_half<FMT>(w, scales_offset, cols, r, c * 16, v);
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] *= scale;
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = 0.f;
    }
    const size_t o = static_cast<size_t>(i) * cols + c * 16;
    if constexpr (OUT == QMV_F32) {
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        *reinterpret_cast<float4*>(static_cast<float*>(out) + o + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
    } else {
      uint32_t h[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (OUT == QMV_F16) {
          h[e] = f32_to_f16_rne(v[2 * e]) | f32_to_f16_rne(v[2 * e + 1]) << 16;
        } else {
          typedef __bf16 b2 __attribute__((ext_vector_type(2)));
          h[e] = __builtin_bit_cast(uint32_t, b2{static_cast<__bf16>(v[2 * e]), static_cast<__bf16>(v[2 * e + 1])});
        }
      }
      uint4* p = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + o);
      p[0] = make_uint4(h[0], h[1], h[2], h[3]);
      p[1] = make_uint4(h[4], h[5], h[6], h[7]);
    }
  }
}

template <int FMT, int OUT>
static hipError_t embed_typed(const qmv_weights& W, const int32_t* ids, int64_t n, float scale, void* out,
                              hipStream_t s) {
  const int rows = static_cast<int>(W.rows), cols = static_cast<int>(W.cols);
  const int chunks = cols / 16, per = chunks < 256 ? 256 / chunks : 1, pieces = (chunks + 255) / 256;
  // A launch's work-items along x are counted in 32 bits (2^32 of them and more
  // wrap around, with no error): more rows than that take several launches.
  const int64_t most = (int64_t{1} << 23) * per;
  for (int64_t i = 0; i < n; i += most) {
    const int64_t k = n - i < most ? n - i : most;
    const dim3 grid(static_cast<unsigned>((k + per - 1) / per), pieces < 65535 ? pieces : 65535);
    hipLaunchKernelGGL((embed_kernel<FMT, OUT>), grid, dim3(256), 0, s, static_cast<const uint8_t*>(W.data),
                       W.scales_offset, rows, cols, ids + i, k, scale,
                       static_cast<uint8_t*>(out) + i * cols * (OUT == QMV_F32 ? 4 : 2));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int FMT>
static hipError_t embed_fmt(const qmv_weights& W, const int32_t* ids, int64_t n, float scale, void* out, int out_dtype,
                            hipStream_t s) {
  switch (out_dtype) {
    case QMV_F32: return embed_typed<FMT, QMV_F32>(W, ids, n, scale, out, s);
    case QMV_F16: return embed_typed<FMT, QMV_F16>(W, ids, n, scale, out, s);
    case QMV_BF16: return embed_typed<FMT, QMV_BF16>(W, ids, n, scale, out, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t embed(const qmv_weights& W, const int32_t* ids, int64_t n, float scale, void* out, int out_dtype,
                 hipStream_t s) {
  if (W.layout == QMV_LAYOUT_PLANES) {
    if (W.fmt == QMV_Q4_K) return embed_fmt<kQ4KPlanes>(W, ids, n, scale, out, out_dtype, s);
    if (W.fmt == QMV_Q5_K) return embed_fmt<kQ5KPlanes>(W, ids, n, scale, out, out_dtype, s);
    if (W.fmt == QMV_Q6_K) return embed_fmt<kQ6KPlanes>(W, ids, n, scale, out, out_dtype, s);
    return hipErrorInvalidValue;
  }
  switch (W.fmt) {
    case QMV_Q8_0: return embed_fmt<QMV_Q8_0>(W, ids, n, scale, out, out_dtype, s);
    case QMV_Q4_K: return embed_fmt<QMV_Q4_K>(W, ids, n, scale, out, out_dtype, s);
    case QMV_Q5_K: return embed_fmt<QMV_Q5_K>(W, ids, n, scale, out, out_dtype, s);
    case QMV_Q6_K: return embed_fmt<QMV_Q6_K>(W, ids, n, scale, out, out_dtype, s);
    case QMV_INT4_G128: return embed_fmt<QMV_INT4_G128>(W, ids, n, scale, out, out_dtype, s);
    case QMV_MXFP4: return embed_fmt<QMV_MXFP4>(W, ids, n, scale, out, out_dtype, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qmv
