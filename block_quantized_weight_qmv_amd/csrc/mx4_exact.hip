// MXFP4 weights times several fp16 or bf16 activation rows, exactly, on the
// matrix cores: y[b][r] = sum_k W[r][k] x[b][k], fp32.
//
// A weight is a 4-bit float times a power of two: a bf16 number, exactly (where
// it is an fp32 number at all), which the conversion instruction makes of two
// codes and their scale at once.  A bf16 activation is one, an fp16 activation
// the sum of two bf16 numbers (8 + 3 of its 11 bits), which enter one product
// each.  So products are exact and sums fp32, as in the GEMV; the order of sums
// differs from it.
//
// v_mfma_f32_16x16x32_bf16 takes eight numbers of row l % 16 from each lane: a
// quarter of the lane's own MXFP4 block, and the same columns of the
// activations.  The frame is that of the MXFP4 products for few rows: 16 NT
// weight rows x 16 activation rows to a workgroup, every eighth piece of 256
// columns to a wave, the sums joined in LDS.
//
// Bound: few loads in flight and many a byte (an activation row of 16 bits is four
// times a weight row): 3 fp16 rows against 3584 x 18944 take 19.1 us (22.3 in the
// GEMV's passes of two rows), 1.9 TB/s of weights; 16 rows 30 us (against 96).
#include "launch.h"
#include "mx4.h"

namespace qmv {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));


// Eight codes times 2^(p - 127), p as its float.
__device__ __forceinline__ bf16x8_t weights8(uint32_t q, float scale) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 0);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 1);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 2);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 3);
  return bf16x8_t{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// v without its first bits; of an infinity that infinity again, and of a NaN NaN
// (fp16 ends at 65504, which changes no finite number here; 3 rows as above take
// 17.6 us without it, infinities then being NaN)
__device__ __forceinline__ float rest(float v, uint32_t first) {
  return v - __builtin_amdgcn_fmed3f(__uint_as_float(first), -65504.f, 65504.f);
}

// Eight fp16 numbers as hi + lo, two bf16 numbers each: the first eight bits,
// and the rest.
__device__ __forceinline__ void halves8(const uint4& raw, bf16x8_t& hi, bf16x8_t& lo) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = f16_to_f32(w[i] & 0xFFFFu), b = f16_to_f32(w[i] >> 16);
    const uint32_t ua = __float_as_uint(a) & 0xFFFF0000u, ub = __float_as_uint(b) & 0xFFFF0000u;
    h[i] = __builtin_amdgcn_perm(ub, ua, 0x07060302);
    l[i] = __builtin_amdgcn_perm(__float_as_uint(rest(b, ub)), __float_as_uint(rest(a, ua)), 0x07060302);
  }
  hi = __builtin_bit_cast(bf16x8_t, make_uint4(h[0], h[1], h[2], h[3]));
  lo = __builtin_bit_cast(bf16x8_t, make_uint4(l[0], l[1], l[2], l[3]));
}

template <int NT, int W, typename XT>
__global__ void __launch_bounds__(64 * W)
mx4_exact_kernel(const uint8_t* w, const uint8_t* ws, int rows, int cols, const XT* x, int batch, float* y, int tiles_n) {
  __shared__ float part[W][NT * 4][64];
  const int tn = blockIdx.x % tiles_n, tm = blockIdx.x / tiles_n;
  const int lane = __lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
  const int blocks = cols / 32, pieces = (blocks + 7) / 8;
  const uint8_t *codes[NT], *powers[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {  // (past the end: the last row again, not stored)
    const int64_t j = min((tn * NT + t) * 16 + r, rows - 1);
    codes[t] = w + j * blocks * 16;
    powers[t] = ws + j * blocks;
  }
  const XT* xr = x + static_cast<int64_t>(min(tm * 16 + r, batch - 1)) * cols;
  f32x4_t acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  struct Piece {
    uint4 c[NT][2], x[2][4];
    uint32_t p[NT][2];
  };
  auto load = [&](Piece& f, int u) {  // blocks 8 u + g and 8 u + 4 + g (past the row's last: that one)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t b = min(8 * u + 4 * h + g, blocks - 1);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        f.c[t][h] = ld16(codes[t] + 16 * b);
        f.p[t][h] = powers[t][b];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) f.x[h][j] = reinterpret_cast<const uint4*>(xr + 32 * b)[j];
    }
  };
  Piece f[2];
  auto use = [&](Piece& f, int u) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = 8 * u + 4 * h + g < blocks;
      float scale[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) scale[t] = mx4_scale(f.p[t][h]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint4 raw = f.x[h][j];
        if (!in) raw = make_uint4(0, 0, 0, 0);  // past the row's end: a zero factor
        bf16x8_t hi, lo;
        if constexpr (__is_same(XT, bf16_t))
          hi = __builtin_bit_cast(bf16x8_t, raw);
        else
          halves8(raw, hi, lo);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const uint32_t q = j == 0 ? f.c[t][h].x : j == 1 ? f.c[t][h].y : j == 2 ? f.c[t][h].z : f.c[t][h].w;
          const bf16x8_t v = weights8(q, scale[t]);
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, hi, acc[t], 0, 0, 0);
          if constexpr (!__is_same(XT, bf16_t)) acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, lo, acc[t], 0, 0, 0);
        }
      }
    }
  };
  if (wave < pieces) load(f[0], wave);
  if (wave + W < pieces) load(f[1], wave + W);
  for (int u = wave; u < pieces; u += 2 * W) {
    use(f[0], u);
    if (u + 2 * W < pieces) load(f[0], u + 2 * W);
    if (u + W < pieces) use(f[1], u + W);
    if (u + 3 * W < pieces) load(f[1], u + 3 * W);
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[wave][t * 4 + i][lane] = acc[t][i];
  __syncthreads();
  for (int j = wave; j < NT * 4; j += W) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) v += part[k][j][lane];
    const int row = (tn * NT + j / 4) * 16 + 4 * g + (j & 3), b = tm * 16 + r;
    if (row < rows && b < batch) y[static_cast<int64_t>(b) * rows + row] = v;
  }
}

template <int NT, int W, typename XT>
static hipError_t launch_exact(const GemvCall& c, int64_t batch, hipStream_t s) {
  const uint8_t* w = static_cast<const uint8_t*>(c.W->data);
  const int tiles_n = static_cast<int>((c.W->rows + 16 * NT - 1) / (16 * NT));
  const int64_t tiles = tiles_n * ((batch + 15) / 16);
  if (tiles >= int64_t{1} << 22) return hipErrorInvalidValue;
  hipLaunchKernelGGL((mx4_exact_kernel<NT, W, XT>), dim3(static_cast<unsigned>(tiles)), dim3(64 * W), 0, s, w,
                     w + c.W->scales_offset, static_cast<int>(c.W->rows), static_cast<int>(c.W->cols),
                     static_cast<const XT*>(c.x), static_cast<int>(batch), c.y, tiles_n);
  return hipGetLastError();
}

// Two weight tiles to a workgroup where that still gives every compute unit one.
template <typename XT>
static hipError_t exact(const GemvCall& c, int64_t batch, hipStream_t s) {
  return (c.W->rows + 31) / 32 * ((batch + 15) / 16) >= 256 ? launch_exact<2, 8, XT>(c, batch, s) : launch_exact<1, 16, XT>(c, batch, s);
}

bool mx4_exact_fits(int64_t rows, int64_t batch) {
  return (rows + 15) / 16 * ((batch + 15) / 16) < (int64_t{1} << 22);
}

hipError_t mx4_exact(const GemvCall& c, int x_dtype, int64_t batch, hipStream_t s) {
  return x_dtype == QMV_F16 ? exact<_Float16>(c, batch, s) : exact<bf16_t>(c, batch, s);
}

}  // namespace qmv
