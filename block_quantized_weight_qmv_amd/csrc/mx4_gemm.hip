// Products of MXFP4 activations with MXFP4 weights on the scaled matrix
// instructions, dense or grouped by expert:
//   y[i][j] = sum_k X[idx(i)][k] W[e(i)][j][k],  e(i) the expert whose rows hold i
// optionally silu(gate) * up of the two halves of an expert's rows.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes, from lane (r = l % 16, g = l / 16),
// 32 codes of row r (16 bytes) and their scale byte: exactly one MXFP4 block, so
// codes go from memory to the instruction as they are.  A product of two codes
// is exact, sums are fp32.  Weights are the A operand, activations B: a lane's
// four results are four consecutive outputs of one activation row.
#include <algorithm>

#include "launch.h"
#include "mx4.h"

namespace qmv {

typedef int v8i_t __attribute__((ext_vector_type(8)));
typedef float v4f_t __attribute__((ext_vector_type(4)));

struct Mx4Launch {
  const uint8_t *w, *ws, *x, *xs;  // codes and scales of W and X
  const int32_t *expert_start, *x_index;
  void* y;
  int64_t y_row;
  int experts, rows, n, k, x_rows;  // n: outputs of a row (the gate's rows, with glu)
};

// silu(g) u, g / (1 + 2^(-g log2 e)): the exponent's rounding is put back to
// first order (it would cost |g| 2^-24); beyond |g| = 120 the quotient is 0 or g.
__device__ __forceinline__ float silu_mul(float g, float u) {
  constexpr float kL = 1.44269504088896f, kL2 = 1.92596299e-8f, kLn2 = 0.69314718f;  // kL + kL2: log2 e
  const float c = fminf(fmaxf(g, -120.f), 120.f);
  const float t = -c * kL;
  const float r = fmaf(-c, kL, -t) - c * kL2;
  const float e = __builtin_amdgcn_exp2f(t) * fmaf(r, kLn2, 1.f);
  return g * __builtin_amdgcn_rcpf(1.f + e) * u;
}

// Tile t of BM rows over the experts' groups: its expert, first row and the
// group's end.  Groups come from expert_start as its running maximum, clamped
// to the rows there are, so that no content reaches outside them.  All lanes of
// a wave call it together.  False: there are fewer tiles.
__device__ __forceinline__ bool find_tile(const Mx4Launch& a, int bm, int t, int& e, int& row, int& end) {
  if (!a.expert_start) {
    e = 0, row = t * bm, end = a.rows;
    return row < end;
  }
  const int lane = __lane_id();
  int carry = min(max(a.expert_start[0], 0), a.rows);
  for (int base = 0; base < a.experts; base += 64) {
    const int i = base + lane;
    int last = i < a.experts ? min(max(a.expert_start[i + 1], 0), a.rows) : 0;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(last, d);
      last = lane >= d ? max(last, o) : last;
    }
    last = max(last, carry);
    int first = __shfl_up(last, 1);
    first = lane ? first : carry;
    const int mine = (last - first + bm - 1) / bm;
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(sum, d);
      sum = lane >= d ? sum + o : sum;
    }
    const uint64_t past = __ballot(t < sum);
    if (past) {
      const int l = __builtin_ctzll(past);
      e = base + l;
      row = __shfl(first, l) + (t - __shfl(sum - mine, l)) * bm;
      end = __shfl(last, l);
      return true;
    }
    t -= __shfl(sum, 63);
    carry = __shfl(last, 63);
  }
  return false;
}

__device__ __forceinline__ v4f_t mfma4(const uint4& a, const uint4& b, v4f_t c, uint32_t sa, uint32_t sb) {
  const v8i_t va = {static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z), static_cast<int>(a.w), 0, 0, 0, 0};
  const v8i_t vb = {static_cast<int>(b.x), static_cast<int>(b.y), static_cast<int>(b.z), static_cast<int>(b.w), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(va, vb, c, 4, 4, 0, static_cast<int>(sa), 0,
                                                          static_cast<int>(sb));
}

template <int OUT>
__device__ __forceinline__ void store_one(void* y, int64_t at, float v) {
  if constexpr (OUT == QMV_F32)
    static_cast<float*>(y)[at] = v;
  else if constexpr (OUT == QMV_F16)
    static_cast<_Float16*>(y)[at] = static_cast<_Float16>(v);
  else
    static_cast<uint16_t*>(y)[at] = static_cast<uint16_t>(pack_bf16(v, 0.f));
}

// Few activation rows: 16 MT of them against 32 weight rows (with GLU 16 of the
// gate and the same 16 of up) to a workgroup, whose four waves share the
// columns (every fourth piece of 512) and add their sums in LDS.
template <int MT, int OUT, bool GLU>
__global__ void __launch_bounds__(256)
mx4_stream_kernel(const Mx4Launch a, int tiles_n) {
  __shared__ float part[4][2 * MT * 4][64];
  const int tn = blockIdx.x % tiles_n, tm = blockIdx.x / tiles_n;
  int e, row, end;
  if (!find_tile(a, 16 * MT, tm, e, row, end)) return;
  const int lane = __lane_id(), wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int blocks = a.k / 32;
  const int64_t kc = a.k / 2;
  // rows of the two weight tiles and of the activation tiles (past the end: the last one again, not stored)
  const uint8_t *wc[2], *wp[2], *xc[MT], *xp[MT];
  const int64_t base = static_cast<int64_t>(e) * (GLU ? 2 : 1) * a.n;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int64_t j = base + (GLU ? min(16 * tn + r, a.n - 1) + t * a.n : min(32 * tn + 16 * t + r, a.n - 1));
    wc[t] = a.w + j * kc;
    wp[t] = a.ws + j * blocks;
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int i = min(row + 16 * t + r, end - 1);
    int64_t j = a.x_index ? a.x_index[i] : i;
    if (j < 0 || j >= a.x_rows) j = 0;  // (such a row's outputs are zeros below)
    xc[t] = a.x + j * kc;
    xp[t] = a.xs + j * blocks;
  }
  v4f_t acc[2][MT];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[t][m] = v4f_t{0.f, 0.f, 0.f, 0.f};
  for (int b0 = 4 * wave; b0 < blocks; b0 += 16) {  // 128 columns: block b0 + g of each lane's row
    const int b = min(b0 + g, blocks - 1);
    uint4 wv[2], xv[MT];
    uint32_t wq[2], xq[MT];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      wv[t] = ld16(wc[t] + 16 * b);
      wq[t] = wp[t][b];
      if (b0 + g >= blocks) wv[t] = make_uint4(0, 0, 0, 0);  // past the row: a zero factor
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      xv[m] = ld16(xc[m] + 16 * b);
      xq[m] = xp[m][b];
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[t][m] = mfma4(wv[t], xv[m], acc[t][m], wq[t], xq[m]);
  }
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[wave][(t * MT + m) * 4 + i][lane] = acc[t][m][i];
  __syncthreads();
  // a wave joins a quarter of the results
  for (int j = wave; j < (GLU ? 1 : 2) * MT * 4; j += 4) {
    float v = 0.f, u = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) v += part[w][j][lane];
    const int m = j / 4 % MT, i = j & 3, t = j / (4 * MT);
    const int yr = row + 16 * m + r, col = (GLU ? 16 : 32) * tn + 16 * t + 4 * g + i;
    if constexpr (GLU) {
#pragma unroll
      for (int w = 0; w < 4; ++w) u += part[w][j + 4 * MT][lane];
      v = silu_mul(v, u);
    }
    if (yr >= end || col >= a.n) continue;
    if (a.x_index && (a.x_index[yr] < 0 || a.x_index[yr] >= a.x_rows)) v = 0.f;
    store_one<OUT>(a.y, yr * a.y_row + col, v);
  }
}

// Tiles of bm rows that the experts' groups have at most.
static int64_t most_tiles(const Mx4Launch& a, int bm) {
  const int64_t whole = (a.rows + bm - 1) / bm;
  if (!a.expert_start) return whole;
  return whole + std::min(a.experts, a.rows);
}

template <int OUT, bool GLU>
static hipError_t launch(const Mx4Launch& a, hipStream_t s) {
  const int tiles_n = (a.n + (GLU ? 15 : 31)) / (GLU ? 16 : 32);
  const int64_t tiles_m = most_tiles(a, 16);
  hipLaunchKernelGGL((mx4_stream_kernel<1, OUT, GLU>), dim3(static_cast<unsigned>(tiles_m * tiles_n)), dim3(256), 0, s, a,
                     tiles_n);
  return hipGetLastError();
}

template <int OUT>
static hipError_t launch_glu(const Mx4Launch& a, bool glu, hipStream_t s) {
  return glu ? launch<OUT, true>(a, s) : launch<OUT, false>(a, s);
}

static Mx4Launch describe(const qmv_mx4_args& m) {
  Mx4Launch a;
  a.w = static_cast<const uint8_t*>(m.W->data), a.ws = a.w + m.W->scales_offset;
  a.x = static_cast<const uint8_t*>(m.X->data), a.xs = a.x + m.X->scales_offset;
  a.expert_start = m.expert_start, a.x_index = m.x_index;
  a.y = m.y, a.y_row = m.y_row;
  a.experts = m.experts ? m.experts : 1;
  a.rows = static_cast<int>(m.rows);
  a.n = static_cast<int>(m.W->rows / a.experts / (m.epilogue == QMV_MX4_SWIGLU ? 2 : 1));
  a.k = static_cast<int>(m.W->cols), a.x_rows = static_cast<int>(m.X->rows);
  return a;
}

bool mx4_gemm_fits(const qmv_mx4_args& m) {
  const Mx4Launch a = describe(m);
  return most_tiles(a, 16) * ((static_cast<int64_t>(a.n) + 15) / 16) < (int64_t{1} << 24);
}

hipError_t mx4_gemm(const qmv_mx4_args& m, hipStream_t s) {
  const Mx4Launch a = describe(m);
  const bool glu = m.epilogue == QMV_MX4_SWIGLU;
  switch (m.y_dtype) {
    case QMV_F32: return launch_glu<QMV_F32>(a, glu, s);
    case QMV_F16: return launch_glu<QMV_F16>(a, glu, s);
    default: return launch_glu<QMV_BF16>(a, glu, s);
  }
}

}  // namespace qmv
