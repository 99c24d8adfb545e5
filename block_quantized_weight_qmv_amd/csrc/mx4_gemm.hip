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
#include <type_traits>

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

typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));

// N neighbours at y + at, aligned by their type alone.
template <int OUT, int N>
__device__ __forceinline__ void store_many(void* y, int64_t at, const float* v) {
  if constexpr (OUT == QMV_F32) {
    u32x4_a2* p = reinterpret_cast<u32x4_a2*>(static_cast<float*>(y) + at);
#pragma unroll
    for (int i = 0; i < N; i += 4)
      p[i / 4] = u32x4_a2{__float_as_uint(v[i]), __float_as_uint(v[i + 1]), __float_as_uint(v[i + 2]), __float_as_uint(v[i + 3])};
  } else {
    u32x4_a2* p = reinterpret_cast<u32x4_a2*>(static_cast<uint16_t*>(y) + at);
    auto two = [&](int k) { return OUT == QMV_F16 ? pack_f16(v[k], v[k + 1]) : pack_bf16(v[k], v[k + 1]); };
#pragma unroll
    for (int i = 0; i < N; i += 8) p[i / 8] = u32x4_a2{two(i), two(i + 2), two(i + 4), two(i + 6)};
  }
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

template <int N, class F>
__device__ __forceinline__ void unrolled(F f) {
  if constexpr (N > 0) {
    unrolled<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
  }
}

template <int SA, int SB>
__device__ __forceinline__ v4f_t mfma4s(const uint4& a, const uint4& b, v4f_t c, uint32_t sa, uint32_t sb) {
  const v8i_t va = {static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z), static_cast<int>(a.w), 0, 0, 0, 0};
  const v8i_t vb = {static_cast<int>(b.x), static_cast<int>(b.y), static_cast<int>(b.z), static_cast<int>(b.w), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(va, vb, c, 4, 4, SA, static_cast<int>(sa), SB,
                                                          static_cast<int>(sb));
}

// 16 bytes of each lane from memory to LDS at `lds` + 16 x lane.  (The s_nop
// covers an M0 or address written just before, which the compiler cannot see
// being used here; waits and barriers that no memory access crosses keep LDS
// reads apart from the copies.)
__device__ __forceinline__ void copy16(const uint8_t* src, uint32_t lds) {
  __asm__ __volatile__("s_mov_b32 m0, %1\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(src), "s"(lds) : "m0");
}

// Sixteen-row groups of a tile whose scales share a dword.
constexpr int kQuad = 4;

// Many activation rows: a tile of 16 WN TN weight rows x 16 WM TM activation
// rows, WN x WM waves of TN x TM matrix instructions each.
template <int WN, int WM, int TN, int TM, int OUT, bool GLU>
__global__ void __launch_bounds__(64 * WN * WM)
mx4_tile_kernel(const Mx4Launch a, int tiles_n) {
  constexpr int kWaves = WN * WM, BN = 16 * WN * TN, BM = 16 * WM * TM, kRows = BN + BM;
  constexpr int kCopies = kRows / 8 / kWaves;  // copy instructions of a wave for a stage: 8 rows x 128 bytes each
  constexpr int kScaleRows = (kRows + 64 * kWaves - 1) / (64 * kWaves);
  constexpr int kQuads = kRows / 16 / kQuad;
  static_assert(kRows % (8 * kWaves) == 0 && TN % kQuad == 0 && TM % kQuad == 0, "whole copies and scale dwords");
  __shared__ __attribute__((aligned(128))) uint8_t tile[2][kRows * 128];
  __shared__ uint32_t scales[2][8][kQuads][16];  // [stage][block][four groups][row]: a byte for each group
  const int total = gridDim.x, tn = blockIdx.x % tiles_n, tm = blockIdx.x / tiles_n;
  (void)total;
  int e, row, end;
  if (!find_tile(a, BM, tm, e, row, end)) return;
  const int lane = __lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int blocks = a.k / 32, stages = (blocks + 7) / 8;
  const int64_t kc = a.k / 2;

  // The matrix row of row t of the tile: weights first.  A wave's groups of 16
  // weight rows are dealt so that a lane's results are neighbours in y.
  auto source = [&](int t, const uint8_t*& codes, const uint8_t*& powers) {
    if (t < BN) {
      const int w = t / (16 * TN), g = t / 16 % TN, q = t / 4 & 3, i = t & 3;
      int64_t j;
      if constexpr (GLU) {
        const int n = tn * (BN / 2) + w * (8 * TN) + q * (2 * TN) + (g >> 1) * 4 + i;
        j = min(n, a.n - 1) + static_cast<int64_t>(g & 1) * a.n;
      } else {
        j = min(tn * BN + w * (16 * TN) + q * (4 * TN) + g * 4 + i, a.n - 1);
      }
      j += static_cast<int64_t>(e) * (GLU ? 2 : 1) * a.n;
      codes = a.w + j * kc;
      powers = a.ws + j * blocks;
    } else {
      const int i = min(row + t - BN, end - 1);
      int64_t j = a.x_index ? a.x_index[i] : i;
      if (j < 0 || j >= a.x_rows) j = 0;  // (such a row's outputs are zeros below)
      codes = a.x + j * kc;
      powers = a.xs + j * blocks;
    }
  };

  // Copies: lane l of copy c takes 16 bytes of row 8 (kCopies wave + c) + l / 8,
  // the block that the permutation puts into slot l % 8.
  const uint8_t* src[kCopies];
  int block[kCopies];
#pragma unroll
  for (int c = 0; c < kCopies; ++c) {
    const int t = 8 * (kCopies * wave + c) + (lane >> 3);
    const uint8_t* unused;
    source(t, src[c], unused);
    block[c] = (lane & 7) ^ ((t >> 1) & 7);
  }
  const uint32_t lds = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(&tile[0][0]));
  const uint8_t* sp[kScaleRows];
#pragma unroll
  for (int c = 0; c < kScaleRows; ++c) {
    const uint8_t* unused;
    source(min(static_cast<int>(threadIdx.x) + c * 64 * kWaves, kRows - 1), unused, sp[c]);
  }
  auto copy_stage = [&](int s) {
#pragma unroll
    for (int c = 0; c < kCopies; ++c)
      copy16(src[c] + 16 * min(8 * s + block[c], blocks - 1),
             lds + (s & 1) * (kRows * 128) + 1024 * (kCopies * wave + c));
  };
  uint2 sv[kScaleRows];
  auto load_scales = [&](int s) {
#pragma unroll
    for (int c = 0; c < kScaleRows; ++c) {
      if (8 * s + 8 <= blocks) {
        sv[c] = ld8_any(sp[c] + 8 * s);
      } else {
        uint32_t d[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i / 4] |= static_cast<uint32_t>(sp[c][min(8 * s + i, blocks - 1)]) << (8 * (i & 3));
        sv[c] = make_uint2(d[0], d[1]);
      }
    }
  };
  auto keep_scales = [&](int s) {
#pragma unroll
    for (int c = 0; c < kScaleRows; ++c) {
      const int t = static_cast<int>(threadIdx.x) + c * 64 * kWaves;
      if (kRows % (64 * kWaves) != 0 && t >= kRows) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        reinterpret_cast<uint8_t*>(&scales[s & 1][i][t / 16 / kQuad][t & 15])[t / 16 % kQuad] =
            static_cast<uint8_t>((i < 4 ? sv[c].x : sv[c].y) >> (8 * (i & 3)));
    }
  };

  const int wn = wave % WN, wm = wave / WN, r = lane & 15, g = lane >> 4;
  v4f_t acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = v4f_t{0.f, 0.f, 0.f, 0.f};

  copy_stage(0);
  load_scales(0);
  for (int s = 0; s < stages; ++s) {
    keep_scales(s);
    __asm__ __volatile__("s_waitcnt vmcnt(0)" ::: "memory");
    lds_barrier();
    if (s + 1 < stages) {
      copy_stage(s + 1);
      load_scales(s + 1);
    }
    const uint8_t* buf = tile[s & 1];
    const bool tail = 8 * s + 8 > blocks;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int slot = 16 * ((4 * h + g) ^ ((r >> 1) & 7));
      uint32_t sa[TN / kQuad], sb[TM / kQuad];
      uint4 xb[TM];
#pragma unroll
      for (int i = 0; i < TN / kQuad; ++i) sa[i] = scales[s & 1][4 * h + g][wn * (TN / kQuad) + i][r];
#pragma unroll
      for (int j = 0; j < TM / kQuad; ++j) sb[j] = scales[s & 1][4 * h + g][BN / 16 / kQuad + wm * (TM / kQuad) + j][r];
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        xb[j] = *reinterpret_cast<const uint4*>(buf + (BN + 16 * (wm * TM + j) + r) * 128 + slot);
        if (tail && 8 * s + 4 * h + g >= blocks) xb[j] = make_uint4(0, 0, 0, 0);  // past the row: a zero factor
      }
      unrolled<TN>([&](auto i) {
        const uint4 w = *reinterpret_cast<const uint4*>(buf + (16 * (wn * TN + i) + r) * 128 + slot);
        unrolled<TM>([&](auto j) {
          acc[i][j] = mfma4s<i % kQuad, j % kQuad>(w, xb[j], acc[i][j], sa[i / kQuad], sb[j / kQuad]);
        });
      });
    }
  }

  // Lane (r, q): activation row 16 j + r of the wave's, neighbouring outputs.
  constexpr int kOuts = GLU ? 2 * TN : 4 * TN;
  const int n0 = (GLU ? tn * (BN / 2) + wn * (8 * TN) : tn * BN + wn * (16 * TN)) + g * kOuts;
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    const int yr = row + 16 * (wm * TM + j) + r;
    if (yr >= end || n0 >= a.n) continue;
    float v[kOuts];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if constexpr (GLU) {
          if (i & 1) v[(i >> 1) * 4 + c] = silu_mul(acc[i - 1][j][c], acc[i][j][c]);
        } else {
          v[i * 4 + c] = acc[i][j][c];
        }
      }
    if (a.x_index && (a.x_index[yr] < 0 || a.x_index[yr] >= a.x_rows)) {
#pragma unroll
      for (int i = 0; i < kOuts; ++i) v[i] = 0.f;
    }
    const int64_t at = yr * a.y_row + n0;
    if (n0 + kOuts <= a.n) {
      store_many<OUT, kOuts>(a.y, at, v);
    } else {
#pragma unroll
      for (int i = 0; i < kOuts; ++i)
        if (n0 + i < a.n) store_one<OUT>(a.y, at + i, v[i]);
    }
  }
}

// Tiles of bm rows that the experts' groups have at most.
static int64_t most_tiles(const Mx4Launch& a, int bm) {
  const int64_t whole = (a.rows + bm - 1) / bm;
  if (!a.expert_start) return whole;
  return whole + std::min(a.experts, a.rows);
}

template <int WN, int WM, int TN, int TM, int OUT, bool GLU>
static hipError_t launch_tile(const Mx4Launch& a, hipStream_t s) {
  constexpr int outs = 16 * WN * TN / (GLU ? 2 : 1);
  const int64_t tiles_n = (static_cast<int64_t>(a.n) + outs - 1) / outs, tiles_m = most_tiles(a, 16 * WM * TM);
  hipLaunchKernelGGL((mx4_tile_kernel<WN, WM, TN, TM, OUT, GLU>), dim3(static_cast<unsigned>(tiles_m * tiles_n)),
                     dim3(64 * WN * WM), 0, s, a, static_cast<int>(tiles_n));
  return hipGetLastError();
}

template <int OUT, bool GLU>
static hipError_t launch(const Mx4Launch& a, hipStream_t s) {
  const int64_t per = a.rows / a.experts;  // rows of a matrix, on average
  if (per > 512) return launch_tile<2, 4, 8, 4, OUT, GLU>(a, s);
  if (per > 32) return launch_tile<2, 2, 4, 4, OUT, GLU>(a, s);
  const int64_t tiles_n = (static_cast<int64_t>(a.n) + (GLU ? 15 : 31)) / (GLU ? 16 : 32);
  const int64_t tiles_m = most_tiles(a, 16);
  hipLaunchKernelGGL((mx4_stream_kernel<1, OUT, GLU>), dim3(static_cast<unsigned>(tiles_m * tiles_n)), dim3(256), 0, s, a,
                     static_cast<int>(tiles_n));
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
