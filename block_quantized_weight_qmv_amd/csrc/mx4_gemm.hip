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
#include <math.h>

#include <algorithm>
#include <cmath>
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

// The experts' groups of rows come from expert_start as its running maximum,
// clamped to the rows there are, so that no content reaches outside them.  All
// lanes of a wave call together; lane l holds expert base + l: its first row,
// its end, and the tiles of bm rows up to and with its own.
struct Groups {
  int first, last, sum;
  __device__ __forceinline__ void load(const Mx4Launch& a, int bm, int base, int carry, int before) {
    const int lane = __lane_id(), i = base + lane;
    last = i < a.experts ? min(max(a.expert_start[i + 1], 0), a.rows) : 0;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(last, d);
      last = lane >= d ? max(last, o) : last;
    }
    last = max(last, carry);
    first = __shfl_up(last, 1);
    first = lane ? first : carry;
    sum = (last - first + bm - 1) / bm;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(sum, d);
      sum = lane >= d ? sum + o : sum;
    }
    sum += before;
  }
};

// The lane's number, or what follows from it, worked out here again: numbers that
// stay the same from tile to tile would otherwise be kept in registers, which
// the products need.
__device__ __forceinline__ int again(int v) {
  __asm__ __volatile__("" : "+v"(v));
  return v;
}

// A tile: its expert, first row and end of the group, and its column of tiles.
struct Tile {
  int e, row, end, tn;
};

// The tiles of a launch in the order they are worked on.  Workgroups go to the
// eight XCDs in turn, each with an L2 of its own: an XCD takes a run of
// consecutive tiles, in bands of kBand tiles of rows, so that the 32 tiles it
// works on together share eight row tiles and four column tiles.
constexpr int kBand = 8;
struct Tiles {
  Groups g;
  int tiles_m, tiles_n, bm, carry;

  __device__ __forceinline__ void init(const Mx4Launch& a, int bm_, int tiles_n_) {
    bm = bm_, tiles_n = tiles_n_;
    if (!a.expert_start) {
      tiles_m = (a.rows + bm - 1) / bm;
      return;
    }
    carry = min(max(a.expert_start[0], 0), a.rows);
    int c = carry;
    tiles_m = 0;
    for (int base = 0; base < a.experts; base += 64) {
      g.load(a, bm, base, c, tiles_m);
      c = __builtin_amdgcn_readlane(g.last, 63), tiles_m = __builtin_amdgcn_readlane(g.sum, 63);
    }
  }

  // This XCD's run: first tile and end.
  __device__ __forceinline__ void run(int& first, int& end) const {
    const int total = tiles_m * tiles_n, xcd = blockIdx.x & 7, each = total >> 3;
    first = xcd * each + min(xcd, total & 7);
    end = first + each + (xcd < (total & 7));
  }

  __device__ __forceinline__ Tile at(const Mx4Launch& a, int i) {
    const int band = i / (kBand * tiles_n), in = i - band * (kBand * tiles_n), wide = min(kBand, tiles_m - band * kBand);
    Tile t;
    t.tn = in / wide;
    const int m = band * kBand + in - t.tn * wide;
    if (!a.expert_start) {
      t.e = 0, t.row = m * bm, t.end = a.rows;
      return t;
    }
    t.e = 0;
    if (a.experts > 64) {  // more than one scan: find its part again
      int c = carry, before = 0;
      for (;; t.e += 64) {
        g.load(a, bm, t.e, c, before);
        before = __builtin_amdgcn_readlane(g.sum, 63);
        if (m < before) break;
        c = __builtin_amdgcn_readlane(g.last, 63);
      }
    }
    const int l = __builtin_ctzll(__ballot(m < g.sum));
    const int first = __builtin_amdgcn_readlane(g.first, l);
    t.e += l;
    t.end = __builtin_amdgcn_readlane(g.last, l);
    // tiles of this group from m on: those up to its end
    t.row = first + (m - (__builtin_amdgcn_readlane(g.sum, l) - (t.end - first + bm - 1) / bm)) * bm;
    return t;
  }
};

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

// 16 bytes of each lane, from base + off, to LDS at `lds` + 16 x lane.  (The s_nop
// covers an M0, base or offset written just before, which the compiler cannot see
// being used here; waits and barriers that no memory access crosses keep LDS
// reads apart from the copies.)
__device__ __forceinline__ void copy16(const uint8_t* base, uint32_t off, uint32_t lds) {
  __asm__ __volatile__("s_mov_b32 m0, %2\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(off), "s"(base), "s"(lds) : "m0");
}

// Eight scale bytes of a row from block b on (a multiple of eight before its
// end; bytes past the end are anything), at any alignment and within the row.
__device__ __forceinline__ uint2 scales8(const uint8_t* p, int b, int blocks) {
  if (b + 8 <= blocks) return ld8_any(p + b);
  uint64_t v = 0;
  if (blocks >= 8) {
    const uint2 d = ld8_any(p + blocks - 8);
    v = (d.x | static_cast<uint64_t>(d.y) << 32) >> (8 * (b + 8 - blocks));
  } else {
    for (int i = 0; i < blocks - b; ++i) v |= static_cast<uint64_t>(p[b + i]) << (8 * i);
  }
  return make_uint2(static_cast<uint32_t>(v), static_cast<uint32_t>(v >> 32));
}

// Few activation rows: 16 MT of them against 16 NT weight rows (with GLU every
// other sixteen of the gate and of up) to a workgroup.  Its W waves take every
// W-th piece of 256 columns (a whole line of every row) and add their sums in
// LDS.  Fragments go from memory to the matrix instruction without LDS, D
// pieces of a wave ahead: the weights' bytes bound it, and what is in flight
// decides how near it comes (16 rows against 2 x 18944 x 3584 with GLU 18.1 us,
// 4.0 TB/s; 32 rows of 18 experts of 2 x 2560 x 3584 41.4 us, 4.2 TB/s).
template <int NT, int MT, int W, int D, int OUT, bool GLU>
__global__ void __launch_bounds__(64 * W)
mx4_stream_kernel(const Mx4Launch a, int tiles_n) {
  constexpr int kOuts = 16 * NT / (GLU ? 2 : 1);
  __shared__ float part[W][NT * MT * 4][64];
  Tiles tiles;
  tiles.init(a, 16 * MT, tiles_n);
  int first, run_end;
  tiles.run(first, run_end);
  first += blockIdx.x >> 3;
  if (first >= run_end) return;
  const Tile at = tiles.at(a, first);
  const int lane = __lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
  const int blocks = a.k / 32, pieces = (blocks + 7) / 8;
  // rows of the weight tiles, then of the activation tiles (past the end: the last one again, not stored)
  const uint8_t *codes[NT + MT], *powers[NT + MT];
  const int64_t base = static_cast<int64_t>(at.e) * (GLU ? 2 : 1) * a.n;
  unrolled<NT + MT>([&](auto t) {
    int64_t j;
    if constexpr (t < NT) {
      const int n = at.tn * kOuts + 16 * (GLU ? t / 2 : t) + r;
      j = base + min(n, a.n - 1) + (GLU && (t & 1) ? a.n : 0);
    } else {
      const int i = min(at.row + 16 * (t - NT) + r, at.end - 1);
      j = a.x_index ? a.x_index[i] : i;
      if (j < 0 || j >= a.x_rows) j = 0;  // (such a row's outputs are zeros below)
    }
    codes[t] = (t < NT ? a.w : a.x) + j * blocks * 16;
    powers[t] = (t < NT ? a.ws : a.xs) + j * blocks;
  });
  v4f_t acc[NT][MT];
  unrolled<NT>([&](auto t) { unrolled<MT>([&](auto m) { acc[t][m] = v4f_t{0.f, 0.f, 0.f, 0.f}; }); });
  struct Piece {
    uint4 c[NT + MT][2];
    uint2 p[NT + MT];
  } f[D];
  auto load = [&](Piece& f, int u) {  // blocks 8 u + g and 8 u + 4 + g of each lane's row (past the last: that one)
    unrolled<NT + MT>([&](auto t) {
      f.c[t][0] = ld16(codes[t] + 16 * static_cast<int64_t>(min(8 * u + g, blocks - 1)));
      f.c[t][1] = ld16(codes[t] + 16 * static_cast<int64_t>(min(8 * u + 4 + g, blocks - 1)));
    });
    unrolled<NT + MT>([&](auto t) { f.p[t] = scales8(powers[t], 8 * u, blocks); });
  };
  unrolled<D>([&](auto d) {
    if (wave + d * W < pieces) load(f[d], wave + d * W);
  });
  for (int u0 = wave; u0 < pieces; u0 += D * W) {
    unrolled<D>([&](auto d) {
      const int u = u0 + d * W;
      if (u >= pieces) return;
      if (8 * u + 8 > blocks) {  // past the row's end: a zero factor
        unrolled<MT>([&](auto m) {
          if (8 * u + g >= blocks) f[d].c[NT + m][0] = make_uint4(0, 0, 0, 0);
          if (8 * u + 4 + g >= blocks) f[d].c[NT + m][1] = make_uint4(0, 0, 0, 0);
        });
      }
      unrolled<2>([&](auto h) {
        uint32_t p[NT + MT];
        unrolled<NT + MT>([&](auto t) { p[t] = (h ? f[d].p[t].y : f[d].p[t].x) >> (8 * g); });
        unrolled<NT>([&](auto t) {
          unrolled<MT>([&](auto m) { acc[t][m] = mfma4(f[d].c[t][h], f[d].c[NT + m][h], acc[t][m], p[t], p[NT + m]); });
        });
      });
      if (u + D * W < pieces) load(f[d], u + D * W);
    });
  }
  unrolled<NT>([&](auto t) {
    unrolled<MT>([&](auto m) {
#pragma unroll
      for (int i = 0; i < 4; ++i) part[wave][(t * MT + m) * 4 + i][lane] = acc[t][m][i];
    });
  });
  __syncthreads();
  // the waves share the results
  constexpr int kResults = (GLU ? NT / 2 : NT) * MT * 4;
  for (int j = wave; j < kResults; j += W) {
    const int i = j & 3, m = j / 4 % MT, t = j / (4 * MT);
    auto sum = [&](int of) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) v += part[w][(of * MT + m) * 4 + i][lane];
      return v;
    };
    const int yr = at.row + 16 * m + r, col = at.tn * kOuts + 16 * t + 4 * g + i;
    float v = GLU ? silu_mul(sum(2 * t), sum(2 * t + 1)) : sum(t);
    if (yr >= at.end || col >= a.n) continue;
    if (a.x_index && (a.x_index[yr] < 0 || a.x_index[yr] >= a.x_rows)) v = 0.f;
    store_one<OUT>(a.y, yr * a.y_row + col, v);
  }
}

// The first of the four outputs that lane quarter q holds of group p, among
// its wave's: 16 bytes of a lane, and 64 of four, are neighbours in y.
template <int OUT>
__device__ __forceinline__ int place(int p, int q) {
  return OUT == QMV_F32 ? 16 * p + 4 * q : 32 * (p >> 1) + 8 * q + 4 * (p & 1);
}

// Place of the 16-byte piece `piece` among the four of row r (of 64 bytes in
// LDS): a read of 16 rows at one piece meets 16 different places of the 256
// bytes that LDS serves a clock, in the order it takes lanes.
__device__ __forceinline__ int slot4(int piece, int r) { return piece ^ (0x78 >> (r >> 1 & 6) & 3); }

// Many activation rows: tiles of 16 WN TN weight rows x 16 WM TM activation
// rows, WN x WM waves of TN x TM matrix instructions each.
//
// A stage is 128 columns of all the tile's rows, copied straight to LDS, into a
// ring of four: while stage s is multiplied, stage s + 1 is read into registers
// two fragments ahead of its use, and s + 2 and s + 3 are on their way.  One
// barrier a stage says both that stage s + 1 has come and that stage s - 1 is
// read.  Scales take another way (a row's are few bytes, at any alignment): 32
// blocks' bytes of each row are loaded by four lanes, turned so that a lane's
// four stages are a dword, and kept in LDS; the matrix instruction picks the
// stage's byte.
//
// A workgroup stays for as many tiles as there are (grid = what the GPU holds):
// the next tile's first stages, and its scales, are loaded while this one's
// last stages are multiplied, and its results leave while the next one begins.
//
// Bound: the copies to LDS (a wave's instruction of 1 KB takes about 27 clocks,
// four a stage and wave) and what is done once a stage, beside the matrix
// instructions: their pipes are busy 37 % of the clocks, and waves wait for a third
// of theirs.  4096 rows against 18944 x 3584 take 162 us (3.4 PFLOP/s; with random
// codes and operands in registers alone 6.5 to 7.2), 32768 rows of 27 experts of
// 2 x 2560 x 2048 258 us (2.7).
template <int WN, int WM, int TN, int TM, int OUT, bool GLU>
__global__ void __launch_bounds__(64 * WN * WM) __attribute__((amdgpu_waves_per_eu(2, 2)))
mx4_tile_kernel(const Mx4Launch a, int tiles_n) {
  constexpr int kWaves = WN * WM, BN = 16 * WN * TN, BM = 16 * WM * TM, kRows = BN + BM, kStage = kRows * 64;
  constexpr int kCopies = kRows / 16 / kWaves;  // a wave's copy instructions of a stage: 16 rows x 64 bytes each
  constexpr int kOuts = 16 * TN / (GLU ? 2 : 1);  // outputs of a wave's rows
  constexpr int kAhead = 2;                       // weight fragments read ahead of their use
  static_assert(kRows == 64 * kWaves, "whole copies, and 4 KB of a stage, to a wave");
  __shared__ __attribute__((aligned(128))) uint8_t ring[4 * kStage];
  __shared__ __attribute__((aligned(128))) uint8_t scales[kRows * 32];
  const int lane = __lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave % WN, wm = wave / WN, r = lane & 15, g = lane >> 4;
  const int blocks = a.k / 32, stages = (blocks + 3) / 4;
  Tiles tiles;
  tiles.init(a, BM, tiles_n);
  int at, run_end;
  tiles.run(at, run_end);
  at += blockIdx.x >> 3;
  const int step = gridDim.x >> 3;
  if (at >= run_end) return;
  Tile tile = tiles.at(a, at), next = tile;

  // Row t of a tile in the matrices: weights first.  A wave's groups of 16
  // weight rows are dealt so that a lane's results are neighbours in y.
  auto weight_row = [&](const Tile& to, int t) {
    const int w = t / (16 * TN), gr = t / 16 % TN, q = t / 4 & 3, i = t & 3;
    const int n = to.tn * (WN * kOuts) + w * kOuts + place<OUT>(GLU ? gr >> 1 : gr, q) + i;
    return (GLU ? gr & 1 : 0) * a.n + min(n, a.n - 1);
  };
  auto activation_row = [&](int i) {  // (past the group's end: its last row again, not stored)
    const int j = a.x_index ? a.x_index[i] : i;
    return j >= 0 && j < a.x_rows ? j : -1;
  };

  // Lane l of copy c serves row 16 (kCopies wave + c) + l / 4, piece l % 4.  A
  // row is known by its bytes from the start of its expert's codes, or of the
  // activations' (a sixteenth of that in the scales).
  const bool weights = wave < BN / 16 / kCopies;  // this wave copies weight rows, or activation rows
  const int64_t matrix = static_cast<int64_t>(GLU ? 2 : 1) * a.n * blocks;  // blocks of an expert's matrix
  struct Source {
    const uint8_t *codes, *powers;
    uint32_t row[kCopies];
  } from, next_from;
  uint32_t none = 0, next_none = 0;  // bit j: this lane's activation row 16 j + r has no index
  auto find_rows = [&](const Tile& to) {
    const int lane = again(threadIdx.x & 63), r = lane & 15;
    unrolled<kCopies>([&](auto c) {
      const int t = 16 * (kCopies * wave + c) + (lane >> 2);
      next_from.row[c] = weights ? 0 : max(activation_row(min(to.row + t - BN, to.end - 1)), 0);
    });
    next_none = 0;
    if (a.x_index) {
#pragma unroll
      for (int j = 0; j < TM; ++j)
        next_none |= activation_row(min(to.row + 16 * (wm * TM + j) + r, to.end - 1)) < 0 ? 1u << j : 0;
    }
  };
  auto find_blocks = [&](const Tile& to) {
    const int lane = again(threadIdx.x & 63);
    unrolled<kCopies>([&](auto c) {
      const int t = 16 * (kCopies * wave + c) + (lane >> 2);
      next_from.row[c] = (weights ? weight_row(to, t) : next_from.row[c]) * static_cast<uint32_t>(blocks) * 16;
    });
    next_from.codes = weights ? a.w + 16 * (to.e * matrix) : a.x;
    next_from.powers = weights ? a.ws + to.e * matrix : a.xs;
  };
  const uint32_t lds = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(&ring[0]));
  const int block = slot4(lane & 3, lane >> 2);
  auto copy_stage = [&](const Source& f, int s, int to) {
    const uint32_t off = 16 * min(4 * s + block, blocks - 1);
    unrolled<kCopies>([&](auto c) { copy16(f.codes, f.row[c] + off, lds + to * kStage + 1024 * (kCopies * wave + c)); });
  };

  // Scales of 32 blocks from 32 S on: piece l % 4 of a row is 8 bytes, its last
  // ones moved to their places where the row ends inside.
  uint2 sv[kCopies];
  auto load_scales = [&](const Source& f, int S) {
    const int b0 = 32 * S + 8 * (again(lane) & 3);
    unrolled<kCopies>([&](auto c) {
      if (b0 < blocks) sv[c] = scales8(f.powers + (f.row[c] >> 4), b0, blocks);
    });
  };
  // Bytes g and 4 + g of a piece are two stages of lanes of quarter g.
  auto keep_scales = [&]() {
    const int lane = again(threadIdx.x & 63);
    unrolled<kCopies>([&](auto c) {
      const int t = 16 * (kCopies * wave + c) + (lane >> 2), piece = lane & 3;
      uint8_t* to = &scales[32 * t + 4 * ((piece >> 1) ^ (t >> 3 & 1)) + 2 * (piece & 1)];
      const uint32_t lo = __builtin_amdgcn_perm(sv[c].y, sv[c].x, 0x05010400);
      const uint32_t hi = __builtin_amdgcn_perm(sv[c].y, sv[c].x, 0x07030602);
      *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(lo);
      *reinterpret_cast<uint16_t*>(to + 8) = static_cast<uint16_t>(lo >> 16);
      *reinterpret_cast<uint16_t*>(to + 16) = static_cast<uint16_t>(hi);
      *reinterpret_cast<uint16_t*>(to + 24) = static_cast<uint16_t>(hi >> 16);
    });
    __asm__ __volatile__("s_waitcnt lgkmcnt(0)" ::: "memory");
  };

  const int lane_at = 64 * r + 16 * slot4(g, r);
  v4f_t acc[TN][TM];
  uint4 wf[TN + kAhead], xf[2][TM];  // activations of even and odd stages
  uint32_t sa[TN], sb[TM], sbn[TM];
  int base = 0;  // the ring's place of the tile's first stage
  auto read_w = [&](int s, int i) {
    return *reinterpret_cast<const uint4*>(&ring[((base + s) & 3) * kStage + 1024 * (wn * TN + i) + lane_at]);
  };
  auto read_x = [&](int s, int j) {
    return *reinterpret_cast<const uint4*>(&ring[((base + s) & 3) * kStage + 64 * BN + 1024 * (wm * TM + j) + lane_at]);
  };
  // scales of four stages from s on: byte j for stage s + j
  auto read_scale = [&](int s, int t) -> uint32_t {
    return *reinterpret_cast<const uint32_t*>(&scales[32 * (t + r) + 8 * g + 4 * ((s >> 2 & 1) ^ (r >> 3))]);
  };

  bool begun = false;  // the tile's first stages and scales came while the one before was worked on
  int ahead_of = 0, wait_from = 0;  // stages that copies are ahead of; the first stage that waits
  const int tail = (blocks & 3) ? stages - 1 : -1;
  bool has_next = false;
  const bool ahead = stages >= 4;  // tiles of fewer stages begin only when the one before has ended
  auto stage = [&](auto quarter, int s) {
    // (a tile begun ahead has its first three stages, and the results of the
    // one before may still be leaving)
    if (quarter >= 2 || s >= wait_from) __asm__ __volatile__("s_waitcnt vmcnt(%0)" ::"n"(kCopies) : "memory");
    __asm__ __volatile__("s_barrier" ::: "memory");
    if constexpr (quarter == 1) {
      if ((s & 4) && s + 3 < stages) keep_scales();  // read from stage s + 2 on
    }
    if (s + 3 == stages && has_next) from = next_from, ahead_of = stages;
    // (after the last tile's last stage: its last blocks again, read by nobody)
    copy_stage(from, s + 3 - ahead_of, (base + s + 3) & 3);
    if constexpr (quarter == 2) {
      if (!(s & 4) && s + 6 < stages) load_scales(from, (s >> 3) + 1);
    }
    if (s == tail) {  // the row ends inside: a zero factor behind its end
#pragma unroll
      for (int j = 0; j < TM; ++j)
        if (4 * s + g >= blocks) xf[quarter & 1][j] = make_uint4(0, 0, 0, 0);
    }
    unrolled<TN>([&](auto i) {
      if constexpr (i + kAhead < TN)
        wf[i + kAhead] = read_w(s, i + kAhead);
      else
        wf[i + kAhead] = read_w(s + 1, i + kAhead - TN);
      if constexpr (i >= TN - TM) xf[~quarter & 1][i - (TN - TM)] = read_x(s + 1, i - (TN - TM));
      if constexpr ((quarter == 3) && i < TM) sbn[i] = read_scale(s + 1, BN + 16 * (wm * TM + i));
      unrolled<TM>([&](auto j) { acc[i][j] = mfma4s<quarter, quarter>(wf[i], xf[quarter & 1][j], acc[i][j], sa[i], sb[j]); });
      if constexpr (quarter == 3) sa[i] = read_scale(s + 1, 16 * (wn * TN + i));
      __builtin_amdgcn_sched_barrier(0);
    });
#pragma unroll
    for (int i = 0; i < kAhead; ++i) wf[i] = wf[TN + i];
    if constexpr (quarter == 3) {
#pragma unroll
      for (int j = 0; j < TM; ++j) sb[j] = sbn[j];
    }
  };

  for (;;) {
    if (!begun) {
      find_rows(tile);
      find_blocks(tile);
      load_scales(next_from, 0);
#pragma unroll
      for (int s = 0; s < 3; ++s) copy_stage(next_from, s, (base + s) & 3);
      keep_scales();
      __asm__ __volatile__("s_waitcnt vmcnt(0)" ::: "memory");
    }
    none = next_none;
    from = next_from;
    ahead_of = 0;
    wait_from = begun ? 2 : 0;
    lds_barrier();
#pragma unroll
    for (int j = 0; j < TM; ++j) xf[0][j] = read_x(0, j), sb[j] = read_scale(0, BN + 16 * (wm * TM + j));
#pragma unroll
    for (int i = 0; i < TN; ++i) sa[i] = read_scale(0, 16 * (wn * TN + i));
#pragma unroll
    for (int i = 0; i < kAhead; ++i) wf[i] = read_w(0, i);
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) acc[i][j] = v4f_t{0.f, 0.f, 0.f, 0.f};
    at += step;
    const bool more = at < run_end;
    has_next = more && ahead;
    if (more) next = tiles.at(a, at);
    // (the next tile's rows are looked up once this one's loads are under way)
    const int look = stages >= 12 ? 4 : 0, number = 2 * look;
    for (int s = 0; s < stages; s += 4) {
      if (has_next) {
        if (s == look) find_rows(next);
        if (s == number) find_blocks(next);
        if (s + 4 >= stages) load_scales(next_from, 0);
      }
      stage(std::integral_constant<int, 0>{}, s);
      if (s + 1 < stages) stage(std::integral_constant<int, 1>{}, s + 1);
      if (s + 2 < stages) stage(std::integral_constant<int, 2>{}, s + 2);
      if (s + 3 < stages) stage(std::integral_constant<int, 3>{}, s + 3);
    }
    // all waves have read the last stage and the scales
    __asm__ __volatile__("s_waitcnt vmcnt(0)" ::: "memory");
    lds_barrier();
    if (has_next) keep_scales();
    base = (base + stages) & 3;

    // Results, 16 rows by 256 bytes at a time, through the wave's share of the
    // ring's free stage, so that a store instruction writes four whole pieces of
    // 256 bytes.  Lane (r, g) holds activation row 16 j + r and, of a group or
    // (16-bit outputs) two, neighbours of 16 bytes.
    constexpr int kSize = OUT == QMV_F32 ? 4 : 2, kPer = 16 / kSize, kEach = kPer / 4;
    constexpr int kGroups = GLU ? TN / 2 : TN, kRowBytes = kOuts * kSize < 256 ? kOuts * kSize : 256;
    constexpr int kTurns = kOuts * kSize / kRowBytes, kTurn = kGroups / kTurns, kChunks = kRowBytes / 16;
    static_assert(kTurn % kEach == 0 && kChunks >= 4 && 16 * kRowBytes <= 4096, "a turn's rows fit a wave's share");
    uint8_t* out = &ring[((base + 3) & 3) * kStage + 4096 * wave];
    const int lane = again(threadIdx.x & 63), r = lane & 15, g = lane >> 4;
    unrolled<TM * kTurns>([&](auto turn) {
      constexpr int j = turn / kTurns, p0 = turn % kTurns * kTurn;
      const bool zero = none >> j & 1;
#pragma unroll
      for (int p = 0; p < kTurn; p += kEach) {
        float v[kPer];
#pragma unroll
        for (int c = 0; c < kPer; ++c) {
          const int i = p0 + p + c / 4;
          if constexpr (GLU)
            v[c] = silu_mul(acc[2 * i][j][c % 4], acc[2 * i + 1][j][c % 4]);
          else
            v[c] = acc[i][j][c % 4];
          v[c] = zero ? 0.f : v[c];
        }
        uint4 d;
        if constexpr (OUT == QMV_F32)
          d = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        else if constexpr (OUT == QMV_F16)
          d = make_uint4(pack_f16(v[0], v[1]), pack_f16(v[2], v[3]), pack_f16(v[4], v[5]), pack_f16(v[6], v[7]));
        else
          d = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
        const int chunk = place<OUT>(p, g) / kPer;
        *reinterpret_cast<uint4*>(out + r * kRowBytes + 16 * ((chunk ^ r) & (kChunks - 1))) = d;
      }
      __asm__ __volatile__("s_waitcnt lgkmcnt(0)" ::: "memory");
      constexpr int kLines = 64 / kChunks;  // rows of a store instruction
#pragma unroll
      for (int i = 0; i < 16 / kLines; ++i) {
        const int o = i * kLines + lane / kChunks, chunk = lane % kChunks;
        const int yr = tile.row + 16 * (wm * TM + j) + o;
        const int n = tile.tn * (WN * kOuts) + wn * kOuts + place<OUT>(p0, 0) + chunk * kPer;
        const uint4 d = *reinterpret_cast<const uint4*>(out + o * kRowBytes + 16 * ((chunk ^ o) & (kChunks - 1)));
        if (yr >= tile.end || n >= a.n) continue;
        uint8_t* y = static_cast<uint8_t*>(a.y) + (yr * a.y_row + n) * kSize;
        if (n + kPer <= a.n) {
          __builtin_nontemporal_store(u32x4_a2{d.x, d.y, d.z, d.w}, reinterpret_cast<u32x4_a2*>(y));
        } else {
          const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
          for (int c = 0; c < kPer; ++c)
            if (n + c < a.n) {
              if constexpr (kSize == 4)
                reinterpret_cast<uint32_t*>(y)[c] = w[c];
              else
                reinterpret_cast<uint16_t*>(y)[c] = static_cast<uint16_t>(w[c / 2] >> (16 * (c & 1)));
            }
        }
      }
      __asm__ __volatile__("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before the next turn's writes
    });
    if (!more) return;
    tile = next;
    begun = has_next;
    if (!begun) lds_barrier();  // everybody's results are out of the ring
  }
}

// Tiles of bm rows that the experts' groups have at most.
static int64_t most_tiles(const Mx4Launch& a, int bm) {
  const int64_t whole = (a.rows + bm - 1) / bm;
  if (!a.expert_start) return whole;
  return whole + std::min(a.experts, a.rows);
}

// Tiles that rows spread unevenly over the experts are likely to take.
static double usual_tiles(const Mx4Launch& a, int bm) {
  if (!a.expert_start) return (a.rows + bm - 1) / bm;
  const double used = std::min(a.experts, a.rows), each = a.rows / (used * bm);
  return used * (each <= 0.5 ? 1 : each + 0.5);
}

// Columns of tiles of 16 nt weight rows.
static double tiles_n_of(const Mx4Launch& a, bool glu, int nt) {
  return std::ceil(a.n / (16.0 * nt / (glu ? 2 : 1)));
}

template <int WN, int WM, int TN, int TM, int OUT, bool GLU>
static hipError_t launch_tile(const Mx4Launch& a, hipStream_t s) {
  constexpr int outs = 16 * WN * TN / (GLU ? 2 : 1);
  const int64_t tiles_n = (static_cast<int64_t>(a.n) + outs - 1) / outs, tiles_m = most_tiles(a, 16 * WM * TM);
  const int64_t held = static_cast<int64_t>(device_cus()) * (WN * WM == 8 ? 1 : 2);
  const int64_t grid = (std::min(tiles_m * tiles_n, held) + 7) / 8 * 8;  // each XCD's workgroups share its run
  hipLaunchKernelGGL((mx4_tile_kernel<WN, WM, TN, TM, OUT, GLU>), dim3(static_cast<unsigned>(grid)),
                     dim3(64 * WN * WM), 0, s, a, static_cast<int>(tiles_n));
  return hipGetLastError();
}

template <int NT, int MT, int W, int D, int OUT, bool GLU>
static hipError_t launch_stream(const Mx4Launch& a, hipStream_t s) {
  constexpr int outs = 16 * NT / (GLU ? 2 : 1);
  const int64_t tiles_n = (static_cast<int64_t>(a.n) + outs - 1) / outs, tiles_m = most_tiles(a, 16 * MT);
  hipLaunchKernelGGL((mx4_stream_kernel<NT, MT, W, D, OUT, GLU>),
                     dim3(static_cast<unsigned>((tiles_m * tiles_n + 7) / 8 * 8)), dim3(64 * W), 0, s, a,
                     static_cast<int>(tiles_n));
  return hipGetLastError();
}

// What a launch of tiles of 16 nt weight rows x 16 mt activation rows is expected
// to take (us), at 3584 columns: `lone` where no CU has more than one, else `each`
// for every one of the fullest CU's.
static double stream_cost(const Mx4Launch& a, bool glu, int nt, int mt, double each, double lone) {
  const double tiles = tiles_n_of(a, glu, nt) * usual_tiles(a, 16 * mt);
  // (a launch's work-items along x are counted in 32 bits)
  if (tiles_n_of(a, glu, nt) * most_tiles(a, 16 * mt) >= 1 << 22) return 1e30;
  return 2.5 + a.k / 3584.0 * (tiles <= 256 ? lone : each * std::ceil(tiles / 256));
}

template <int OUT, bool GLU>
static hipError_t launch(const Mx4Launch& a, hipStream_t s) {
  // The kernel that is expected to end first.  The figures are measured ones at
  // 3584 columns: for a stream kernel, time a tile takes of a CU that has several,
  // and a lone tile's; for the tile kernels, time of one tile on each CU, and
  // (128 x 128) of two.  All seven in this order, us (bf16 outputs, no GLU, weights
  // beyond the caches), * the one chosen:
  //   rows x outputs x columns
  //     16 x  1024 x  3584    4.5*   5.4    8.1    6.0    6.9   15.4   28.1
  //     16 x 18944 x  3584   13.9   13.1*  15.0   17.3   20.9   17.9   31.9
  //     16 x  3584 x 18944   14.0*  18.6   32.3   21.3   26.1   66.2    122
  //     64 x  3584 x  3584   10.2    8.3    8.4    6.9*   9.5   15.7   28.2
  //     64 x 18944 x  3584   37.9   33.1   29.1   30.4   27.8   18.3*  31.4
  //    256 x  3584 x  3584   28.0   23.1   22.4   23.2   17.8   16.1*  29.3
  //    512 x 18944 x  3584    265    223    180    212    164   44.4   35.9*
  //   1024 x  3584 x  3584    100   84.8   69.6   78.1   59.0   17.1*  29.9
  //   4096 x 18944 x  3584   2072   1725   1380   1649   1256    240    186*
  // (with GLU, 32 rows of 18 of 32 experts of 2560 outputs: 64.8, 49.0, 40.7*, 72.5,
  // 83.9, 46.1, 70.9)
  const double small = tiles_n_of(a, GLU, 8) * usual_tiles(a, 128), large = tiles_n_of(a, GLU, 16) * usual_tiles(a, 256);
  const double rest = small - 512 * std::floor(small / 512);
  const double cost[7] = {GLU ? 1e30 : stream_cost(a, GLU, 1, 1, 2.2, 2.1), stream_cost(a, GLU, 2, 1, 3.4, 2.8),
                          stream_cost(a, GLU, 4, 1, 5.2, 5.7),            stream_cost(a, GLU, 2, 2, 5.8, 4.0),
                          stream_cost(a, GLU, 2, 4, 8.6, 6.5),
                          2.5 + a.k / 3584.0 * (20 * std::floor(small / 512) + (rest == 0 ? 0 : rest <= 256 ? 13.3 : 20)),
                          2.5 + a.k / 3584.0 * 27 * std::max(1.0, large / 256)};
  switch (std::min_element(cost, cost + 7) - cost) {
    case 0: return launch_stream<GLU ? 2 : 1, 1, 8, 2, OUT, GLU>(a, s);
    case 1: return launch_stream<2, 1, 8, 1, OUT, GLU>(a, s);
    case 2: return launch_stream<4, 1, 4, 2, OUT, GLU>(a, s);
    case 3: return launch_stream<2, 2, 8, 2, OUT, GLU>(a, s);
    case 4: return launch_stream<2, 4, 8, 1, OUT, GLU>(a, s);
    case 5: return launch_tile<2, 2, 4, 4, OUT, GLU>(a, s);
    default: return launch_tile<2, 4, 8, 4, OUT, GLU>(a, s);
  }
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

// The tile kernels number their tiles, and the bytes of a matrix and of the
// activations, in 32 bits.
bool mx4_gemm_fits(const qmv_mx4_args& m) {
  const Mx4Launch a = describe(m);
  const int64_t row = a.k / 2, matrix = m.W->rows / a.experts * row;
  return most_tiles(a, 128) * ((static_cast<int64_t>(a.n) + 63) / 64) < (int64_t{1} << 28) &&
         matrix <= (int64_t{1} << 32) && a.x_rows * row <= (int64_t{1} << 32);
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
