// Attention of a step's rows over a prefix that the whole batch shares and
// their own sequences' paged suffixes:
//   o = sum_j p_j v_j / sum_j p_j,  p_j = e^(scale q.k_j - m),  m = max_j scale q.k_j,
// over the prefix tokens and the suffix tokens that the row sees.
//
// One launch walks the keys, a second joins the parts.  The query heads that
// share a key head, of all rows of the step, stand side by side as rows of one
// matrix, so a prefix key is read once per 128 (wide) or 32 (narrow) of them
// and not once per sequence; a sequence's own keys meet its own rows only.
// The keys of the prefix, and of long suffixes, are split over workgroups,
// each of which keeps a running maximum and sum and leaves its unnormalized
// output, maximum and sum in the workspace.
//
// The products are computed transposed, S^T = K Q^T and O^T = V^T P^T, on
// 32x32x16 matrix instructions.  A lane then holds one row's scores (row =
// lane & 31; key 8 (r / 4) + 4 (lane / 32) + r % 4 in register r), so the
// softmax needs no exchange between lanes but one of two halves when the
// maximum moves, and those registers are, in order, the second product's B
// operand: its k index runs over the keys in that same order, which V's
// transposing LDS reads follow.  P never goes through LDS.
//
// K and V tiles go from memory to LDS without passing registers.  16-byte
// chunks of a tile's row are permuted by the row's number so that neither
// product's reads meet in a bank (swz_k, swz_v); the copy fills LDS in order,
// so each lane asks for the chunk that belongs at its place.
#include <float.h>

#include "device_util.h"
#include "launch.h"

namespace qmv {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;
// "No key yet" as a running maximum (finite, so that differences are numbers).
constexpr float kNone = -FLT_MAX;
// A maximum is replaced only when a score passes it by more than this many
// binary orders: until then the exponentials, at most 2^8, lose nothing in
// fp32 or in the second product's types, and the 32..128 outputs of a lane
// need no rescaling.
constexpr float kSlack = 8.f;
// Keys of one workgroup where they lie in pages: their page numbers are held in LDS.
constexpr int kMaxPagedKeys = 2048;

// Where the keys of a workgroup come from.
struct KeySource {
  const uint8_t* k;       // key head's first element of token or page 0
  const uint8_t* v;
  const int32_t* table;   // NULL: contiguous tokens
  int64_t row;            // bytes from one token to the next (within a page)
  int64_t page;           // bytes from one page to the next
  int shift, npages;      // log2 of the page size
};

struct AttnPlan {
  int groups;        // query heads per key head
  int wide;          // prefix: 128-row tiles of four waves (else 32-row tiles, four waves along the keys)
  int row_tiles;     // prefix row tiles per key head
  int psplits, pseg; // prefix key ranges and their keys
  int srow_tiles;    // suffix row tiles per sequence and key head
  int ssplits, sseg;
  int64_t prefix_wgs;  // workgroups before the suffixes'
  int64_t suffix_wgs;
};

struct AttnKernelArgs {
  qmv_attn_args a;
  AttnPlan p;
  float* po;         // [slot][row * heads + head][D]
  float2* pml;       // [slot][row * heads + head]: maximum (log2), sum
};

// What tokens past a range's end and pages outside the pool are read from.
__device__ const uint4 g_zero_row[32] = {};

template <int DP>
__device__ __forceinline__ int swz_k(int row) {
  return DP == 64 ? (row >> 1) & 7 : row & 7;
}
template <int DP>
__device__ __forceinline__ int swz_v(int row) {
  return DP == 64 ? ((row >> 1) & 3) * 2 : (row & 7) * 2;
}

// 64 lanes x 16 bytes from memory to LDS at `lds` (+ 16 x lane).  The s_nop
// covers an M0 or address written just before, which the compiler cannot see
// being used here.
__device__ __forceinline__ void copy_to_lds(const void* src, uint32_t lds) {
  __asm__ __volatile__("s_mov_b32 m0, %1\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %0, off"
                       :
                       : "v"(src), "s"(lds)
                       : "memory");
}
__device__ __forceinline__ void copy_to_lds(const void* base, uint32_t off, uint32_t lds) {
  __asm__ __volatile__("s_mov_b32 m0, %2\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %0, %1"
                       :
                       : "v"(off), "s"(base), "s"(lds)
                       : "memory");
}
template <int N>
__device__ __forceinline__ void wait_copies() {  // all but the last N
  __asm__ __volatile__("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}
// The wave's own LDS reads are done: what they read may be overwritten.
__device__ __forceinline__ void wait_lds() { __asm__ __volatile__("s_waitcnt lgkmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void order_memory() { __asm__ __volatile__("" ::: "memory"); }

template <bool BF>
__device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// x and y as two values of the type each: hi + lo holds 16 bits or more.
template <bool BF>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t& hi, uint32_t& lo) {
  if constexpr (BF) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    const uint32_t bx = __float_as_uint(x), by = __float_as_uint(y);
    hi = __builtin_amdgcn_perm(by, bx, 0x07060302);
    const float rx = x - __uint_as_float(bx & 0xFFFF0000u), ry = y - __uint_as_float(by & 0xFFFF0000u);
    lo = __builtin_bit_cast(uint32_t, b2{static_cast<__bf16>(rx), static_cast<__bf16>(ry)});
  } else {
    const h2_t h = __builtin_bit_cast(h2_t, __builtin_amdgcn_cvt_pkrtz(x, y));
    hi = __builtin_bit_cast(uint32_t, h);
    lo = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(x - static_cast<float>(h.x), y - static_cast<float>(h.y)));
  }
}

// A wave's 32 rows against a stream of key tiles.
template <bool BF, int DP>
struct RowTile {
  static constexpr int KS = DP / 16, DT = DP / 32, CPR = DP / 8, ROWB = DP * 2;
  u32x4 q[KS];
  f32x16 o[DT];
  float m, l;
  float c;  // scale log2 e

  // qp: this lane's row (its first element); d past D counts as zero.
  __device__ __forceinline__ void init(const uint16_t* qp, int D, float scale, int lane) {
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int d = s * 16 + 8 * (lane >> 5);
      u32x4 z = {0, 0, 0, 0};
      q[s] = d < D ? *reinterpret_cast<const u32x4*>(qp + d) : z;
    }
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[t][i] = 0.f;
    m = kNone;
    l = 0.f;
    c = scale * kLog2e;
  }

  // Scores of NT x 32 keys.
  template <int NT>
  __device__ __forceinline__ void scores(const lds_u8* kt, int lane, f32x16* s) {
    const int r = lane & 31, h = lane >> 5;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < 16; ++i) s[t][i] = 0.f;
      const lds_u8* row = kt + (t * 32 + r) * ROWB;
      const int z = swz_k<DP>(r);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const u32x4 kf = *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>(row + (((2 * ks + h) ^ z) << 4));
        s[t] = mfma<BF>(kf, q[ks], s[t]);
      }
    }
  }

  // Scores to unnormalized probabilities, the running maximum and sum.
  template <int NT>
  __device__ __forceinline__ void softmax(f32x16* s) {
    float mx = s[0][0];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[t][i]);
    if (__any(mx * c > m + kSlack)) {
      const float both = fmaxf(mx, __shfl_xor(mx, 32));
      const float mn = fmaxf(m, both * c);
      const float f = __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[t][i] *= f;
    }
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[t][i] = __builtin_amdgcn_exp2f(fmaf(s[t][i], c, -m));
        sum[i & 3] += s[t][i];
      }
    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
  }

  // o += V^T P^T over NT x 32 keys.
  template <int NT>
  __device__ __forceinline__ void values(const lds_u8* vt, int lane, const f32x16* s) {
    const int h = lane >> 5, g = (lane >> 4) & 1, a = (lane >> 2) & 3, b = lane & 3;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        u32x4 hi, lo;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t x, y;
          split_pair<BF>(s[t][8 * ks + 2 * k], s[t][8 * ks + 2 * k + 1], x, y);
          hi[k] = x;
          lo[k] = y;
        }
        // lane (h, g, a, b): key 4 h + a (and + 8), columns 32 dt + 16 g + 4 b ..
        const int r0 = t * 32 + ks * 16 + 4 * h + a;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) {
          const int ch = 4 * dt + 2 * g + (b >> 1), in = (b & 1) * 8;
          typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
          const i16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_i16x4*)(vt + r0 * ROWB + ((ch ^ swz_v<DP>(r0)) << 4) + in));
          const i16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_i16x4*)(vt + (r0 + 8) * ROWB + ((ch ^ swz_v<DP>(r0 + 8)) << 4) + in));
          const uint2 w0 = __builtin_bit_cast(uint2, v0), w1 = __builtin_bit_cast(uint2, v1);
          const u32x4 vf = {w0.x, w0.y, w1.x, w1.y};
          o[dt] = mfma<BF>(vf, hi, o[dt]);
          o[dt] = mfma<BF>(vf, lo, o[dt]);
        }
      }
  }
};

// Copies of one tile: this wave's NI instructions of 64 / CPR rows each, from
// row `row0` of the tile at LDS address `lds`, whose row 0 is key `key0`;
// keys from `end` on, and keys of pages outside the pool, are zeros.
template <int DP, int NI, bool ISV>
struct TileCopy {
  static constexpr int CPR = DP / 8, RPI = 64 / CPR;
  uint32_t off[NI];  // contiguous tokens: byte offset from the tile's first token

  __device__ __forceinline__ static int chunk(int row, int lane, int D) {
    const int ch = (lane % CPR) ^ (ISV ? swz_v<DP>(row) : swz_k<DP>(row));
    return ch * 8 < D ? ch : 0;  // (columns past D: anything of the row; they meet zeros of q, or are not stored)
  }
  __device__ __forceinline__ void init(const KeySource& src, int row0, int lane, int D) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int row = row0 + i * RPI + lane / CPR;
      off[i] = static_cast<uint32_t>(row * static_cast<uint32_t>(src.row)) + chunk(row, lane, D) * 16;
    }
  }
  __device__ __forceinline__ void fast(const uint8_t* tile, int row0, uint32_t lds) const {
#pragma unroll
    for (int i = 0; i < NI; ++i) copy_to_lds(tile, off[i], lds + (row0 + i * RPI) * DP * 2);
  }
  __device__ __forceinline__ static void slow(const KeySource& src, const uint8_t* base, const int* pages, int first,
                                              int key0, int end, int row0, uint32_t lds, int lane, int D) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int row = row0 + i * RPI + lane / CPR, key = key0 + row, ch = chunk(row, lane, D);
      const uint8_t* p = reinterpret_cast<const uint8_t*>(g_zero_row);
      if (key < end) {
        if (pages) {
          const int pg = pages[(key >> src.shift) - first];
          if (pg >= 0) p = base + pg * src.page + (key & ((1 << src.shift) - 1)) * src.row;
        } else {
          p = base + key * src.row;
        }
      }
      copy_to_lds(p + ch * 16, lds + (row0 + i * RPI) * DP * 2);
    }
  }
};

// Page numbers of keys [k0, k1) to LDS, -1 for those outside the pool.
// Returns whether there is one (to every thread; includes a barrier).
__device__ __forceinline__ bool load_pages(const KeySource& src, int k0, int k1, int* pages) {
  bool bad = false;
  const int first = k0 >> src.shift, n = ((k1 - 1) >> src.shift) - first + 1;
  for (int i = threadIdx.x; i < n; i += 256) {
    const int pg = src.table[first + i];
    const bool in = pg >= 0 && pg < src.npages;
    pages[i] = in ? pg : -1;
    bad |= !in;
  }
  return __syncthreads_or(bad);
}

// Key j of subtile register i.
__device__ __forceinline__ int key_of(int i, int lane) { return 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3); }

template <bool BF, int DP>
struct Attn {
  typedef RowTile<BF, DP> Tile;
  static constexpr int CPR = DP / 8, RPI = 64 / CPR, ROWB = DP * 2;
  static constexpr int kWideKeys = DP == 256 ? 32 : 64;        // keys of a wide tile
  static constexpr int kTileBytes = kWideKeys * ROWB;          // its K or V
  static constexpr int kWaveBytes = 32 * ROWB;                 // narrow: a wave's K or V
  static constexpr int kLds = 4 * kTileBytes > 8 * kWaveBytes ? 4 * kTileBytes : 8 * kWaveBytes;

  // The unnormalized output of a lane's row to the workspace (wide).
  static __device__ __forceinline__ void store(const Tile& t, float* po, float2* pml, int D, int lane) {
    const float l = t.l + __shfl_xor(t.l, 32);
#pragma unroll
    for (int dt = 0; dt < Tile::DT; ++dt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = 32 * dt + 8 * i + 4 * (lane >> 5);
        if (d < D)
          *reinterpret_cast<float4*>(po + d) =
              make_float4(t.o[dt][4 * i], t.o[dt][4 * i + 1], t.o[dt][4 * i + 2], t.o[dt][4 * i + 3]);
      }
    if (lane < 32) *pml = make_float2(t.m, l);
  }

  // 128 rows (32 a wave) against keys [k0, k1) of the prefix; the four waves
  // share each tile, double-buffered: one barrier a tile, and a tile's copies
  // run while the one before it is multiplied.
  static __device__ __forceinline__ void wide(const AttnKernelArgs& g, const KeySource& src, int slot, int hk, int rt,
                                              int k0, int k1, uint8_t* smem, int* pages) {
    const qmv_attn_args& a = g.a;
    const int lane = __lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), D = a.head_dim;
    const int G = g.p.groups, M = static_cast<int>(a.rows) * G;
    const int m0 = rt * 128 + wave * 32, mi = min(m0 + (lane & 31), M - 1);
    const int row = mi / G, head = hk * G + mi % G;
    Tile t;
    t.init(static_cast<const uint16_t*>(a.q) + row * a.q_row + head * a.q_head, D, a.scale, lane);
    bool bad = false;
    if (src.table) bad = load_pages(src, k0, k1, pages);
    const int first = src.table ? k0 >> src.shift : 0;
    const int* pg = src.table ? pages : nullptr;
    constexpr int NI = kWideKeys / 4 / RPI;
    const int row0 = wave * (kWideKeys / 4);
    TileCopy<DP, NI, false> ck;
    TileCopy<DP, NI, true> cv;
    ck.init(src, row0, lane, D);
    cv.init(src, row0, lane, D);
    const bool plain = !src.table && src.row < (int64_t{1} << 25);
    const uint32_t lds = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_u8*)smem));
    auto copy = [&](int tile) {
      const int key0 = k0 + tile * kWideKeys;
      const uint32_t at = lds + (tile & 1) * 2 * kTileBytes;
      if (plain && key0 + kWideKeys <= k1) {
        ck.fast(src.k + key0 * src.row, row0, at);
        cv.fast(src.v + key0 * src.row, row0, at + kTileBytes);
      } else {
        ck.slow(src, src.k, pg, first, key0, k1, row0, at, lane, D);
        cv.slow(src, src.v, pg, first, key0, k1, row0, at + kTileBytes, lane, D);
      }
    };
    const int tiles = (k1 - k0 + kWideKeys - 1) / kWideKeys;
    constexpr int NT = kWideKeys / 32;
    copy(0);
#pragma unroll 1
    for (int tile = 0; tile < tiles; ++tile) {
      wait_copies<0>();
      lds_barrier();
      if (tile + 1 < tiles) copy(tile + 1);
      if (m0 >= M) continue;  // (whole waves: they only copy)
      const lds_u8* kt = (const lds_u8*)smem + (tile & 1) * 2 * kTileBytes;
      f32x16 s[NT];
      t.template scores<NT>(kt, lane, s);
      const int left = k1 - k0 - tile * kWideKeys;
      if (left < kWideKeys || bad) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int j = 32 * n + key_of(i, lane);
            bool seen = j < left;
            if (bad && seen) seen = pages[((k0 + tile * kWideKeys + j) >> src.shift) - first] >= 0;
            s[n][i] = seen ? s[n][i] : -INFINITY;
          }
      }
      t.template softmax<NT>(s);
      t.template values<NT>(kt + kTileBytes, lane, s);
    }
    if (m0 + (lane & 31) < M) {
      const size_t at = static_cast<size_t>(slot) * a.rows * a.heads + static_cast<size_t>(row) * a.heads + head;
      store(t, g.po + at * D, g.pml + at, D, lane);
    }
  }

  // 32 rows against keys [k0, k1) of the prefix or of a sequence's suffix:
  // each wave takes every fourth tile of 32 keys through its own LDS, with no
  // barrier; a tile's K and V are copied again as soon as the wave has read
  // them.  The waves' parts are joined at the end.
  // draft0: the suffix position of the sequence's first row (prefix: k1).
  static __device__ __forceinline__ void narrow(const AttnKernelArgs& g, const KeySource& src, int slot, int hk,
                                                int rbase, int nrows, int r0, int k0, int k1, int draft0,
                                                uint8_t* smem, int* pages) {
    const qmv_attn_args& a = g.a;
    const int lane = __lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), D = a.head_dim;
    const int G = g.p.groups, M = nrows * G;
    const int mi = min(r0 + (lane & 31), M - 1);
    const int row = rbase + mi / G, head = hk * G + mi % G;
    Tile t;
    t.init(static_cast<const uint16_t*>(a.q) + row * a.q_row + head * a.q_head, D, a.scale, lane);
    const uint64_t mask = a.tree_mask && draft0 < k1 ? a.tree_mask[row] : 0;
    bool bad = false;
    if (src.table) bad = load_pages(src, k0, k1, pages);
    const int first = src.table ? k0 >> src.shift : 0;
    const int* pg = src.table ? pages : nullptr;
    constexpr int NI = 32 / RPI;
    TileCopy<DP, NI, false> ck;
    TileCopy<DP, NI, true> cv;
    ck.init(src, 0, lane, D);
    cv.init(src, 0, lane, D);
    const bool plain = !src.table && src.row < (int64_t{1} << 25);
    lds_u8* kt = (lds_u8*)smem + wave * 2 * kWaveBytes;
    lds_u8* vt = kt + kWaveBytes;
    const uint32_t klds = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(kt)), vlds = klds + kWaveBytes;
    auto copy_k = [&](int tile) {
      const int key0 = k0 + tile * 32;
      if (plain && key0 + 32 <= k1) ck.fast(src.k + key0 * src.row, 0, klds);
      else ck.slow(src, src.k, pg, first, key0, k1, 0, klds, lane, D);
    };
    auto copy_v = [&](int tile) {
      const int key0 = k0 + tile * 32;
      if (plain && key0 + 32 <= k1) cv.fast(src.v + key0 * src.row, 0, vlds);
      else cv.slow(src, src.v, pg, first, key0, k1, 0, vlds, lane, D);
    };
    const int tiles = (k1 - k0 + 31) / 32;
    if (wave < tiles) {
      copy_k(wave);
      copy_v(wave);
    }
#pragma unroll 1
    for (int tile = wave; tile < tiles; tile += 4) {
      const int key0 = k0 + tile * 32;
      f32x16 s[1];
      wait_copies<NI>();
      t.template scores<1>(kt, lane, s);
      wait_lds();
      copy_k(tile + 4);  // (past the last tile: zeros that nobody reads)
      const bool drafts = key0 + 32 > draft0;
      if (drafts || key0 + 32 > k1 || bad) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = key0 + key_of(i, lane);
          bool seen = j < k1;
          const int at = j - draft0;
          if (at >= 0) seen = seen && (a.tree_mask ? at < 64 && ((mask >> (at & 63)) & 1) : at <= row - rbase);
          if (bad && seen) seen = pages[(j >> src.shift) - first] >= 0;
          s[0][i] = seen ? s[0][i] : -INFINITY;
        }
      }
      t.template softmax<1>(s);
      wait_copies<NI>();
      if (drafts) unseen_values(t, s[0], vt, lane, max(draft0 - key0, 0), D);
      t.template values<1>(vt, lane, s);
      wait_lds();
      copy_v(tile + 4);
    }
    wait_copies<0>();
    __syncthreads();

    // The waves' parts: [wave][row][DP] in the tiles' place, maxima and sums in `pages`.
    float* parts = reinterpret_cast<float*>(smem);
    float2* ml = reinterpret_cast<float2*>(pages);
    const float l = t.l + __shfl_xor(t.l, 32);
    {
      // rows are 16-byte chunks, permuted by the row against bank conflicts
      float4* p = reinterpret_cast<float4*>(parts + (wave * 32 + (lane & 31)) * DP);
#pragma unroll
      for (int dt = 0; dt < Tile::DT; ++dt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          p[(8 * dt + 2 * i + (lane >> 5)) ^ (lane & 7)] =
              make_float4(t.o[dt][4 * i], t.o[dt][4 * i + 1], t.o[dt][4 * i + 2], t.o[dt][4 * i + 3]);
      if (lane < 32) ml[wave * 32 + lane] = make_float2(t.m, l);
    }
    __syncthreads();
    constexpr int kQuads = DP / 4;
    for (int e = threadIdx.x; e < 32 * kQuads; e += 256) {
      const int r = e / kQuads, ch = e % kQuads, m = r0 + r;
      if (m >= M || ch * 4 >= D) continue;
      float2 w[4];
      float mx = kNone;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        w[k] = ml[k * 32 + r];
        mx = fmaxf(mx, w[k].x);
      }
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      float sl = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float f = __builtin_amdgcn_exp2f(w[k].x - mx);
        const float4 v = reinterpret_cast<const float4*>(parts + (k * 32 + r) * DP)[ch ^ (r & 7)];
        sum.x = fmaf(f, v.x, sum.x);
        sum.y = fmaf(f, v.y, sum.y);
        sum.z = fmaf(f, v.z, sum.z);
        sum.w = fmaf(f, v.w, sum.w);
        sl = fmaf(f, w[k].y, sl);
      }
      const size_t at = static_cast<size_t>(slot) * a.rows * a.heads +
                        static_cast<size_t>(rbase + m / G) * a.heads + hk * G + m % G;
      *reinterpret_cast<float4*>(g.po + at * D + ch * 4) = sum;
      if (ch == 0) g.pml[at] = make_float2(mx, sl);
    }
  }

  // Drafted keys are seen by some of the rows only, and 0 x infinity or NaN is
  // not 0: values of tile rows from `from` on that are not finite are added
  // here to the rows that see them, and zeroed for the product.
  static __device__ __forceinline__ void unseen_values(Tile& t, const f32x16& p, lds_u8* vt, int lane, int from,
                                                       int D) {
    const int r = lane & 31;
    constexpr uint32_t kExp = BF ? 0x7F80u : 0x7C00u;
    bool odd = false;
#pragma unroll 1
    for (int ch = lane >> 5; ch * 8 < D; ch += 2) {
      const u32x4 w = *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>(
          vt + r * ROWB + ((ch ^ swz_v<DP>(r)) << 4));
#pragma unroll
      for (int k = 0; k < 4; ++k)
        odd |= (w[k] & kExp) == kExp || ((w[k] >> 16) & kExp) == kExp;
    }
    const uint64_t all = __ballot(odd && r >= from);
    uint32_t rows = static_cast<uint32_t>(all | (all >> 32));
    while (rows) {
      const int kk = __builtin_ctz(rows);
      rows &= rows - 1;
      const int ri = ((kk >> 3) << 2) | (kk & 3);
      float pk = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) pk = i == ri ? p[i] : pk;
      const float other = __shfl_xor(pk, 32);
      pk = (lane >> 5) == ((kk >> 2) & 1) ? pk : other;
      const bool seen = !(pk == 0.f);
#pragma unroll
      for (int dt = 0; dt < Tile::DT; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int d = 32 * dt + key_of(i, lane);
          const uint32_t b = *reinterpret_cast<const __attribute__((address_space(3))) uint16_t*>(
              vt + kk * ROWB + (((d >> 3) ^ swz_v<DP>(kk)) << 4) + (d & 7) * 2);
          const float v = BF ? bf16_to_f32(b) : f16_to_f32(b);
          t.o[dt][i] = seen ? fmaf(pk, v, t.o[dt][i]) : t.o[dt][i];
        }
      order_memory();
      if (lane < CPR) {
        const u32x4 z = {0, 0, 0, 0};
        *reinterpret_cast<__attribute__((address_space(3))) u32x4*>(vt + kk * ROWB + lane * 16) = z;
      }
      order_memory();
    }
  }
};

template <bool BF, int DP>
__global__ void __launch_bounds__(256, DP == 256 ? 1 : 2) attn_parts_kernel(const AttnKernelArgs g) {
  typedef Attn<BF, DP> A;
  extern __shared__ __attribute__((aligned(16))) uint8_t attn_lds[];
  int* pages = reinterpret_cast<int*>(attn_lds + A::kLds);
  const qmv_attn_args& a = g.a;
  KeySource src;
  int shift = 31 - __builtin_clz(a.page_size > 0 ? a.page_size : 1);
  src.shift = shift;
  src.npages = static_cast<int>(a.num_pages);
  src.page = a.page_stride * 2;
  int id = blockIdx.x;
  const int before = static_cast<int>(g.p.prefix_wgs);
  if (id < before) {
    // workgroups of one key head and key range are a multiple of 8 apart where
    // there are a multiple of 8 such pairs: on one XCD, sharing its L2
    const int pairs = a.kv_heads * g.p.psplits;
    const int rt = id / pairs, pair = id % pairs;
    const int hk = pair % a.kv_heads, split = pair / a.kv_heads;
    const int k0 = split * g.p.pseg, k1 = min(k0 + g.p.pseg, static_cast<int>(a.prefix_len));
    src.table = a.prefix_pages;
    src.k = static_cast<const uint8_t*>(src.table ? a.k_pages : a.k_prefix) + hk * (src.table ? a.page_head : a.prefix_head) * 2;
    src.v = static_cast<const uint8_t*>(src.table ? a.v_pages : a.v_prefix) + hk * (src.table ? a.page_head : a.prefix_head) * 2;
    src.row = (src.table ? a.page_row : a.prefix_row) * 2;
    if (g.p.wide)
      A::wide(g, src, split, hk, rt, k0, k1, attn_lds, pages);
    else
      A::narrow(g, src, split, hk, 0, static_cast<int>(a.rows), rt * 32, k0, k1, k1, attn_lds, pages);
    return;
  }
  id -= before;
  const int hk = id % a.kv_heads;
  id /= a.kv_heads;
  const int rt = id % g.p.srow_tiles;
  id /= g.p.srow_tiles;
  const int split = id % g.p.ssplits, b = id / g.p.ssplits;
  const int rows = static_cast<int>(a.rows);
  const int start = a.row_start[b], end = a.row_start[b + 1];
  if (start < 0 || end > rows || start >= end) return;
  const int n = min(end - start, a.max_rows);
  if (rt * 32 >= n * g.p.groups) return;
  const int len = min(max(a.suffix_len[b], 0), static_cast<int>(a.max_suffix));
  const int k0 = split * g.p.sseg, k1 = min(k0 + g.p.sseg, len);
  if (k0 >= k1) return;
  src.table = a.block_table + b * a.table_stride;
  src.k = static_cast<const uint8_t*>(a.k_pages) + hk * a.page_head * 2;
  src.v = static_cast<const uint8_t*>(a.v_pages) + hk * a.page_head * 2;
  src.row = a.page_row * 2;
  A::narrow(g, src, g.p.psplits + split, hk, start, n, rt * 32, k0, k1, len - (end - start), attn_lds, pages);
}

// A (row, head)'s parts joined, in the order of their slots: one wave each.
template <bool BF, int VEC>
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnKernelArgs g) {
  const qmv_attn_args& a = g.a;
  const int lane = __lane_id(), D = a.head_dim;
  const int64_t e = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int64_t all = a.rows * a.heads;
  if (e >= all) return;
  const int row = static_cast<int>(e / a.heads), head = static_cast<int>(e % a.heads);
  // the row's sequence: the last that starts at or before it
  int seq = -1;
  for (int b0 = 0; b0 < a.nseq; b0 += 64) {
    const int b = b0 + lane;
    seq += __popcll(__ballot(b < a.nseq && a.row_start[min(b, a.nseq)] <= row));
  }
  int slots = g.p.psplits;
  bool past = false;
  if (seq >= 0) {
    const int start = a.row_start[seq], end = a.row_start[seq + 1];
    if (start >= 0 && row >= start && row < end && end <= a.rows) {
      past = row - start >= a.max_rows;
      const int len = a.max_suffix > 0 ? min(max(a.suffix_len[seq], 0), static_cast<int>(a.max_suffix)) : 0;
      if (!past && len > 0) slots += (len + g.p.sseg - 1) / g.p.sseg;
    }
  }
  float mx = kNone;
  for (int s = lane; s < slots; s += 64) mx = fmaxf(mx, g.pml[s * all + e].x);
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) mx = fmaxf(mx, __shfl_xor(mx, k));
  float acc[VEC] = {}, l = 0.f;
  const int d = lane * VEC;
  if (d < D) {
#pragma unroll 4
    for (int s = 0; s < slots; ++s) {
      const float2 ml = g.pml[s * all + e];
      const float f = __builtin_amdgcn_exp2f(ml.x - mx);
      const float* p = g.po + (s * all + e) * D + d;
      l = fmaf(f, ml.y, l);
#pragma unroll
      for (int k = 0; k < VEC; ++k) acc[k] = fmaf(f, p[k], acc[k]);
    }
    uint16_t* out = static_cast<uint16_t*>(a.out) + row * a.out_row + head * a.out_head + d;
    const float inv = past ? __builtin_nanf("") : l == 0.f ? 0.f : 1.f / l;
    uint32_t w[VEC / 2];
#pragma unroll
    for (int k = 0; k < VEC; k += 2) {
      const float x = l == 0.f && !past ? 0.f : acc[k] * inv, y = l == 0.f && !past ? 0.f : acc[k + 1] * inv;
      if (BF)
        w[k / 2] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(x)) |
                   (__builtin_bit_cast(uint16_t, static_cast<__bf16>(y)) << 16);
      else
        w[k / 2] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(x)) |
                   (__builtin_bit_cast(uint16_t, static_cast<_Float16>(y)) << 16);
    }
    if constexpr (VEC == 2)
      *reinterpret_cast<uint32_t*>(out) = w[0];
    else
      *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
  }
  if (a.lse && lane == 0)
    a.lse[e] = past ? __builtin_nanf("") : l == 0.f ? -INFINITY : (mx + __builtin_amdgcn_logf(l)) * kLn2;
}

static int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

static AttnPlan plan_attn(const qmv_attn_args& a) {
  constexpr int kSlots = 512;  // two workgroups a compute unit
  AttnPlan p = {};
  p.groups = a.heads / a.kv_heads;
  const int64_t M = a.rows * p.groups;
  p.wide = M > 64;
  p.row_tiles = ceil_div(M, p.wide ? 128 : 32);
  const int step = p.wide ? 256 : 128;  // fewest keys of a range
  if (a.prefix_len > 0) {
    const int64_t units = static_cast<int64_t>(p.row_tiles) * a.kv_heads;
    int64_t splits = std::min<int64_t>(ceil_div(a.prefix_len, step), std::max<int64_t>(1, kSlots / units));
    if (a.prefix_pages) splits = std::max<int64_t>(splits, ceil_div(a.prefix_len, kMaxPagedKeys));
    p.pseg = ceil_div(ceil_div(a.prefix_len, splits), 64) * 64;
    p.psplits = ceil_div(a.prefix_len, p.pseg);
    p.prefix_wgs = units * p.psplits;
  }
  if (a.max_suffix > 0) {
    p.srow_tiles = ceil_div(static_cast<int64_t>(std::min<int64_t>(a.max_rows, a.rows)) * p.groups, 32);
    const int64_t units = static_cast<int64_t>(a.nseq) * a.kv_heads * p.srow_tiles;
    int64_t splits = std::min<int64_t>(ceil_div(a.max_suffix, 128), std::max<int64_t>(1, kSlots / units));
    splits = std::max<int64_t>(splits, ceil_div(a.max_suffix, kMaxPagedKeys));
    p.sseg = ceil_div(ceil_div(a.max_suffix, splits), 128) * 128;
    p.ssplits = ceil_div(a.max_suffix, p.sseg);
    p.suffix_wgs = units * p.ssplits;
  }
  return p;
}

bool attn_fits(const qmv_attn_args& a) {
  const AttnPlan p = plan_attn(a);
  return p.prefix_wgs + p.suffix_wgs <= INT32_MAX;
}

static size_t ml_bytes(const qmv_attn_args& a, const AttnPlan& p) {
  return (static_cast<size_t>(p.psplits + p.ssplits) * a.rows * a.heads * sizeof(float2) + 255) / 256 * 256;
}

size_t attn_workspace(const qmv_attn_args& a) {
  const AttnPlan p = plan_attn(a);
  return ml_bytes(a, p) + static_cast<size_t>(p.psplits + p.ssplits) * a.rows * a.heads * a.head_dim * sizeof(float);
}

template <bool BF, int DP>
static hipError_t launch_parts(const AttnKernelArgs& g, hipStream_t s) {
  constexpr int lds = Attn<BF, DP>::kLds + kMaxPagedKeys * 4;
  const unsigned grid = static_cast<unsigned>(g.p.prefix_wgs + g.p.suffix_wgs);
  if (grid) hipLaunchKernelGGL((attn_parts_kernel<BF, DP>), dim3(grid), dim3(256), lds, s, g);
  return hipGetLastError();
}

template <bool BF>
static hipError_t attn_typed(const AttnKernelArgs& g, hipStream_t s) {
  const int D = g.a.head_dim;
  const hipError_t e = D <= 64    ? launch_parts<BF, 64>(g, s)
                       : D <= 128 ? launch_parts<BF, 128>(g, s)
                                  : launch_parts<BF, 256>(g, s);
  if (e != hipSuccess) return e;
  const dim3 grid(ceil_div(g.a.rows * g.a.heads, 4));
  if (D <= 128)
    hipLaunchKernelGGL((attn_join_kernel<BF, 2>), grid, dim3(256), 0, s, g);
  else
    hipLaunchKernelGGL((attn_join_kernel<BF, 4>), grid, dim3(256), 0, s, g);
  return hipGetLastError();
}

hipError_t attn(const qmv_attn_args& a, void* ws, hipStream_t s) {
  AttnKernelArgs g;
  g.a = a;
  g.p = plan_attn(a);
  g.pml = static_cast<float2*>(ws);
  g.po = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + ml_bytes(a, g.p));
  return a.dtype == QMV_BF16 ? attn_typed<true>(g, s) : attn_typed<false>(g, s);
}

}  // namespace qmv
