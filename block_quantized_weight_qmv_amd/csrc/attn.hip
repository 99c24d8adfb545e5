// Attention of a step's rows over a prefix that the whole batch shares and
// their own sequences' paged suffixes:
//   o = sum_j p_j v_j / sum_j p_j,  p_j = e^(scale q.k_j - m),  m = max_j scale q.k_j,
// over the prefix tokens and the suffix tokens that the row sees.
//
// One launch walks the keys, a second joins the parts.  The query heads that
// share a key head, of all rows of the step, stand side by side as rows of one
// matrix, so a prefix key is read once per 128 (wide) or 32 or 16 (narrow) of them
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
// Measured (kernel times are the fastest of 40 traced).  64 sequences of up to
// 8 rows on 32768 shared tokens and up to 1024 of their own (28 query and 4 key
// heads of 128, bf16), 137.6 GFLOP: 176 us a call, 780 TFLOP/s, where a large
// matrix product reaches 1340; 167 us and 16 us to join.  Counters: matrix
// pipes busy for 39 % of the time, 6.8 vector instructions to a matrix
// instruction.  32 sequences of up to 2111 own tokens (12 heads of 80, fp16,
// 150 MB): 43 us and 5.1 us; waves wait for 40 % of their time, most likely
// for copies, with two workgroups of 64 KB to a compute unit.  One row on 1000
// tokens: 5.8 us and 3 us, latencies in a row.
//
// K and V tiles go from memory to LDS without passing registers.  16-byte
// chunks of a tile's row are permuted by the row's number so that neither
// product's reads meet in a bank (swz); the copy fills LDS in order,
// so each lane asks for the chunk that belongs at its place.
#include <float.h>

#include <algorithm>
#include <type_traits>

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
// A row's exponentials are held as 2^kLift of its largest when the maximum is
// set, and the maximum is replaced only when one passes 2^kTop: until then the
// 32..128 outputs of a lane need no rescaling.  bf16 has fp32's exponents.  An
// fp16 number below 2^-14 is a multiple of 2^-24, so fp16's exponentials stand as
// high as its range allows: what weighs little beside the maximum -- many keys beside
// an attention sink -- is off by 2^-37 of the maximum's weight at most, where
// exponentials of 1 to 2^8 are off by 2^-25.  (The more frequent rescaling:
// 5 draft trees on 4099 tokens take 13.2 us instead of 12.6, 64 x 8 rows in fp16 on
// 32768 tokens 188 instead of 182.)
template <bool BF>
constexpr float kLift = BF ? 0.f : 12.f;
template <bool BF>
constexpr float kTop = BF ? 8.f : 15.f;
// Pages of one workgroup's keys: their numbers are held in LDS.
constexpr int kMaxPages = 2048;

// Where the keys of a workgroup come from.
struct KeySource {
  const uint8_t* k;       // key head's first element of token or page 0
  const uint8_t* v;
  const int32_t* table;   // NULL: contiguous tokens
  int64_t row;            // bytes from one token to the next (within a page)
  int64_t page;           // bytes from one page to the next
  int shift, npages;      // log2 of the page size
  int dim;                // D
};

// n / d for 0 <= n < 2^31, as a multiplication (Granlund and Montgomery,
// "Division by Invariant Integers using Multiplication", 1994).
struct FastDiv {
  uint32_t d, mul, shift;
};

static FastDiv fast_div(int64_t d) {
  FastDiv f{static_cast<uint32_t>(d), 0, 0};
  while ((int64_t{1} << f.shift) < d) ++f.shift;
  f.mul = static_cast<uint32_t>(((uint64_t{1} << 32) * ((uint64_t{1} << f.shift) - d)) / d + 1);
  return f;
}

__device__ __forceinline__ int quotient(int n, const FastDiv& f) {
  return static_cast<int>((__umulhi(static_cast<uint32_t>(n), f.mul) + static_cast<uint32_t>(n)) >> f.shift);
}
__device__ __forceinline__ int remainder_of(int n, int q, const FastDiv& f) { return n - q * static_cast<int>(f.d); }

struct AttnPlan {
  int groups;        // query heads per key head
  int each;          // a copy instruction's rows lie in one page, at 32-bit offsets (suffix, and prefix in pages)
  int suffix_first;  // the suffixes' workgroups run longer: they are launched first
  int wide;          // prefix: 128-row tiles of four waves (else narrow tiles, four waves along the keys)
  int rows;          // of a narrow tile: 16 or 32
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
  FastDiv groups, pairs, kv_heads, srow_tiles, nseq, heads;
  float* po;         // [slot][row * heads + head][D]
  float2* pml;       // [slot][row * heads + head]: maximum (log2), sum
};

// The permutation of a tile row's 16-byte chunks.  LDS serves 256 bytes a
// clock, 16 chunks of different banks: the first product reads 16 rows at one
// chunk, the second's transposing reads four rows x four chunks, and either
// set meets 16 different places (4.4 clocks a 16-byte read measured, against
// 7.9 where pairs of them meet).
template <int DP>
__device__ __forceinline__ int swz(int row) {
  return DP == 64 ? ((row >> 1) & 1) << 2 | ((row >> 2) & 3) : (row & 3) << 2 | ((row >> 2) & 3);
}

// 16 bytes of each lane of `lanes` from memory to LDS at `lds` + 16 x lane.  The
// s_nop covers an M0 or address written just before, which the compiler cannot see
// being used here.  LDS accesses are kept apart from copies by the waits and
// barriers between them (wait_copies, wait_lds, lds_barrier, which no memory
// access crosses); so that copies may run among reads of other tiles, they
// themselves are no such border.
__device__ __forceinline__ void copy_to_lds(const void* src, uint32_t lds, uint64_t lanes) {
  uint64_t all;
  __asm__ __volatile__(
      "s_mov_b32 m0, %2\n\ts_and_saveexec_b64 %0, %3\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, off\n\ts_mov_b64 exec, %0"
      : "=&s"(all)
      : "v"(src), "s"(lds), "s"(lanes)
      : "m0", "scc");
}
__device__ __forceinline__ void copy_to_lds(const void* base, uint32_t off, uint32_t lds, uint64_t lanes) {
  uint64_t all;
  __asm__ __volatile__(
      "s_mov_b32 m0, %3\n\ts_and_saveexec_b64 %0, %4\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %2\n\ts_mov_b64 exec, %0"
      : "=&s"(all)
      : "v"(off), "s"(base), "s"(lds), "s"(lanes)
      : "m0", "scc");
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

// x and y as two values of the type each, and what they sum to.  hi + lo holds
// 16 bits or more; in fp16, where lo ends at 2^-24, it is rounded there, and
// the sum takes what hi and lo hold.
template <bool BF>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t& hi, uint32_t& lo, float& sum) {
  if constexpr (BF) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    sum += x + y;
    const uint32_t bx = __float_as_uint(x), by = __float_as_uint(y);
    hi = __builtin_amdgcn_perm(by, bx, 0x07060302);
    const float rx = x - __uint_as_float(bx & 0xFFFF0000u), ry = y - __uint_as_float(by & 0xFFFF0000u);
    lo = __builtin_bit_cast(uint32_t, b2{static_cast<__bf16>(rx), static_cast<__bf16>(ry)});
  } else {
    const h2_t h = __builtin_bit_cast(h2_t, __builtin_amdgcn_cvt_pkrtz(x, y));
    const h2_t r = {static_cast<_Float16>(x - static_cast<float>(h.x)), static_cast<_Float16>(y - static_cast<float>(h.y))};
    const h2_t one = {static_cast<_Float16>(1.0f), static_cast<_Float16>(1.0f)};
    sum = __builtin_amdgcn_fdot2(r, one, __builtin_amdgcn_fdot2(h, one, sum, false), false);
    hi = __builtin_bit_cast(uint32_t, h);
    lo = __builtin_bit_cast(uint32_t, r);
  }
}

// x and y each rounded once to the type, and what the two sum to.
template <bool BF>
__device__ __forceinline__ uint32_t round_pair(float x, float y, float& sum) {
  if constexpr (BF) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    const b2 h = {static_cast<__bf16>(x), static_cast<__bf16>(y)};
    const b2 one = {static_cast<__bf16>(1.0f), static_cast<__bf16>(1.0f)};
    sum = __builtin_amdgcn_fdot2_f32_bf16(h, one, sum, false);
    return __builtin_bit_cast(uint32_t, h);
  } else {
    const h2_t h = {static_cast<_Float16>(x), static_cast<_Float16>(y)};
    const h2_t one = {static_cast<_Float16>(1.0f), static_cast<_Float16>(1.0f)};
    sum = __builtin_amdgcn_fdot2(h, one, sum, false);
    return __builtin_bit_cast(uint32_t, h);
  }
}

// A wave's 32 rows against a stream of key tiles.  SPLIT: the probabilities
// enter the second product as two values of the type (split_pair), so that an
// output is off by little but its own rounding.  Where many rows share the
// keys the products bound the kernel, and each probability is rounded once:
// an output's error grows by the square root of 2 at most (independent
// roundings of weights and of the output; in bf16 2.3e-3 of the outputs'
// norm, where 1.7e-3 is what fp32 arithmetic rounded at the end leaves), and 64 sequences of up to 8 rows on 32768 tokens
// took 195 us where the split took 227.  The sum takes the rounded
// probabilities too, so that they stay a mean's weights.
template <bool BF, int DP, bool SPLIT>
struct RowTile {
  static constexpr int KS = DP / 16, DT = DP / 32, CPR = DP / 8, ROWB = DP * 2;
  u32x4 q[KS];
  f32x16 o[DT];
  float m, l;
  float c;                    // scale log2 e
  uint32_t koff[KS], voff[DT][2];  // this lane's place in a tile's K for step ks, in V for columns dt

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
    // K: key lane & 31, chunk 2 ks + lane / 32
    const int r = lane & 31, h = lane >> 5;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) koff[ks] = r * ROWB + (((2 * ks + h) ^ swz<DP>(r)) << 4);
    // V, lane (h, g, a, b): key 4 h + a (and + 8), columns 32 dt + 16 g + 4 b ..
    const int g = (lane >> 4) & 1, a = (lane >> 2) & 3, b = lane & 3, k = 4 * h + a;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        voff[dt][i] = (k + 8 * i) * ROWB + (((4 * dt + 2 * g + (b >> 1)) ^ swz<DP>(k + 8 * i)) << 4) + (b & 1) * 8;
  }

  // Waits for q here, before the loop over the keys: the compiler would wait
  // inside it, for every load, the next tile's copies among them.
  __device__ __forceinline__ void arrived() {
#pragma unroll
    for (int s = 0; s < KS; ++s) __asm__ __volatile__("" : "+v"(q[s]));
  }

  // Scores of NT x 32 keys.  Reads of K lead by four fragments; between(n) is
  // called before matrix instruction n.
  template <int NT, class F>
  __device__ __forceinline__ void scores(const lds_u8* kt, f32x16* s, F&& between) {
    constexpr int kSteps = NT * KS, kLead = kSteps < 4 ? kSteps : 4;
    typedef const __attribute__((address_space(3))) u32x4 lds_u32x4;
    auto frag = [&](int n) { return *reinterpret_cast<lds_u32x4*>(kt + (n % NT) * 32 * ROWB + koff[n / NT]); };
    u32x4 kf[kSteps];
#pragma unroll
    for (int n = 0; n < kLead; ++n) kf[n] = frag(n);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[t][i] = 0.f;
#pragma unroll
    for (int n = 0; n < kSteps; ++n) {
      if (n + kLead < kSteps) kf[n + kLead] = frag(n + kLead);
      between(n);
      s[n % NT] = mfma<BF>(kf[n], q[n / NT], s[n % NT]);
    }
  }
  template <int NT>
  __device__ __forceinline__ void scores(const lds_u8* kt, f32x16* s) {
    scores<NT>(kt, s, [](int) {});
  }

  // Whether a score passes the maximum by enough to replace it; the largest of the lane's.
  template <int NT>
  __device__ __forceinline__ bool moves(const f32x16* s, float& mx) const {
    mx = s[0][0];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[t][i]);
    return __any(fmaf(mx, c, -m) > kTop<BF>);
  }
  __device__ __forceinline__ void move(float mx) {
    const float both = fmaxf(mx, __shfl_xor(mx, 32));
    const float mn = fmaxf(m, both * c - kLift<BF>);
    const float f = __builtin_amdgcn_exp2f(m - mn);
    m = mn;
    l *= f;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[t][i] *= f;
  }

  // NT x 32 keys' unnormalized probabilities as the second product takes them.
  template <int NT>
  struct Probs {
    u32x4 hi[2 * NT], lo[SPLIT ? 2 * NT : 1];
  };

  // Registers 2 n and 2 n + 1 of the scores, exponentiated, summed and split.
  template <int NT>
  __device__ __forceinline__ void exp_pair(f32x16* s, int n, Probs<NT>& p) {
    const int t = n >> 3, i = 2 * (n & 7);
    const float x = __builtin_amdgcn_exp2f(fmaf(s[t][i], c, -m)), y = __builtin_amdgcn_exp2f(fmaf(s[t][i + 1], c, -m));
    s[t][i] = x;
    s[t][i + 1] = y;
    if constexpr (SPLIT) {
      uint32_t hi, lo;
      split_pair<BF>(x, y, hi, lo, l);
      p.hi[n >> 2][n & 3] = hi;
      p.lo[n >> 2][n & 3] = lo;
    } else {
      p.hi[n >> 2][n & 3] = round_pair<BF>(x, y, l);
    }
  }

  // V^T of 16 keys (step ks of the tile) and 32 columns (dt).
  __device__ __forceinline__ u32x4 value_frag(const lds_u8* vt, int ks, int dt) const {
    typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
    const lds_u8* p = vt + ks * 16 * ROWB;
    const uint2 w0 = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + voff[dt][0])));
    const uint2 w1 = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + voff[dt][1])));
    return u32x4{w0.x, w0.y, w1.x, w1.y};
  }

  // o += V^T P^T over NT x 32 keys.
  template <int NT>
  __device__ __forceinline__ void values(const lds_u8* vt, const Probs<NT>& p) {
#pragma unroll
    for (int ks = 0; ks < 2 * NT; ++ks)
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) {
        const u32x4 vf = value_frag(vt, ks, dt);
        o[dt] = mfma<BF>(vf, p.hi[ks], o[dt]);
        if constexpr (SPLIT) o[dt] = mfma<BF>(vf, p.lo[ks], o[dt]);
      }
  }

  // The same for one tile, p, among the exponentials of the next, s to next:
  // a matrix instruction takes as long as the half dozen vector instructions
  // of a pair of scores, and the two kinds run side by side.  Reads of V lead
  // by four fragments.
  template <int NT, class F>
  __device__ __forceinline__ void values_and_exps(const lds_u8* vt, const Probs<NT>& p, f32x16* s, Probs<NT>& next,
                                                  F&& between) {
    static_assert(!SPLIT, "");
    constexpr int kSteps = 2 * NT * DT, kPairs = 8 * NT, kLead = kSteps < 4 ? kSteps : 4;
    u32x4 vf[kSteps];
#pragma unroll
    for (int n = 0; n < kLead; ++n) vf[n] = value_frag(vt, n / DT, n % DT);
    __builtin_amdgcn_sched_group_barrier(0x100, 2 * kLead, 0);  // LDS reads
#pragma unroll
    for (int n = 0; n < kSteps; ++n) {
      if (n + kLead < kSteps) {
        vf[n + kLead] = value_frag(vt, (n + kLead) / DT, (n + kLead) % DT);
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
      }
      between(n);
      o[n % DT] = mfma<BF>(vf[n], p.hi[n / DT], o[n % DT]);
#pragma unroll
      for (int k = n * kPairs / kSteps; k < (n + 1) * kPairs / kSteps; ++k) exp_pair<NT>(s, k, next);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // matrix
      __builtin_amdgcn_sched_group_barrier(0x002, 6 * kPairs / kSteps, 0);  // vector
    }
  }
};

// Key j of subtile register i.
__device__ __forceinline__ int key_of(int i, int lane) { return 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3); }

// Elements of V's tile row kk in LDS.
template <bool BF, int DP>
__device__ __forceinline__ float value_at(const lds_u8* vt, int kk, int d) {
  const uint32_t b = *reinterpret_cast<const __attribute__((address_space(3))) uint16_t*>(
      vt + kk * DP * 2 + (((d >> 3) ^ swz<DP>(kk)) << 4) + (d & 7) * 2);
  return BF ? bf16_to_f32(b) : f16_to_f32(b);
}

// The narrow workgroups' row tiles, a tile of 32 keys at a time: 32 rows ...
template <bool BF, int DP>
struct Narrow32 : RowTile<BF, DP, true> {
  typedef RowTile<BF, DP, true> Base;
  static constexpr int kRows = 32;
  struct Keys {
    f32x16 s[1];
  };
  typedef typename Base::template Probs<1> P;

  __device__ __forceinline__ void keys(const lds_u8* kt, Keys& k) { this->template scores<1>(kt, k.s); }
  // seen: bit j for key j
  static __device__ __forceinline__ void hide(Keys& k, uint32_t seen, int lane) {
    seen >>= 4 * (lane >> 5);
#pragma unroll
    for (int i = 0; i < 16; ++i) k.s[0][i] = (seen >> (8 * (i >> 2) + (i & 3))) & 1 ? k.s[0][i] : -INFINITY;
  }
  __device__ __forceinline__ void exps(Keys& k, P& p) {
    float mx;
    if (this->template moves<1>(k.s, mx)) this->move(mx);
#pragma unroll
    for (int n = 0; n < 8; ++n) this->template exp_pair<1>(k.s, n, p);
  }
  __device__ __forceinline__ void product(const lds_u8* vt, const P& p) { this->template values<1>(vt, p); }
  // The lane's row's probability of key kk.
  static __device__ __forceinline__ float prob(const Keys& k, int kk, int lane) {
    const int ri = ((kk >> 3) << 2) | (kk & 3);
    float pk = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) pk = i == ri ? k.s[0][i] : pk;
    const float other = __shfl_xor(pk, 32);
    return (lane >> 5) == ((kk >> 2) & 1) ? pk : other;
  }
  __device__ __forceinline__ void add_value(const lds_u8* vt, int kk, float pk, int lane) {
#pragma unroll
    for (int dt = 0; dt < Base::DT; ++dt)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        this->o[dt][i] = fmaf(pk, value_at<BF, DP>(vt, kk, 32 * dt + key_of(i, lane)), this->o[dt][i]);
  }
  __device__ __forceinline__ float total() const { return this->l + __shfl_xor(this->l, 32); }
  // The outputs as quads of columns.
  template <class F>
  __device__ __forceinline__ void each_quad(int lane, F&& f) const {
#pragma unroll
    for (int dt = 0; dt < Base::DT; ++dt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        f(8 * dt + 2 * i + (lane >> 5), make_float4(this->o[dt][4 * i], this->o[dt][4 * i + 1], this->o[dt][4 * i + 2],
                                                    this->o[dt][4 * i + 3]));
  }
};

// ... or 16, on 16x16x32 instructions, where a sequence has no more (one token
// of a group of up to 16 heads): half the matrix work, exponentials and
// outputs of a lane.  A lane (q, n) of the products holds row n and, in the
// first, keys 16 t + 4 q + r; one second product then spans the 32 keys, its
// k index 8 q + j over keys 4 q + j and 16 + 4 q + j - 4.
template <bool BF, int DP>
struct Narrow16 {
  typedef float f32x4 __attribute__((ext_vector_type(4)));
  static constexpr int kRows = 16, KS = DP / 32, DT = DP / 16, ROWB = DP * 2;
  struct Keys {
    f32x4 s[2];
  };
  struct P {
    u32x4 hi, lo;
  };
  u32x4 q[KS];
  f32x4 o[DT];
  float m, l, c;
  uint32_t koff[KS], voff[DT][2];

  static __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (BF)
      return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
      return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  __device__ __forceinline__ void init(const uint16_t* qp, int D, float scale, int lane) {
    const int n = lane & 15, g = lane >> 4, a = (lane >> 2) & 3, b = lane & 3;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int d = ks * 32 + 8 * g;
      const u32x4 z = {0, 0, 0, 0};
      q[ks] = d < D ? *reinterpret_cast<const u32x4*>(qp + d) : z;
      koff[ks] = n * ROWB + (((4 * ks + g) ^ swz<DP>(n)) << 4);
    }
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) {
      o[dt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = 4 * g + a + 16 * i;
        voff[dt][i] = k * ROWB + (((2 * dt + (b >> 1)) ^ swz<DP>(k)) << 4) + (b & 1) * 8;
      }
    }
    m = kNone;
    l = 0.f;
    c = scale * kLog2e;
  }
  __device__ __forceinline__ void arrived() {
#pragma unroll
    for (int s = 0; s < KS; ++s) __asm__ __volatile__("" : "+v"(q[s]));
  }
  __device__ __forceinline__ void keys(const lds_u8* kt, Keys& k) {
    typedef const __attribute__((address_space(3))) u32x4 lds_u32x4;
    u32x4 kf[2 * KS];
#pragma unroll
    for (int n = 0; n < 2 * KS; ++n) kf[n] = *reinterpret_cast<lds_u32x4*>(kt + (n & 1) * 16 * ROWB + koff[n >> 1]);
    k.s[0] = k.s[1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int n = 0; n < 2 * KS; ++n) k.s[n & 1] = mma(kf[n], q[n >> 1], k.s[n & 1]);
  }
  static __device__ __forceinline__ void hide(Keys& k, uint32_t seen, int lane) {
    seen >>= 4 * (lane >> 4);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) k.s[t][r] = (seen >> (16 * t + r)) & 1 ? k.s[t][r] : -INFINITY;
  }
  __device__ __forceinline__ void exps(Keys& k, P& p) {
    float mx = k.s[0][0];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) mx = fmaxf(mx, k.s[t][r]);
    if (__any(fmaf(mx, c, -m) > kTop<BF>)) {
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      const float mn = fmaxf(m, mx * c - kLift<BF>), f = __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) o[dt] *= f;
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int r = 0; r < 4; ++r) k.s[t][r] = __builtin_amdgcn_exp2f(fmaf(k.s[t][r], c, -m));
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t hi, lo;
        split_pair<BF>(k.s[t][2 * r], k.s[t][2 * r + 1], hi, lo, l);
        p.hi[2 * t + r] = hi;
        p.lo[2 * t + r] = lo;
      }
    }
  }
  __device__ __forceinline__ void product(const lds_u8* vt, const P& p) {
    typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) {
      const uint2 w0 = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(vt + voff[dt][0])));
      const uint2 w1 = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(vt + voff[dt][1])));
      const u32x4 vf = {w0.x, w0.y, w1.x, w1.y};
      o[dt] = mma(vf, p.hi, o[dt]);
      o[dt] = mma(vf, p.lo, o[dt]);
    }
  }
  static __device__ __forceinline__ float prob(const Keys& k, int kk, int lane) {
    float pk = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) pk = i == ((kk >> 4) << 2 | (kk & 3)) ? k.s[i >> 2][i & 3] : pk;
    return __shfl(pk, (kk >> 2 & 3) * 16 + (lane & 15));
  }
  __device__ __forceinline__ void add_value(const lds_u8* vt, int kk, float pk, int lane) {
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int r = 0; r < 4; ++r) o[dt][r] = fmaf(pk, value_at<BF, DP>(vt, kk, 16 * dt + 4 * (lane >> 4) + r), o[dt][r]);
  }
  __device__ __forceinline__ float total() const {
    const float s = l + __shfl_xor(l, 16);
    return s + __shfl_xor(s, 32);
  }
  template <class F>
  __device__ __forceinline__ void each_quad(int lane, F&& f) const {
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) f(4 * dt + (lane >> 4), make_float4(o[dt][0], o[dt][1], o[dt][2], o[dt][3]));
  }
};

// Copies of this wave's NI instructions of a tile, 64 / CPR rows each, from
// row `row0` of the tile on; K and V lie alike, so one set of offsets serves
// both.
template <int DP, int NI>
struct TileCopy {
  static constexpr int CPR = DP / 8, RPI = 64 / CPR;
  static constexpr int NV = 16 / RPI;  // instructions until the permutation repeats
  static constexpr int NM = NV < NI ? NV : NI;
  uint32_t off[NV];    // this lane's bytes from the instruction's first row
  uint64_t lanes[NM];  // those whose chunk lies before column D

  __device__ __forceinline__ static int chunk(int row, int lane) { return (lane % CPR) ^ swz<DP>(row); }
  __device__ __forceinline__ void init(const KeySource& src, int row0, int lane, int D) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = chunk(row0 + i * RPI + lane / CPR, lane);
      off[i] = static_cast<uint32_t>(lane / CPR * static_cast<uint32_t>(src.row)) + ch * 16;
      if (i < NM) lanes[i] = __ballot(ch * 8 < D);
    }
  }
  // The columns from D on, which no copy fills, in this wave's rows of a tile
  // whose row row0 is at `at`: zeros, which the zeros of q meet.
  __device__ __forceinline__ static void clear_past(lds_u8* at, int row0, int lane, int D) {
    constexpr int kRows = NI * RPI;
    const u32x4 z = {0, 0, 0, 0};
    const int r = lane % kRows;
    for (int ch = D / 8 + lane / kRows; ch < CPR; ch += 64 / kRows)
      *reinterpret_cast<__attribute__((address_space(3))) u32x4*>(at + r * DP * 2 + (ch ^ swz<DP>(row0 + r)) * 16) = z;
  }
  // Lane r: where tile row row0 + r begins; an instruction takes its first row's.
  __device__ __forceinline__ static uint64_t starts(const KeySource& src, const uint8_t* base, const int* pages, int first,
                                                    int key0, int end, int row0, int lane) {
    const int mine = min(key0 + row0 + lane, end - 1);
    int64_t at = mine * src.row;
    if (pages)
      at = max(pages[(mine >> src.shift) - first], 0) * src.page + (mine & ((1 << src.shift) - 1)) * src.row;
    return reinterpret_cast<uint64_t>(base) + static_cast<uint64_t>(at);
  }
  __device__ __forceinline__ static const void* start(uint64_t from, int i) {
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(from), i * RPI);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(from >> 32), i * RPI);
    return reinterpret_cast<const void*>(static_cast<uint64_t>(hi) << 32 | lo);
  }
  // The instructions' offsets for the tile at key0, whose rows from `end` on repeat the last key before it.
  __device__ __forceinline__ void offsets(const KeySource& src, int key0, int end, int row0, int lane, uint32_t* o) const {
#pragma unroll
    for (int i = 0; i < NI; ++i) o[i] = off[i % NV];
    if (key0 + row0 + NI * RPI > end) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int rows = lane / CPR, have = max(end - 1 - (key0 + row0 + i * RPI), 0);
        o[i] -= static_cast<uint32_t>(rows - min(rows, have)) * static_cast<uint32_t>(src.row);
      }
    }
  }
  // Instruction i of a tile whose row row0 is at `lds`.
  __device__ __forceinline__ void one(uint64_t from, uint32_t o, int i, uint32_t lds) const {
    copy_to_lds(start(from, i), o, lds + i * RPI * DP * 2, lanes[i % NM]);
  }

  // Key key0 is the tile's row 0.  Rows past the last key before `end` repeat
  // it, and keys of pages outside the pool are page 0's: what they hold is not
  // used.  each: every instruction's rows lie in one page of the pool (or
  // tokens are contiguous) and `off` holds.
  __device__ __forceinline__ void copy(const KeySource& src, const uint8_t* base, const int* pages, int first, bool each,
                                       int key0, int end, int row0, uint32_t lds, int lane) const {
    const int in_page = (1 << src.shift) - 1;
    if (each) {
      const uint64_t from = starts(src, base, pages, first, key0, end, row0, lane);
      uint32_t o[NI];
      offsets(src, key0, end, row0, lane, o);
#pragma unroll
      for (int i = 0; i < NI; ++i) one(from, o[i], i, lds + row0 * DP * 2);
      return;
    }
#pragma unroll 1
    for (int i = 0; i < NI; ++i) {
      const int row = row0 + i * RPI + lane / CPR, key = min(key0 + row, end - 1);
      const int64_t page = pages ? max(pages[(key >> src.shift) - first], 0) : 0, in = pages ? key & in_page : key;
      const int64_t at = page * src.page + in * src.row;
      const int ch = chunk(row, lane);
      copy_to_lds(base + at + ch * 16, lds + (row0 + i * RPI) * DP * 2, __ballot(ch * 8 < src.dim));
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

template <bool BF, int DP, class Tile>
struct Attn {
  typedef RowTile<BF, DP, false> WideTile;
  static constexpr int CPR = DP / 8, RPI = 64 / CPR, ROWB = DP * 2;
  static constexpr int kWideKeys = DP == 256 ? 32 : 64;        // keys of a wide tile
  static constexpr int kTileBytes = kWideKeys * ROWB;          // its K or V
  static constexpr int kWaveBytes = 32 * ROWB;                 // narrow: a wave's K or V
  static constexpr int kLds = 4 * kTileBytes > 8 * kWaveBytes ? 4 * kTileBytes : 8 * kWaveBytes;

  static __device__ __forceinline__ void zero_chunk(lds_u8* at) {
    const u32x4 z = {0, 0, 0, 0};
    *reinterpret_cast<__attribute__((address_space(3))) u32x4*>(at) = z;
  }

  // The unnormalized output of a lane's row to the workspace (wide).
  static __device__ __forceinline__ void store(const WideTile& t, float* po, float2* pml, int D, int lane) {
    const float l = t.l + __shfl_xor(t.l, 32);
#pragma unroll
    for (int dt = 0; dt < WideTile::DT; ++dt)
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
  // share each tile, K and V double-buffered, with one barrier a tile.
  static __device__ __forceinline__ void wide(const AttnKernelArgs& g, const KeySource& src, int slot, int hk, int rt,
                                              int k0, int k1, uint8_t* smem, int* pages) {
    const qmv_attn_args& a = g.a;
    const int lane = __lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), D = a.head_dim;
    const int G = g.p.groups, M = static_cast<int>(a.rows) * G;
    const int m0 = rt * 128 + wave * 32, mi = min(m0 + (lane & 31), M - 1);
    const int row = quotient(mi, g.groups), head = hk * G + remainder_of(mi, row, g.groups);
    bool bad = false;
    if (src.table) bad = load_pages(src, k0, k1, pages);
    const int first = src.table ? k0 >> src.shift : 0;
    const int* pg = src.table ? pages : nullptr;
    constexpr int NI = kWideKeys / 4 / RPI, NT = kWideKeys / 32;
    const int row0 = wave * (kWideKeys / 4);
    TileCopy<DP, NI> cp;
    cp.init(src, row0, lane, D);
    const uint32_t lds = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_u8*)smem));
    const int tiles = src.table && src.npages == 0 ? 0 : (k1 - k0 + kWideKeys - 1) / kWideKeys;
    // K of tile i in buffer i & 1, V in the two after them
    auto copy_k = [&](int tile) {
      cp.copy(src, src.k, pg, first, true, k0 + tile * kWideKeys, k1, row0, lds + (tile & 1) * kTileBytes, lane);
    };
    auto copy_v = [&](int tile) {
      cp.copy(src, src.v, pg, first, true, k0 + tile * kWideKeys, k1, row0, lds + (2 + (tile & 1)) * kTileBytes, lane);
    };
    auto partial = [&](int tile) { return bad || k1 - k0 - tile * kWideKeys < kWideKeys; };
    auto hide = [&](int tile, f32x16* s) {
      if (!partial(tile)) return;
      // bit j: key j of the tile is seen
      const int left = k1 - k0 - tile * kWideKeys;
      uint64_t seen = left >= 64 ? ~uint64_t{0} : (uint64_t{1} << left) - 1;
      if (bad) {
        const int key = min(k0 + tile * kWideKeys + lane, k1 - 1);
        seen &= ~__ballot(pages[(key >> src.shift) - first] < 0);
      }
      seen >>= 4 * (lane >> 5);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          s[n][i] = (static_cast<uint32_t>(seen >> (32 * n)) >> (8 * (i >> 2) + (i & 3))) & 1 ? s[n][i] : -INFINITY;
    };
    // (values of keys that are not there: 0 x infinity or NaN is not 0)
    auto clear = [&](int tile) {
      if (!partial(tile)) return;
      const int left = k1 - k0 - tile * kWideKeys;
      for (int r = threadIdx.x / CPR; r < kWideKeys; r += 256 / CPR)
        if (r >= left || (bad && pages[((k0 + tile * kWideKeys + r) >> src.shift) - first] < 0))
          zero_chunk((lds_u8*)smem + (2 + (tile & 1)) * kTileBytes + r * ROWB + threadIdx.x % CPR * 16);
      lds_barrier();
    };
    WideTile t;
    typename WideTile::template Probs<NT> p;
    f32x16 s[NT];
    float mx;
    const lds_u8* lk = (const lds_u8*)smem;
    if (tiles) {
      copy_k(0);
      copy_v(0);
      if (tiles > 1) copy_k(1);
    }
    if (D < DP)
      for (int i = 0; i < 4; ++i) cp.clear_past((lds_u8*)smem + i * kTileBytes + row0 * ROWB, row0, lane, D);
    t.init(static_cast<const uint16_t*>(a.q) + row * a.q_row + head * a.q_head, D, a.scale, lane);
    t.arrived();
    wait_copies<0>();
    lds_barrier();
    if (tiles) {
      t.template scores<NT>(lk, s);
      hide(0, s);
      if (t.template moves<NT>(s, mx)) t.move(mx);
#pragma unroll
      for (int n = 0; n < 8 * NT; ++n) t.template exp_pair<NT>(s, n, p);
    }
    // Tile i's second product runs beside tile i + 1's exponentials; the copies
    // of V one tile and of K two tiles ahead are issued among tile i + 1's
    // first product (in a row, they wait for each other).  Even and odd tiles
    // are written out: every LDS address is then a lane's constant and an
    // immediate.
    typename WideTile::template Probs<NT> q;
    auto step = [&](auto odd, int tile, auto& now, auto& next) __attribute__((always_inline)) {
      constexpr int kOdd = decltype(odd)::value;
      const lds_u8* kt = lk + (1 - kOdd) * kTileBytes;
      const lds_u8* vt = lk + (2 + kOdd) * kTileBytes;
      wait_copies<0>();
      lds_barrier();
      // (past the last tile the copies repeat its last key, into a buffer that nobody reads)
      const int key0 = k0 + (tile + 1) * kWideKeys;
      const uint64_t fv = cp.starts(src, src.v, pg, first, key0, k1, row0, lane);
      const uint64_t fk = cp.starts(src, src.k, pg, first, key0 + kWideKeys, k1, row0, lane);
      uint32_t ov[NI], ok[NI];
      cp.offsets(src, key0, k1, row0, lane, ov);
      cp.offsets(src, key0 + kWideKeys, k1, row0, lane, ok);
      const uint32_t at = lds + row0 * ROWB;
      clear(tile);
      constexpr int kEveryK = NT * WideTile::KS / NI, kEveryV = 2 * NT * WideTile::DT / NI;
      t.template scores<NT>(kt, s, [&](int n) {
        if (n % kEveryK == 0) cp.one(fv, ov[n / kEveryK], n / kEveryK, at + (3 - kOdd) * kTileBytes);
      });
      hide(tile + 1, s);
      if (t.template moves<NT>(s, mx)) {
        t.template values<NT>(vt, now);  // (what it was made with the old maximum)
        t.move(mx);
#pragma unroll
        for (int k = 0; k < 2 * NT; ++k) now.hi[k] = u32x4{0, 0, 0, 0};
      }
      t.template values_and_exps<NT>(vt, now, s, next, [&](int n) {
        if (n % kEveryV == 0) cp.one(fk, ok[n / kEveryV], n / kEveryV, at + kOdd * kTileBytes);
      });
    };
#pragma unroll 1
    for (int tile = 0; tile + 1 < tiles; tile += 2) {
      step(std::integral_constant<int, 0>{}, tile, p, q);
      if (tile + 2 >= tiles) {
        p = q;
        break;
      }
      step(std::integral_constant<int, 1>{}, tile + 1, q, p);
    }
    if (tiles) {
      wait_copies<0>();
      lds_barrier();
      clear(tiles - 1);
      t.template values<NT>(lk + (2 + ((tiles - 1) & 1)) * kTileBytes, p);
    }
    if (m0 + (lane & 31) < M) {
      const size_t at = static_cast<size_t>(slot) * a.rows * a.heads + static_cast<size_t>(row) * a.heads + head;
      store(t, g.po + at * D, g.pml + at, D, lane);
    }
  }

  // A row tile against keys [k0, k1) of the prefix or of a sequence's suffix:
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
    const int mi = min(r0 + lane % Tile::kRows, M - 1), ri = quotient(mi, g.groups);
    const int row = rbase + ri, head = hk * G + remainder_of(mi, ri, g.groups);
    bool bad = false;
    if (src.table) bad = load_pages(src, k0, k1, pages);
    const int first = src.table ? k0 >> src.shift : 0;
    const int* pg = src.table ? pages : nullptr;
    constexpr int NI = 32 / RPI;
    TileCopy<DP, NI> cp;
    cp.init(src, 0, lane, D);
    const bool each = src.table ? g.p.each : src.row < (int64_t{1} << 28);
    lds_u8* kt = (lds_u8*)smem + wave * 2 * kWaveBytes;
    lds_u8* vt = kt + kWaveBytes;
    const uint32_t klds = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(kt)), vlds = klds + kWaveBytes;
    const int tiles = src.table && src.npages == 0 ? 0 : (k1 - k0 + 31) / 32;
    if (wave < tiles) {
      cp.copy(src, src.k, pg, first, each, k0 + wave * 32, k1, 0, klds, lane);
      cp.copy(src, src.v, pg, first, each, k0 + wave * 32, k1, 0, vlds, lane);
      if (D < DP) {
        cp.clear_past(kt, 0, lane, D);
        cp.clear_past(vt, 0, lane, D);
      }
    }
    Tile t;
    t.init(static_cast<const uint16_t*>(a.q) + row * a.q_row + head * a.q_head, D, a.scale, lane);
    uint64_t mask = a.tree_mask && draft0 < k1 ? a.tree_mask[row] : 0;
    t.arrived();
    __asm__ __volatile__("" : "+v"(mask));
#pragma unroll 1
    for (int tile = wave; tile < tiles; tile += 4) {
      const int key0 = k0 + tile * 32;
      const bool more = tile + 4 < tiles;
      typename Tile::Keys s;
      wait_copies<NI>();  // outstanding: this tile's K, its V
      t.keys(kt, s);
      wait_lds();
      if (more) cp.copy(src, src.k, pg, first, each, key0 + 128, k1, 0, klds, lane);
      const bool partly = key0 + 32 > min(draft0, k1) || bad;  // some rows do not see some of the keys
      if (partly) {
        // bit j: the lane's row sees key key0 + j
        const int left = k1 - key0, at = draft0 - key0;
        uint32_t seen = left >= 32 ? ~0u : (1u << left) - 1;
        if (a.tree_mask)
          seen &= at >= 32 ? ~0u : at >= 0 ? ((1u << at) - 1) | static_cast<uint32_t>(mask << at)
                                           : at > -64 ? static_cast<uint32_t>(mask >> -at) : 0u;
        else
          seen &= at + ri >= 31 ? ~0u : at + ri >= 0 ? (2u << (at + ri)) - 1 : 0u;
        if (bad) {
          const int key = min(key0 + (lane & 31), k1 - 1);
          seen &= ~static_cast<uint32_t>(__ballot(pages[(key >> src.shift) - first] < 0));
        }
        t.hide(s, seen, lane);
      }
      typename Tile::P p;
      t.exps(s, p);
      if (more) wait_copies<NI>(); else wait_copies<0>();
      if (partly) unseen_values(t, s, vt, lane, bad ? 0 : min(draft0, k1) - key0);
      t.product(vt, p);
      wait_lds();
      if (more) cp.copy(src, src.v, pg, first, each, key0 + 128, k1, 0, vlds, lane);
    }
    __syncthreads();

    // The waves' parts: [wave][row][DP] in the tiles' place, maxima and sums in `pages`.
    float* parts = reinterpret_cast<float*>(smem);
    float2* ml = reinterpret_cast<float2*>(pages);
    const float l = t.total();
    // (rows are 16-byte chunks, permuted by the row against bank conflicts)
    constexpr int kRows = Tile::kRows;
    float4* mine = reinterpret_cast<float4*>(parts + (wave * kRows + lane % kRows) * DP);
    t.each_quad(lane, [&](int ch, float4 v) { mine[ch ^ (lane & 7)] = v; });
    if (lane < kRows) ml[wave * kRows + lane] = make_float2(t.m, l);
    __syncthreads();
    constexpr int kQuads = DP / 4;
    for (int e = threadIdx.x; e < min(kRows, M - r0) * kQuads; e += 256) {
      const int r = e / kQuads, ch = e % kQuads, m = r0 + r;
      if (ch * 4 >= D) continue;
      float2 w[4];
      float mx = kNone;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        w[k] = ml[k * kRows + r];
        mx = fmaxf(mx, w[k].x);
      }
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      float sl = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float f = __builtin_amdgcn_exp2f(w[k].x - mx);
        const float4 v = reinterpret_cast<const float4*>(parts + (k * kRows + r) * DP)[ch ^ (r & 7)];
        sum.x = fmaf(f, v.x, sum.x);
        sum.y = fmaf(f, v.y, sum.y);
        sum.z = fmaf(f, v.z, sum.z);
        sum.w = fmaf(f, v.w, sum.w);
        sl = fmaf(f, w[k].y, sl);
      }
      const int mr = quotient(m, g.groups);
      const size_t at = static_cast<size_t>(slot) * a.rows * a.heads + static_cast<size_t>(rbase + mr) * a.heads +
                        hk * G + remainder_of(m, mr, g.groups);
      *reinterpret_cast<float4*>(g.po + at * D + ch * 4) = sum;
      if (ch == 0) g.pml[at] = make_float2(mx, sl);
    }
  }

  // Drafted keys are seen by some of the rows only (and keys past the range's
  // end or on pages outside the pool by none), and 0 x infinity or NaN is not
  // 0: values of tile rows from `from` on that are not finite are added here
  // to the rows that see them, and zeroed for the product.
  static __device__ __forceinline__ void unseen_values(Tile& t, const typename Tile::Keys& s, lds_u8* vt, int lane,
                                                       int from) {
    const int r = lane & 31;
    constexpr uint16_t kExp = BF ? 0x7F80u : 0x7C00u;
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u32x4 w[CPR / 2];
#pragma unroll
    for (int k = 0; k < CPR / 2; ++k)
      w[k] = *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>(vt + r * ROWB + ((2 * k + (lane >> 5)) << 4));
    u16x2 top = {0, 0};
#pragma unroll
    for (int k = 0; k < CPR / 2; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, w[k][i] & 0x7FFF7FFFu));
    const bool odd = top.x >= kExp || top.y >= kExp;
    const uint64_t all = __ballot(odd && r >= from);
    uint32_t rows = static_cast<uint32_t>(all | (all >> 32));
    while (rows) {
      const int kk = __builtin_ctz(rows);
      rows &= rows - 1;
      const float pk = t.prob(s, kk, lane);
      if (!(pk == 0.f)) t.add_value(vt, kk, pk, lane);
      order_memory();
      if (lane < CPR) zero_chunk(vt + kk * ROWB + lane * 16);
      order_memory();
    }
  }
};

template <bool BF, int DP, class Tile>
__global__ void __launch_bounds__(256, DP == 256 ? 1 : 2) attn_parts_kernel(const AttnKernelArgs g) {
  typedef Attn<BF, DP, Tile> A;
  extern __shared__ __attribute__((aligned(16))) uint8_t attn_lds[];
  int* pages = reinterpret_cast<int*>(attn_lds + A::kLds);
  const qmv_attn_args& a = g.a;
  KeySource src;
  int shift = 31 - __builtin_clz(a.page_size > 0 ? a.page_size : 1);
  src.shift = shift;
  src.npages = static_cast<int>(a.num_pages);
  src.dim = a.head_dim;
  src.page = a.page_stride * 2;
  int id = blockIdx.x;
  const int before = static_cast<int>(g.p.suffix_first ? g.p.suffix_wgs : g.p.prefix_wgs);
  const bool prefix = (id < before) != (g.p.suffix_first != 0);
  if (id >= before) id -= before;
  int hk, rt, slot, k0, k1, rbase = 0, n = static_cast<int>(a.rows), draft0;
  if (prefix) {
    // workgroups of one key head and key range are a multiple of 8 apart where
    // there are a multiple of 8 such pairs: on one XCD, sharing its L2
    rt = quotient(id, g.pairs);
    const int pair = remainder_of(id, rt, g.pairs);
    slot = quotient(pair, g.kv_heads);
    hk = remainder_of(pair, slot, g.kv_heads);
    k0 = slot * g.p.pseg;
    k1 = draft0 = min(k0 + g.p.pseg, static_cast<int>(a.prefix_len));
    src.table = a.prefix_pages;
  } else {
    // A sequence's key heads share lines: of 8 x kv_heads workgroups, those of
    // one XCD are one sequence's heads (another place of the eight each time,
    // so that no XCD gets all the long sequences of a regular batch).  First
    // ranges come before second ones, which only long sequences have.
    const int eights = quotient(id >> 3, g.kv_heads), base = eights * 8 * a.kv_heads;
    if (base + 8 * a.kv_heads <= static_cast<int>(g.p.suffix_wgs))
      id = base + ((id + eights) & 7) * a.kv_heads + remainder_of(id >> 3, eights, g.kv_heads);
    const int q1 = quotient(id, g.kv_heads), q2 = quotient(q1, g.srow_tiles), split = quotient(q2, g.nseq);
    hk = remainder_of(id, q1, g.kv_heads);
    rt = remainder_of(q1, q2, g.srow_tiles);
    const int b = remainder_of(q2, split, g.nseq);
    const int end = a.row_start[b + 1];
    rbase = a.row_start[b];
    const int len = min(max(a.suffix_len[b], 0), static_cast<int>(a.max_suffix));
    if (rbase < 0 || end > n || rbase >= end) return;
    n = min(end - rbase, a.max_rows);
    if (rt * Tile::kRows >= n * g.p.groups) return;
    k0 = split * g.p.sseg;
    k1 = min(k0 + g.p.sseg, len);
    if (k0 >= k1) return;
    slot = g.p.psplits + split;
    draft0 = len - (end - rbase);
    src.table = a.block_table + b * a.table_stride;
  }
  const bool pool = src.table != nullptr;
  src.k = static_cast<const uint8_t*>(pool ? a.k_pages : a.k_prefix) + hk * (pool ? a.page_head : a.prefix_head) * 2;
  src.v = static_cast<const uint8_t*>(pool ? a.v_pages : a.v_prefix) + hk * (pool ? a.page_head : a.prefix_head) * 2;
  src.row = (pool ? a.page_row : a.prefix_row) * 2;
  if (g.p.wide && prefix)
    A::wide(g, src, slot, hk, rt, k0, k1, attn_lds, pages);
  else
    A::narrow(g, src, slot, hk, rbase, n, rt * Tile::kRows, k0, k1, draft0, attn_lds, pages);
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) v = fmaxf(v, __shfl_xor(v, k));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) v += __shfl_xor(v, k);
  return v;
}

// A (row, head) whose output is not finite though its scores are, again,
// plainly.  The products above add 0 x infinity to an infinite value's column
// where the low half of a probability is 0 or the probabilities are used up
// before a new maximum, and their unnormalized sums, of up to 2^15 of every
// value, may pass fp32's range.  Here it is 64 keys at a time, one a lane, in
// fp32: a walk for the maximum and the sum, and one for the output, to which a
// weight of 0 adds nothing.  Every row of 16 x 1 on 8192 tokens this way takes
// 3 ms instead of 18 us, of 64 x 8 on 32768 tokens 45 ms.
// seq, len, draft0, ri: the row's sequence (-1: the prefix alone), its keys,
// those before its rows, and the row's number in it.
template <bool BF, int VEC>
__device__ __forceinline__ void plain_row(const qmv_attn_args& a, int row, int head, int hk, int seq, int len, int draft0,
                                          int ri, float* out, float& lse) {
  const int lane = __lane_id(), D = a.head_dim, d = min(lane * VEC, D - VEC);
  const int shift = 31 - __builtin_clz(a.page_size > 0 ? a.page_size : 1);
  const uint16_t* q = static_cast<const uint16_t*>(a.q) + row * a.q_row + head * a.q_head;
  const uint64_t mask = a.tree_mask ? a.tree_mask[row] : 0;
  const float c = a.scale * kLog2e;
  auto number = [](uint32_t b) { return BF ? bf16_to_f32(b) : f16_to_f32(b); };
  // A walk over the prefix's keys or the row's own, 64 at a time: body(k, v, seen), the lane's key and value.
  auto walk = [&](bool own, auto&& body) __attribute__((always_inline)) {
    const int32_t* table = own ? a.block_table + seq * a.table_stride : a.prefix_pages;
    const bool pool = table != nullptr;
    const uint16_t* k = static_cast<const uint16_t*>(pool ? a.k_pages : a.k_prefix) + hk * (pool ? a.page_head : a.prefix_head);
    const uint16_t* v = static_cast<const uint16_t*>(pool ? a.v_pages : a.v_prefix) + hk * (pool ? a.page_head : a.prefix_head);
    const int n = own ? len : static_cast<int>(a.prefix_len);
    for (int j0 = 0; j0 < n; j0 += 64) {
      const int j = min(j0 + lane, n - 1), slot = j - draft0;
      bool seen = j0 + lane < n;
      if (own && slot >= 0) seen &= a.tree_mask ? slot < 64 && (mask >> (slot & 63) & 1) : slot <= ri;
      int64_t at = j * a.prefix_row;
      if (pool) {
        const int page = table[j >> shift];
        seen &= page >= 0 && page < a.num_pages;
        at = page * a.page_stride + (j & ((1 << shift) - 1)) * a.page_row;
      }
      body(k + at, v + at, seen);
    }
  };
  auto score = [&](const uint16_t* k) __attribute__((always_inline)) {
    float s = 0.f;
    for (int i = 0; i < D; i += 8) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(k + i), y = *reinterpret_cast<const u32x4*>(q + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s = fmaf(number(x[e] & 0xFFFF), number(y[e] & 0xFFFF), s);
        s = fmaf(number(x[e] >> 16), number(y[e] >> 16), s);
      }
    }
    return s * c;
  };
  float m = kNone, l = 0.f;
  for (int part = 0; part < (seq >= 0 ? 2 : 1); ++part)
    walk(part, [&](const uint16_t* k, const uint16_t*, bool seen) __attribute__((always_inline)) {
      if (!seen) return;
      const float s = score(k), mn = fmaxf(m, s);
      l = fmaf(l, __builtin_amdgcn_exp2f(m - mn), __builtin_amdgcn_exp2f(s - mn));
      m = mn;
    });
  const float mx = wave_max(m);
  l = wave_sum(l * __builtin_amdgcn_exp2f(m - mx));
#pragma unroll
  for (int k = 0; k < VEC; ++k) out[k] = 0.f;
  lse = l == 0.f ? -INFINITY : (mx + __builtin_amdgcn_logf(l)) * kLn2;
  if (l == 0.f) return;
  for (int part = 0; part < (seq >= 0 ? 2 : 1); ++part)
    walk(part, [&](const uint16_t* k, const uint16_t* v, bool seen) __attribute__((always_inline)) {
      float p = 0.f;
      if (seen) p = __builtin_amdgcn_exp2f(score(k) - mx) / l;
      for (uint64_t some = __ballot(!(p == 0.f)); some; some &= some - 1) {
        const int key = __builtin_ctzll(some);
        const uint16_t* at = reinterpret_cast<const uint16_t*>(__shfl(reinterpret_cast<uint64_t>(v), key)) + d;
        const float pk = __shfl(p, key);
#pragma unroll
        for (int e = 0; e < VEC; ++e) out[e] = fmaf(pk, number(at[e]), out[e]);
      }
    });
}

// A (row, head)'s parts joined in a fixed order: by one wave (WAVES = 1), or
// by the four of a workgroup, a quarter of the parts each.  The first loads --
// maxima and sums, row starts, suffix lengths -- go out together, whatever
// they will turn out to be needed for.
template <bool BF, int VEC, int WAVES>
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnKernelArgs g) {
  const qmv_attn_args& a = g.a;
  const int lane = __lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), D = a.head_dim;
  const int64_t all = a.rows * a.heads;
  const int64_t e = WAVES == 4 ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * 4 + wave;
  if (WAVES == 1 && e >= all) return;
  const int row = quotient(static_cast<int>(e), g.heads), head = remainder_of(static_cast<int>(e), row, g.heads);
  const int most = g.p.psplits + g.p.ssplits;
  float2 ml = make_float2(kNone, 0.f);
  if (lane < most) ml = g.pml[lane * all + e];
  // the row's sequence: the last that starts at or before it
  int seq = -1, start = 0, end = 0, len = 0;
  if (a.nseq < 64) {
    const int rs = a.row_start[min(lane, a.nseq)];
    const int sl = a.max_suffix > 0 ? a.suffix_len[min(lane, a.nseq - 1)] : 0;
    seq = __popcll(__ballot(lane < a.nseq && rs <= row)) - 1;
    start = __shfl(rs, max(seq, 0));
    end = __shfl(rs, max(seq, 0) + 1);
    len = __shfl(sl, max(seq, 0));
  } else {
    for (int b0 = 0; b0 < a.nseq; b0 += 64) {
      const int b = b0 + lane;
      seq += __popcll(__ballot(b < a.nseq && a.row_start[min(b, a.nseq)] <= row));
    }
    if (seq >= 0) {
      start = a.row_start[seq];
      end = a.row_start[seq + 1];
      len = a.max_suffix > 0 ? a.suffix_len[seq] : 0;
    }
  }
  int slots = g.p.psplits;
  bool past = false, own = false;
  if (seq >= 0 && start >= 0 && row >= start && row < end && end <= a.rows) {
    past = row - start >= a.max_rows;
    len = min(max(len, 0), static_cast<int>(a.max_suffix));
    own = true;
    if (!past && len > 0) slots += (len + g.p.sseg - 1) / g.p.sseg;
  }
  slots = __builtin_amdgcn_readfirstlane(slots);
  float mx = lane < slots ? ml.x : kNone;
  for (int s = lane + 64; s < slots; s += 64) mx = fmaxf(mx, g.pml[s * all + e].x);
  mx = wave_max(mx);
  float acc[VEC] = {}, l = 0.f;
  const int d = lane * VEC;
  const float* p = g.po + e * D + min(d, D - VEC);
  for (int s0 = 0; s0 < slots; s0 += 64) {
    if (s0) ml = g.pml[min(s0 + lane, slots - 1) * all + e];
    const float f = s0 + lane < slots ? __builtin_amdgcn_exp2f(ml.x - mx) : 0.f;
    l += s0 + lane < slots ? f * ml.y : 0.f;
    const int n = min(slots - s0, 64);
    // eight parts' loads in flight
    constexpr int kBatch = 8;
    for (int s = WAVES == 4 ? wave : 0; s < n; s += kBatch * WAVES) {
      float v[kBatch][VEC];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        __builtin_memcpy(v[u], __builtin_assume_aligned(p + (s0 + min(s + u * WAVES, n - 1)) * all * D, VEC * 4),
                         sizeof(v[u]));
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int su = s + u * WAVES;
        if (su >= n) break;
        const float fs = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(f), su));
#pragma unroll
        for (int k = 0; k < VEC; ++k) acc[k] = fmaf(fs, v[u][k], acc[k]);
      }
    }
  }
  l = wave_sum(l);
  if constexpr (WAVES == 4) {
    __shared__ float part[3][64 * VEC];
    if (wave)
#pragma unroll
      for (int k = 0; k < VEC; ++k) part[wave - 1][k * 64 + lane] = acc[k];
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int w = 0; w < 3; ++w)
#pragma unroll
      for (int k = 0; k < VEC; ++k) acc[k] += part[w][k * 64 + lane];
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  float lse = l == 0.f ? -INFINITY : (mx + __builtin_amdgcn_logf(l)) * kLn2;
  bool odd = false;
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    acc[k] = past ? __builtin_nanf("") : acc[k] * inv;
    odd |= !(fabsf(acc[k]) < INFINITY);
  }
  if (past) {
    lse = __builtin_nanf("");
  } else if (l == l && __any(odd && d < D)) {
    plain_row<BF, VEC>(a, row, head, head / g.p.groups, own ? seq : -1, len, len - (end - start), row - start, acc, lse);
  }
  if (d < D) {
    uint16_t* out = static_cast<uint16_t*>(a.out) + row * a.out_row + head * a.out_head + d;
    uint16_t w[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k)
      w[k] = BF ? __builtin_bit_cast(uint16_t, static_cast<__bf16>(acc[k]))
                : __builtin_bit_cast(uint16_t, static_cast<_Float16>(acc[k]));
    __builtin_memcpy(__builtin_assume_aligned(out, VEC * 2), w, sizeof(w));
  }
  if (a.lse && lane == 0) a.lse[e] = lse;
}

static int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

// Workgroups at a time: two a compute unit.
constexpr int kResident = 512;
// Microseconds that workgroups were measured to take beside a full chip's
// others: to begin and end, a wide tile of 64 keys, the four waves' narrow
// tiles of 32 (128-wide heads).
constexpr double kStartUs = 4.0, kWideTileUs = 2.2, kNarrowTilesUs = 1.5;

// How many ranges to cut `keys` into for each of `units` row tiles: the fewest
// microseconds, by workgroups of `tile` microseconds for each `tile_keys`
// keys, the parts' way through the workspace, written and read at 2 TB/s, and
// `other` microseconds of other workgroups that fill the slots left free.
static int64_t key_ranges(int64_t keys, int64_t units, int tile_keys, double tile, double part_bytes, double other) {
  const int64_t tiles = (keys + tile_keys - 1) / tile_keys;
  double best = 1e30;
  int64_t n = 1;
  for (int64_t s = 1; s <= tiles && s <= 256; ++s) {
    const int64_t rounds = (units * s + kResident - 1) / kResident;
    const double each = kStartUs + tile * static_cast<double>((tiles + s - 1) / s);
    const double left = other - static_cast<double>(rounds * kResident - units * s) * each;
    const double us = static_cast<double>(rounds) * each + (left > 0 ? left / kResident + kStartUs * 2 : 0.0) +
                      static_cast<double>(s) * part_bytes * 2 / 2e6;
    if (us < best) {
      best = us;
      n = s;
    }
  }
  return n;
}

// Most keys of one workgroup where they lie in pages (rounded up to a
// multiple of 128 they and a page that they begin within still fit).
static int64_t paged_keys(const qmv_attn_args& a) {
  return a.page_size >= 128 ? static_cast<int64_t>(a.page_size) * (kMaxPages - 2)
                            : static_cast<int64_t>(a.page_size) * (kMaxPages - 128 / a.page_size - 1) / 128 * 128;
}

static AttnPlan plan_attn(const qmv_attn_args& a) {
  AttnPlan p = {};
  p.groups = a.heads / a.kv_heads;
  const int64_t M = a.rows * p.groups;
  const double part = static_cast<double>(a.rows) * a.heads * a.head_dim * 4;
  // Rows of one copy instruction (TileCopy::RPI at this width).
  const int rpi = a.head_dim <= 64 ? 8 : a.head_dim <= 128 ? 4 : 2;
  const int64_t near = int64_t{1} << 27;  // elements
  const bool pages_fit = a.page_size >= rpi && a.page_row < near;
  p.each = pages_fit;
  // (112 rows: wide tiles take 30 us on 32768 tokens, narrow ones 43; on 1024 tokens 13.0 and 12.1)
  p.wide = M > 64 && (a.prefix_pages ? pages_fit : a.prefix_row < near);
  const int64_t suffix_rows = std::min<int64_t>(a.max_rows, a.rows) * p.groups;
  p.rows = suffix_rows <= 16 && (p.wide || M <= 16 || a.prefix_len == 0) ? 16 : 32;
  p.row_tiles = ceil_div(M, p.wide ? 128 : p.rows);
  const double width = (a.head_dim <= 64 ? 64 : a.head_dim <= 128 ? 128 : 256) / 128.0;
  double suffix_us = 0.0;
  if (a.max_suffix > 0) {
    p.srow_tiles = ceil_div(suffix_rows, p.rows);
    // (sequences are seldom all as long as the longest: with a quarter of the ranges
    // counted, 32 suffixes of 211 to 2111 tokens took 48.5 us, with half 50.6, an eighth 52.5)
    const int64_t units = static_cast<int64_t>(a.nseq) * a.kv_heads * p.srow_tiles;
    const int64_t n = std::max<int64_t>(
        key_ranges(a.max_suffix, (units + 3) / 4, 128, kNarrowTilesUs * width, part, 0.0), ceil_div(a.max_suffix, paged_keys(a)));
    p.sseg = ceil_div(ceil_div(a.max_suffix, n), 128) * 128;
    p.ssplits = ceil_div(a.max_suffix, p.sseg);
    p.suffix_wgs = units * p.ssplits;
    suffix_us = static_cast<double>(p.suffix_wgs) * (kStartUs + kNarrowTilesUs * width * p.sseg / 128.0);
  }
  if (a.prefix_len > 0) {
    const int64_t units = static_cast<int64_t>(p.row_tiles) * a.kv_heads;
    int64_t n = p.wide ? key_ranges(a.prefix_len, units, 64, kWideTileUs * width, part, suffix_us)
                       : key_ranges(a.prefix_len, units, 128, kNarrowTilesUs * width, part, suffix_us);
    if (a.prefix_pages) n = std::max<int64_t>(n, ceil_div(a.prefix_len, paged_keys(a)));
    p.pseg = ceil_div(ceil_div(a.prefix_len, n), 64) * 64;
    p.psplits = ceil_div(a.prefix_len, p.pseg);
    p.prefix_wgs = units * p.psplits;
  }
  p.suffix_first = p.sseg > p.pseg;
  return p;
}

bool attn_fits(const qmv_attn_args& a) {
  const AttnPlan p = plan_attn(a);
  return p.prefix_wgs + p.suffix_wgs <= UINT32_MAX / 256;  // (a launch of 2^32 work-items and more wraps around, with no error)
}

static size_t ml_bytes(const qmv_attn_args& a, const AttnPlan& p) {
  return (static_cast<size_t>(p.psplits + p.ssplits) * a.rows * a.heads * sizeof(float2) + 255) / 256 * 256;
}

size_t attn_workspace(const qmv_attn_args& a) {
  const AttnPlan p = plan_attn(a);
  return ml_bytes(a, p) + static_cast<size_t>(p.psplits + p.ssplits) * a.rows * a.heads * a.head_dim * sizeof(float);
}

template <bool BF, int DP, class Tile>
static hipError_t launch_parts(const AttnKernelArgs& g, hipStream_t s) {
  constexpr int lds = Attn<BF, DP, Tile>::kLds + kMaxPages * 4;
  const unsigned grid = static_cast<unsigned>(g.p.prefix_wgs + g.p.suffix_wgs);
  if (grid) hipLaunchKernelGGL((attn_parts_kernel<BF, DP, Tile>), dim3(grid), dim3(256), lds, s, g);
  return hipGetLastError();
}

template <bool BF>
static hipError_t attn_typed(const AttnKernelArgs& g, hipStream_t s) {
  const int D = g.a.head_dim;
  const auto parts = [&](auto width) {
    constexpr int DP = decltype(width)::value;
    return g.p.rows == 16 ? launch_parts<BF, DP, Narrow16<BF, DP>>(g, s) : launch_parts<BF, DP, Narrow32<BF, DP>>(g, s);
  };
  const hipError_t e = D <= 64    ? parts(std::integral_constant<int, 64>{})
                       : D <= 128 ? parts(std::integral_constant<int, 128>{})
                                  : parts(std::integral_constant<int, 256>{});
  if (e != hipSuccess) return e;
  // Few rows of many parts: four waves to a row (5 draft trees take 13.1 us a
  // call, with one wave 17.1; 256 x 1 rows of few parts 44, with four waves 53).
  const int64_t all = g.a.rows * g.a.heads;
  if (all <= 8192 && g.p.psplits + g.p.ssplits >= 8) {
    const dim3 grid(static_cast<unsigned>(all));
    if (D <= 128)
      hipLaunchKernelGGL((attn_join_kernel<BF, 2, 4>), grid, dim3(256), 0, s, g);
    else
      hipLaunchKernelGGL((attn_join_kernel<BF, 4, 4>), grid, dim3(256), 0, s, g);
  } else {
    const dim3 grid(ceil_div(all, 4));
    if (D <= 128)
      hipLaunchKernelGGL((attn_join_kernel<BF, 2, 1>), grid, dim3(256), 0, s, g);
    else
      hipLaunchKernelGGL((attn_join_kernel<BF, 4, 1>), grid, dim3(256), 0, s, g);
  }
  return hipGetLastError();
}

hipError_t attn(const qmv_attn_args& a, void* ws, hipStream_t s) {
  AttnKernelArgs g;
  g.a = a;
  g.p = plan_attn(a);
  g.groups = fast_div(g.p.groups);
  g.pairs = fast_div(std::max<int64_t>(1, static_cast<int64_t>(a.kv_heads) * g.p.psplits));
  g.kv_heads = fast_div(a.kv_heads);
  g.srow_tiles = fast_div(std::max(1, g.p.srow_tiles));
  g.nseq = fast_div(a.nseq);
  g.heads = fast_div(a.heads);
  g.pml = static_cast<float2*>(ws);
  g.po = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + ml_bytes(a, g.p));
  return a.dtype == QMV_BF16 ? attn_typed<true>(g, s) : attn_typed<false>(g, s);
}

}  // namespace qmv
