// Verification of drafted tokens by rejection sampling (qmv_verify):
//   p = softmax(logits / T); draft x accepted where u q(x) < p(x); the first
//   row that is not accepted draws from max(p - q, 0), all accepted from p.
//
// Two launches.  The first cuts every row of logits into pieces of kPiece and
// leaves each piece's maximum, its first place and the sum of
// e^((l - maximum) / T).  In the second, every workgroup of a sequence settles
// from those sums which drafts are accepted and adds up its pieces of the row
// that draws; the last of a sequence to finish finds the token in the piece
// that holds it.  (A row of accepted drafts draws from p, whose pieces are
// added up already: one workgroup does it.)
//
// Exponentials and sums are in 64 bits.  A draw compares a running sum of up
// to 2^24 probabilities with u times their total; in 32 bits their errors
// would move, by estimate (152064 borders, an error of 2^-24 or so), about one
// draw in a hundred over flat probabilities to a neighbouring token.  An
// exponential takes some eighteen 64-bit instructions.  The first launch takes
// 46 us (the fastest of 40) on 288 rows of 152064 fp32 logits, whose reads
// alone, 175 MB, would take 25 at 7.08 TB/s: a SIMD issues a vector
// instruction every 7.4 clocks, and its waves wait half of their time to issue
// and 37 % for loads (counters).
#include <algorithm>

#include "device_util.h"
#include "launch.h"

namespace qmv {

// The first launch: a wave's piece of a row, and its workgroup's four.
constexpr int kRowThreads = 256, kRowPer = 32, kPiece = 64 * kRowPer;
// The second: a workgroup's slice, a piece again (one or, where there are
// sequences enough to fill the chip, several of them).  Four 64-bit weights to
// a thread: they are the longest step of a lone sequence (with 8192 tokens to
// 1024 threads of one compute unit, 12.3 us against 8.6, the fastest of 40).
constexpr int kThreads = 512, kWaves = kThreads / 64, kPer = 4;
static_assert(kThreads * kPer == kPiece, "a slice is a piece");

struct PieceStat {
  double sum;   // of e^((l - max) / T); of the infinities' ones where max is +inf
  float max;
  int best;     // the first place of max, at temperature 0
};

struct VerifyArgs {
  qmv_verify_args a;
  int pieces;        // of a row
  int span;          // pieces of a workgroup of the second launch
  PieceStat* stat;   // [row][piece]
  double* part;      // [sequence][piece]: the drawing row's weights
  uint32_t* done;    // [sequence]: workgroups that have left their part
};

constexpr double kLog2e = 1.4426950408889634074;

// 2^y for y <= 0, within 3e-14 of itself: 2^n p(f), y = n + f, |f| <= 1/2, p the
// polynomial of degree 9 that equals 2^f at the ten Chebyshev nodes of
// [-1/2, 1/2] (1.8e-14 from it between them).
__device__ __forceinline__ double exp2_neg(double y) {
  y = fmax(y, -1100.0);  // (2^-1100 is 0; -inf too)
  // (adding 1.5 x 2^52 rounds to a whole number and leaves it in the low word)
  const double big = y + 6755399441055744.0, n = big - 6755399441055744.0, f = y - n;
  double p = 1.0205905413765595e-07;
  p = fma(p, f, 1.3259645244887111e-06);
  p = fma(p, f, 1.5252672924850737e-05);
  p = fma(p, f, 0.0001540343375125101);
  p = fma(p, f, 0.0013333558200794592);
  p = fma(p, f, 0.0096181291939343126);
  p = fma(p, f, 0.05550410866465167);
  p = fma(p, f, 0.24022650695640341);
  p = fma(p, f, 0.69314718055994617);
  p = fma(p, f, 1.0000000000000135);
  return __builtin_amdgcn_ldexp(p, __double2loint(big));
}

// e^((l - m) / T), the weight of a logit against the maximum m; a maximum of
// +inf shares everything among the infinities.  c = log2(e) / T.  FINITE: m
// is known to be finite, and no branch parts the exponentials of a loop.
template <bool FINITE = false>
__device__ __forceinline__ double weight(float l, float m, double c) {
  if (!FINITE && m == INFINITY) return l == INFINITY ? 1.0 : 0.0;
  return exp2_neg((static_cast<double>(l) - static_cast<double>(m)) * c);
}

template <int DT>
struct Logits;
template <>
struct Logits<QMV_F32> {
  typedef uint32_t word;
  static __device__ __forceinline__ float get(const uint32_t* w, int i) { return __uint_as_float(w[i]); }
};
template <>
struct Logits<QMV_F16> {
  typedef uint16_t word;
  static __device__ __forceinline__ float get(const uint32_t* w, int i) { return f16_to_f32(w[i / 2] >> (i & 1) * 16 & 0xFFFF); }
};
template <>
struct Logits<QMV_BF16> {
  typedef uint16_t word;
  static __device__ __forceinline__ float get(const uint32_t* w, int i) { return bf16_to_f32(w[i / 2] >> (i & 1) * 16 & 0xFFFF); }
};

// NaN as -inf, in one instruction (fmaxf quiets its operands first).
__device__ __forceinline__ float no_nan(float v) {
  __asm__("v_max_f32 %0, %1, %2" : "=v"(v) : "v"(v), "s"(-INFINITY));
  return v;
}

// One logit, NaN as -inf.
template <int DT>
__device__ __forceinline__ float logit(const qmv_verify_args& a, int64_t row, int64_t i) {
  const typename Logits<DT>::word w = static_cast<const typename Logits<DT>::word*>(a.logits)[row * a.logits_row + i];
  const uint32_t v = w;
  return no_nan(Logits<DT>::get(&v, 0));
}

// Values of one load: 16 bytes, or a thread's N values where they are fewer.
template <int DT, int N>
constexpr int values_of_load() {
  constexpr int k = 16 / static_cast<int>(sizeof(typename Logits<DT>::word));
  return N < k ? N : k;
}

// N consecutive values from place i0 of a row of n, at any alignment of its
// type; places from n on give `past`.
template <int DT, int N>
__device__ __forceinline__ void load_row(const void* row, int64_t i0, int64_t n, float past, float* v) {
  typedef typename Logits<DT>::word word;
  constexpr int kV = values_of_load<DT, N>();
  static_assert(N % kV == 0 && (kV * sizeof(word) == 16 || kV * sizeof(word) == 8), "loads of 8 or 16 bytes");
#pragma unroll
  for (int k = 0; k < N; k += kV) {
    if (i0 + k + kV <= n) {
      const uint8_t* at = reinterpret_cast<const uint8_t*>(static_cast<const word*>(row) + i0 + k);
      uint32_t x[4];
      if constexpr (kV * sizeof(word) == 16) {
        const uint4 w = ld16_any(at);
        x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
      } else {
        const uint2 w = ld8_any(at);
        x[0] = w.x, x[1] = w.y;
      }
#pragma unroll
      for (int j = 0; j < kV; ++j) v[k + j] = Logits<DT>::get(x, j);
    } else {
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        v[k + j] = past;
        if (i0 + k + j < n) {
          const uint32_t w = static_cast<const word*>(row)[i0 + k + j];
          v[k + j] = Logits<DT>::get(&w, 0);
        }
      }
    }
  }
}

// The place of value j of the N of thread t of THREADS, one load a thread at a time.
template <int DT, int THREADS, int N>
__device__ __forceinline__ int place(int t, int j) {
  constexpr int kV = values_of_load<DT, N>();
  return (j / kV) * THREADS * kV + t * kV + j % kV;
}
template <int DT, int THREADS, int N>
__device__ __forceinline__ void load_pieces(const void* row, int64_t s0, int t, int64_t n, float past, float* v) {
  constexpr int kV = values_of_load<DT, N>();
#pragma unroll
  for (int k = 0; k < N; k += kV) load_row<DT, kV>(row, s0 + place<DT, THREADS, N>(t, k), n, past, v + k);
}

// v of the lane that a DPP control names (lanes without one, or outside the
// row mask: zero).
template <int CTRL, int ROWS = 0xF, class T>
__device__ __forceinline__ T dpp_of(T v) {
  if constexpr (sizeof(T) == 8) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), CTRL, ROWS, 0xF, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), CTRL, ROWS, 0xF, true);
    return __builtin_bit_cast(T, static_cast<uint64_t>(hi) << 32 | lo);
  } else {
    return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xF, true));
  }
}

// f over the wave, to every lane, in a fixed order: quads, halves of a row of
// 16 and rows by DPP, then rows and halves of the wave by swaps.
template <class T, class F>
__device__ __forceinline__ T wave_fold(T v, F&& f) {
  v = f(v, dpp_of<0xB1>(v));   // quad_perm [1,0,3,2]
  v = f(v, dpp_of<0x4E>(v));   // quad_perm [2,3,0,1]
  v = f(v, dpp_of<0x141>(v));  // row_half_mirror
  v = f(v, dpp_of<0x140>(v));  // row_mirror
  auto swap16 = [](uint32_t x) { return __builtin_amdgcn_permlane16_swap(x, x, false, false); };
  auto swap32 = [](uint32_t x) { return __builtin_amdgcn_permlane32_swap(x, x, false, false); };
  auto both = [&](auto swap) {
    if constexpr (sizeof(T) == 8) {
      const uint64_t b = __builtin_bit_cast(uint64_t, v);
      const auto lo = swap(static_cast<uint32_t>(b)), hi = swap(static_cast<uint32_t>(b >> 32));
      return f(__builtin_bit_cast(T, static_cast<uint64_t>(hi[0]) << 32 | lo[0]),
               __builtin_bit_cast(T, static_cast<uint64_t>(hi[1]) << 32 | lo[1]));
    } else {
      const auto x = swap(__builtin_bit_cast(uint32_t, v));
      const uint32_t x0 = x[0], x1 = x[1];
      return f(__builtin_bit_cast(T, x0), __builtin_bit_cast(T, x1));
    }
  };
  v = both(swap16);
  v = both(swap32);
  return v;
}
__device__ __forceinline__ double add(double x, double y) { return x + y; }
// (of two numbers that are not NaN; one instruction, as no_nan)
__device__ __forceinline__ float larger(float x, float y) {
  __asm__("v_max_f32 %0, %1, %2" : "=v"(x) : "v"(x), "v"(y));
  return x;
}

// The sequence of a row (the last that starts at or before it), or -1.
__device__ __forceinline__ int sequence_of(const qmv_verify_args& a, int row) {
  int seq = -1;
  for (int b0 = 0; b0 < a.nseq; b0 += 64) {
    const int b = b0 + static_cast<int>(__lane_id());
    seq += __popcll(__ballot(b < a.nseq && a.row_start[min(b, a.nseq)] <= row));
  }
  return seq >= 0 && row < a.row_start[seq + 1] ? seq : -1;
}

__device__ __forceinline__ float temperature_of(const qmv_verify_args& a, int seq) {
  const float t = a.temperature ? a.temperature[seq] : 1.f;
  return t > 0.f ? t : 0.f;
}

template <int DT>
__global__ void __launch_bounds__(kRowThreads) verify_rows_kernel(const VerifyArgs g) {
  const qmv_verify_args& a = g.a;
  const int row = blockIdx.y, lane = __lane_id();
  const int piece = blockIdx.x * (kRowThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (blockIdx.x == 0 && row == 0)
    for (int b = threadIdx.x; b < a.nseq; b += kRowThreads) g.done[b] = 0;
  if (row >= a.rows || piece >= g.pieces) return;  // (a launch without rows only clears the counts)
  const int64_t s0 = static_cast<int64_t>(piece) * kPiece;
  float v[kRowPer];
  load_pieces<DT, 64, kRowPer>(static_cast<const typename Logits<DT>::word*>(a.logits) + row * a.logits_row, s0, lane,
                               a.vocab, -INFINITY, v);
  const int seq = sequence_of(a, row);
  if (seq < 0) {
    if (piece == 0 && lane == 0) a.out_tokens[row] = -1;
    return;
  }
  const float t = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(temperature_of(a, seq))));
  float m4[4];
#pragma unroll
  for (int j = 0; j < kRowPer; ++j) {
    v[j] = no_nan(v[j]);
    m4[j & 3] = j < 4 ? v[j] : larger(m4[j & 3], v[j]);
  }
  float m = wave_fold(larger(larger(m4[0], m4[1]), larger(m4[2], m4[3])), larger);
  m = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(m)));
  int best = 0;
  double s = 0.0;
  if (t == 0.f) {  // only the first place of the maximum counts
    best = INT32_MAX;
#pragma unroll
    for (int j = kRowPer - 1; j >= 0; --j) best = v[j] == m ? place<DT, 64, kRowPer>(lane, j) : best;
    best = wave_fold(best, [](int x, int y) { return min(x, y); });
  } else if (m == INFINITY) {
#pragma unroll
    for (int j = 0; j < kRowPer; ++j) s += v[j] == INFINITY ? 1.0 : 0.0;
    s = wave_fold(s, add);
  } else if (m > -INFINITY) {
    const double c_t = kLog2e / static_cast<double>(t);
    double s2[2] = {0.0, 0.0};
#pragma unroll
    for (int j = 0; j < kRowPer; ++j) s2[j & 1] += weight<true>(v[j], m, c_t);
    s = wave_fold(s2[0] + s2[1], add);
  }
  if (lane == 0) g.stat[static_cast<int64_t>(row) * g.pieces + piece] = PieceStat{s, m, static_cast<int>(s0) + best};
}

// A row's maximum, its first place and its sum, from its pieces' (by a wave).
struct RowStat {
  float max;
  int best;
  double sum;
};
__device__ __forceinline__ RowStat row_stat(const VerifyArgs& g, int row, double c_t) {
  const PieceStat* st = g.stat + static_cast<int64_t>(row) * g.pieces;
  const int lane = __lane_id();
  // (the first pieces are kept, 128 of them)
  constexpr int kKeep = 2;
  PieceStat x[kKeep];
  float m = -INFINITY;
#pragma unroll
  for (int k = 0; k < kKeep; ++k) {
    x[k] = st[min(lane + 64 * k, g.pieces - 1)];
    if (lane + 64 * k >= g.pieces) x[k] = PieceStat{0.0, -INFINITY, INT32_MAX};
    m = larger(m, x[k].max);
  }
  for (int s = lane + 64 * kKeep; s < g.pieces; s += 64) m = larger(m, st[s].max);
  m = wave_fold(m, larger);
  int best = INT32_MAX;
  double sum = 0.0;
  auto take = [&](const PieceStat& y) {
    if (y.max == m) best = min(best, y.best);
    sum += y.sum * weight(y.max, m, c_t);
  };
#pragma unroll
  for (int k = 0; k < kKeep; ++k) take(x[k]);
  for (int s = lane + 64 * kKeep; s < g.pieces; s += 64) take(st[s]);
  best = wave_fold(best, [](int y, int z) { return min(y, z); });
  return RowStat{m, best, wave_fold(sum, add)};
}

// A drawing row: the weights max(p - q, 0) S, S the row's sum, so that
// nothing is divided (q is the draft's probabilities, one at x, or nothing).
struct Draw {
  int64_t row;
  float max;
  double sum, c_t;
  const float* q;  // NULL: one at `hot` (-1: nothing)
  int hot;
};
template <bool FINITE>
__device__ __forceinline__ double draw_weight(const Draw& d, float l, float q, int64_t i) {
  const double w = weight<FINITE>(l, d.max, d.c_t);
  const double take = d.q ? (q > 0.f ? static_cast<double>(q) * d.sum : 0.0) : i == d.hot ? d.sum : 0.0;
  return w > take ? w - take : 0.0;
}

// The weights of kPer logits at the given places of a row of n.
template <class F>
__device__ __forceinline__ void draw_weights(const Draw& d, const float* v, const float* q, int64_t n, double* w, F&& at) {
  if (d.max < INFINITY) {
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      w[j] = at(j) < n ? draw_weight<true>(d, v[j], d.q ? q[j] : 0.f, at(j)) : 0.0;
  } else {
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      w[j] = at(j) < n ? draw_weight<false>(d, v[j], d.q ? q[j] : 0.f, at(j)) : 0.0;
  }
}

// Inclusive running sum over the wave's lanes.
__device__ __forceinline__ double wave_scan(double v) {
  v += dpp_of<0x111>(v);  // row_shr:1
  v += dpp_of<0x112>(v);
  v += dpp_of<0x114>(v);
  v += dpp_of<0x118>(v);
  v += dpp_of<0x142, 0xA>(v);  // row_bcast:15, to rows 1 and 3
  v += dpp_of<0x143, 0xC>(v);  // row_bcast:31, to rows 2 and 3
  return v;
}

// The token: the first whose running sum passes u times the total (by the
// whole workgroup).  target: from the target's own probabilities, whose pieces
// the first launch added up.
template <int DT>
__device__ __forceinline__ int find_token(const VerifyArgs& g, int b, const Draw& d0, float u, bool target) {
  const qmv_verify_args& a = g.a;
  const int tid = threadIdx.x, lane = __lane_id(), wave = tid >> 6;
  __shared__ double sh_goal;
  __shared__ int sh_piece, sh_plain, sh_first[kWaves], sh_last[kWaves];
  __shared__ double sh_sum[kWaves];
  Draw d = d0;
  if (wave == 0) {
    bool plain = target;
    double total = 0.0;
    auto part = [&](int s) {
      if (s >= g.pieces) return 0.0;
      if (!plain) return __hip_atomic_load(g.part + static_cast<int64_t>(b) * g.pieces + s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      const PieceStat st = g.stat[d.row * g.pieces + s];
      return st.sum * weight(st.max, d.max, d.c_t);
    };
    for (;;) {
      total = 0.0;
      for (int s0 = 0; s0 < g.pieces; s0 += 64) total += wave_fold(part(s0 + lane), add);
      if (total > 0.0 || plain) break;
      plain = true;  // nothing is left over q: the target's own probabilities
    }
    const double goal = static_cast<double>(u) * total;
    double before = 0.0;
    int piece = -1, last = 0;
    double base = 0.0;
    for (int s0 = 0; s0 < g.pieces && piece < 0; s0 += 64) {
      const double v = part(s0 + lane), c = wave_scan(v) + before;
      const uint64_t some = __ballot(v > 0.0), over = __ballot(c > goal && v > 0.0);
      if (some) last = s0 + 63 - __builtin_clzll(some);
      if (over) {
        const int l = __builtin_ctzll(over);
        piece = s0 + l;
        base = __shfl(c, l) - __shfl(v, l);
      }
      before = __shfl(c, 63);
    }
    if (lane == 0) {
      sh_piece = piece >= 0 ? piece : last;  // (rounding: the last piece of any weight, to its end)
      sh_goal = piece >= 0 ? goal - base : INFINITY;
      sh_plain = plain;
    }
  }
  __syncthreads();
  if (sh_plain) {
    d.q = nullptr;
    d.hot = -1;
  }
  // contiguous places to a thread
  const int64_t i0 = static_cast<int64_t>(sh_piece) * kPiece + tid * kPer;
  const void* row = static_cast<const typename Logits<DT>::word*>(a.logits) + d.row * a.logits_row;
  float v[kPer], q[kPer];
  load_row<DT, kPer>(row, i0, a.vocab, -INFINITY, v);
#pragma unroll
  for (int j = 0; j < kPer; ++j) v[j] = no_nan(v[j]);
  if (d.q) load_row<QMV_F32, kPer>(d.q, i0, a.vocab, 0.f, q);
  double w[kPer], s = 0.0;
  draw_weights(d, v, q, a.vocab, w, [&](int j) { return i0 + j; });
#pragma unroll
  for (int j = 0; j < kPer; ++j) s += w[j];
  double c = wave_scan(s);
  if (lane == 63) sh_sum[wave] = c;
  __syncthreads();
  for (int k = 0; k < wave; ++k) c += sh_sum[k];
  c -= s;
  int first = INT32_MAX, last = -1;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    c += w[j];
    if (w[j] > 0.0) {
      last = static_cast<int>(i0) + j;
      if (c > sh_goal) first = min(first, last);
    }
  }
  first = wave_fold(first, [](int x, int y) { return min(x, y); });
  last = wave_fold(last, [](int x, int y) { return max(x, y); });
  if (lane == 0) {
    sh_first[wave] = first;
    sh_last[wave] = last;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kWaves; ++k) {
    first = min(first, sh_first[k]);
    last = max(last, sh_last[k]);
  }
  return first == INT32_MAX ? last : first;
}

template <int DT>
__global__ void __launch_bounds__(kThreads) verify_draw_kernel(const VerifyArgs g) {
  const qmv_verify_args& a = g.a;
  const int first_piece = blockIdx.x * g.span, b = blockIdx.y, tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r0 = min(max(a.row_start[b], 0), static_cast<int>(a.rows));
  const int end = min(max(a.row_start[b + 1], r0), static_cast<int>(a.rows));
  const int n = min(end - r0, a.max_rows);
  const float t = temperature_of(a, b), u = a.u_sample[b];
  const bool greedy = t == 0.f;
  const double c_t = greedy ? 0.0 : kLog2e / static_cast<double>(t);

  // The first row whose draft is not accepted, a wave to a row.
  __shared__ int sh_ok[kWaves];
  __shared__ RowStat sh_stat[kWaves];
  int at = 0;
  RowStat rs{-INFINITY, 0, 0.0};
  for (int t0 = 0; t0 < n; t0 += kWaves) {
    const int i = t0 + wave;
    if (i < n) {
      const int r = r0 + i;
      const int draft = i + 1 < n ? a.tokens[r + 1] : -1;
      const bool known = draft >= 0 && draft < a.vocab;
      const float l = known ? logit<DT>(a, r, draft) : -INFINITY;
      const float q = known && a.draft_probs ? fmaxf(a.draft_probs[r * a.draft_row + draft], 0.f) : 1.f;
      const float ua = a.u_accept[r];
      const RowStat x = row_stat(g, r, c_t);
      bool ok = known && x.max > -INFINITY;
      if (ok)
        ok = greedy ? draft == x.best
                    : static_cast<double>(ua) * static_cast<double>(q) * x.sum < weight(l, x.max, c_t);
      if (__lane_id() == 0) {
        sh_ok[wave] = ok;
        sh_stat[wave] = x;
      }
    }
    __syncthreads();
    int k = 0;
    while (k < kWaves && t0 + k < n && sh_ok[k]) ++k;
    at = t0 + k;
    if (k < kWaves && at < n) rs = sh_stat[k];
    if (k < kWaves) break;
    __syncthreads();
  }

  // (n > 0 here has a row that draws: the last row is never accepted)
  const bool draws = n > 0 && !greedy && rs.max > -INFINITY, rejected = at + 1 < n;
  int token = n > 0 && greedy && rs.max > -INFINITY ? rs.best : -1;
  Draw d;
  if (draws) {
    d.row = r0 + at;
    d.max = rs.max;
    d.sum = rs.sum;
    d.c_t = c_t;
    d.q = rejected && a.draft_probs ? a.draft_probs + d.row * a.draft_row : nullptr;
    d.hot = rejected && !a.draft_probs ? a.tokens[d.row + 1] : -1;
  }
  if (draws && rejected) {
    // (no barrier between pieces: the next one's loads run under this one's sums)
    constexpr int kGroup = 4;
    __shared__ double sums[kGroup][kWaves];
    const int last_piece = min(first_piece + g.span, g.pieces);
    for (int s0 = first_piece; s0 < last_piece; s0 += kGroup) {
#pragma unroll
      for (int k = 0; k < kGroup; ++k) {
        if (s0 + k >= last_piece) break;
        const int64_t i0 = static_cast<int64_t>(s0 + k) * kPiece;
        float v[kPer], q[kPer];
        load_pieces<DT, kThreads, kPer>(static_cast<const typename Logits<DT>::word*>(a.logits) + d.row * a.logits_row, i0,
                                        tid, a.vocab, -INFINITY, v);
        if (d.q) {
          // (in the places that v holds)
          constexpr int kV = values_of_load<DT, kPer>();
#pragma unroll
          for (int j = 0; j < kPer; j += kV)
            load_row<QMV_F32, kV>(d.q, i0 + place<DT, kThreads, kPer>(tid, j), a.vocab, 0.f, q + j);
        }
        double w[kPer], s = 0.0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[j] = no_nan(v[j]);
        draw_weights(d, v, q, a.vocab, w, [&](int j) { return i0 + place<DT, kThreads, kPer>(tid, j); });
#pragma unroll
        for (int j = 0; j < kPer; ++j) s += w[j];
        s = wave_fold(s, add);
        if (__lane_id() == 0) sums[k][wave] = s;
      }
      __syncthreads();
      if (tid < min(kGroup, last_piece - s0)) {
        double s = 0.0;
#pragma unroll
        for (int k = 0; k < kWaves; ++k) s += sums[tid][k];
        __hip_atomic_store(g.part + static_cast<int64_t>(b) * g.pieces + s0 + tid, s, __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
      }
      __syncthreads();
    }
    // The last workgroup of the sequence to leave its sums draws the token.
    __shared__ int sh_last;
    if (tid == 0) {
      // Only the parts, which are atomics of the same scope, are passed on:
      // they have to be done before the count (this wave stored them), and no
      // cache to be written back.
      __asm__ __volatile__("s_waitcnt vmcnt(0)" ::: "memory");
      sh_last = __hip_atomic_fetch_add(g.done + b, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1 ==
                gridDim.x;
    }
    __syncthreads();
    if (!sh_last) return;
    token = find_token<DT>(g, b, d, u, false);
  } else if (first_piece != 0) {
    return;
  } else if (draws) {
    token = find_token<DT>(g, b, d, u, true);
  }
  if (tid == 0) a.accepted[b] = n > 0 ? at : 0;
  for (int r = r0 + tid; r < end; r += kThreads)
    a.out_tokens[r] = r < r0 + at ? a.tokens[r + 1] : r == r0 + at ? token : -1;
}

static int pieces_of(const qmv_verify_args& a) { return static_cast<int>((a.vocab + kPiece - 1) / kPiece); }
static size_t up256(size_t n) { return (n + 255) / 256 * 256; }

size_t verify_workspace(const qmv_verify_args& a) {
  return up256(a.rows * static_cast<size_t>(pieces_of(a)) * sizeof(PieceStat)) +
         up256(a.nseq * static_cast<size_t>(pieces_of(a)) * sizeof(double)) + up256(a.nseq * 4);
}

template <int DT>
static hipError_t verify_typed(const VerifyArgs& g, hipStream_t s) {
  const unsigned rows = static_cast<unsigned>(std::max<int64_t>(1, g.a.rows));
  hipLaunchKernelGGL(verify_rows_kernel<DT>, dim3((g.pieces + kRowThreads / 64 - 1) / (kRowThreads / 64), rows),
                     dim3(kRowThreads), 0, s, g);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(verify_draw_kernel<DT>, dim3((g.pieces + g.span - 1) / g.span, g.a.nseq), dim3(kThreads), 0, s, g);
  return hipGetLastError();
}

hipError_t verify(const qmv_verify_args& a, void* ws, hipStream_t s) {
  VerifyArgs g;
  g.a = a;
  g.pieces = pieces_of(a);
  // about two workgroups a compute unit
  g.span = static_cast<int>(std::min<int64_t>(g.pieces, (static_cast<int64_t>(g.pieces) * a.nseq + 511) / 512));
  uint8_t* p = static_cast<uint8_t*>(ws);
  g.stat = reinterpret_cast<PieceStat*>(p);
  p += up256(static_cast<size_t>(a.rows) * g.pieces * sizeof(PieceStat));
  g.part = reinterpret_cast<double*>(p);
  p += up256(static_cast<size_t>(a.nseq) * g.pieces * sizeof(double));
  g.done = reinterpret_cast<uint32_t*>(p);
  switch (a.logits_dtype) {
    case QMV_F32: return verify_typed<QMV_F32>(g, s);
    case QMV_F16: return verify_typed<QMV_F16>(g, s);
    default: return verify_typed<QMV_BF16>(g, s);
  }
}

}  // namespace qmv
