// Verification of drafted tokens by rejection sampling (qmv_verify):
//   p = softmax(logits / T); draft x accepted where u q(x) < p(x); the first
//   row that is not accepted draws from max(p - q, 0), all accepted from p.
//
// Two launches.  The first cuts every row of logits into slices of
// kSlice and leaves each slice's maximum, its first place and the sum of
// e^((l - maximum) / T).  In the second, one workgroup per sequence and slice:
// every one of them settles, from those sums, which drafts are accepted, adds
// up its slice of the row that draws, and the last of a sequence to finish
// finds the token in the slice that holds it.
//
// Exponentials and sums are in 64 bits.  A draw compares a running sum of up
// to 2^24 probabilities with u times their total; in 32 bits their errors
// would move about one draw in a hundred over 152064 flat probabilities to a
// neighbouring token.  The 64-bit exponentials, about twenty instructions
// each, run beside the reads of the logits, which bound the first launch:
// PERF_ROWS
#include <algorithm>

#include "device_util.h"
#include "launch.h"

namespace qmv {

constexpr int kSlice = 8192, kThreads = 256, kPer = kSlice / kThreads;

struct SliceStat {
  double sum;   // of e^((l - max) / T); of the infinities' ones where max is +inf
  float max;
  int best;     // the first place of max
};

struct VerifyArgs {
  qmv_verify_args a;
  int slices;
  SliceStat* stat;   // [row][slice]
  double* part;      // [sequence][slice]: the drawing row's weights
  uint32_t* done;    // [sequence]: workgroups that have left their part
};

// e^x for x <= 0, within 1e-14 of itself: 2^n times the Taylor polynomial of
// degree 11 of e^r, |r| <= ln 2 / 2 (its next term is 7e-15).
__device__ __forceinline__ double exp_neg(double x) {
  x = fmax(x, -800.0);  // (e^-800 is 0; -inf and NaN too)
  const double n = __builtin_rint(x * 1.4426950408889634);
  double r = fma(n, -0.693147180369123816, x);  // ln 2 in two parts, the first with trailing zeros
  r = fma(n, -1.90821492927058770e-10, r);
  double p = 1.0 / 39916800;
  p = fma(p, r, 1.0 / 3628800);
  p = fma(p, r, 1.0 / 362880);
  p = fma(p, r, 1.0 / 40320);
  p = fma(p, r, 1.0 / 5040);
  p = fma(p, r, 1.0 / 720);
  p = fma(p, r, 1.0 / 120);
  p = fma(p, r, 1.0 / 24);
  p = fma(p, r, 1.0 / 6);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  return __builtin_amdgcn_ldexp(p, static_cast<int>(n));
}

// e^((l - m) / T), the weight of a logit against the maximum m; a maximum of
// +inf shares everything among the infinities.
__device__ __forceinline__ double weight(float l, float m, double inv_t) {
  if (m == INFINITY) return l == INFINITY ? 1.0 : 0.0;
  return exp_neg((static_cast<double>(l) - static_cast<double>(m)) * inv_t);
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

// One logit, NaN as -inf.
template <int DT>
__device__ __forceinline__ float logit(const qmv_verify_args& a, int64_t row, int64_t i) {
  const typename Logits<DT>::word w = static_cast<const typename Logits<DT>::word*>(a.logits)[row * a.logits_row + i];
  const uint32_t v = w;
  return fmaxf(Logits<DT>::get(&v, 0), -INFINITY);
}

// N consecutive values from place i0 of a row of n, at any alignment of its
// type; places from n on give `past`.
template <int DT, int N>
__device__ __forceinline__ void load_row(const void* row, int64_t i0, int64_t n, float past, float* v) {
  typedef typename Logits<DT>::word word;
  constexpr int kV = 16 / sizeof(word);
#pragma unroll
  for (int k = 0; k < N; k += kV) {
    if (i0 + k + kV <= n) {
      const uint4 w = ld16_any(reinterpret_cast<const uint8_t*>(static_cast<const word*>(row) + i0 + k));
      const uint32_t x[4] = {w.x, w.y, w.z, w.w};
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

// The place of value j of thread t in a slice read 16 bytes a thread at a time.
template <int DT>
__device__ __forceinline__ int place(int t, int j) {
  constexpr int kV = 16 / static_cast<int>(sizeof(typename Logits<DT>::word));
  return (j / kV) * kThreads * kV + t * kV + j % kV;
}
template <int DT>
__device__ __forceinline__ void load_slice(const void* row, int64_t s0, int64_t n, float past, float* v) {
  constexpr int kV = 16 / static_cast<int>(sizeof(typename Logits<DT>::word));
#pragma unroll
  for (int k = 0; k < kPer; k += kV) load_row<DT, kV>(row, s0 + place<DT>(threadIdx.x, k), n, past, v + k);
}

template <class T, class F>
__device__ __forceinline__ T wave_fold(T v, F&& f) {
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) v = f(v, __shfl_xor(v, k));
  return v;
}
__device__ __forceinline__ double add(double x, double y) { return x + y; }

// The sum of v over the workgroup, to every thread, in a fixed order.
__device__ __forceinline__ double block_sum(double v, double* lds) {
  v = wave_fold(v, add);
  if (__lane_id() == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = (lds[0] + lds[1]) + (lds[2] + lds[3]);
  __syncthreads();
  return v;
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
__global__ void __launch_bounds__(kThreads) verify_rows_kernel(const VerifyArgs g) {
  const qmv_verify_args& a = g.a;
  const int row = blockIdx.y, slice = blockIdx.x, tid = threadIdx.x;
  const int64_t s0 = static_cast<int64_t>(slice) * kSlice;
  if (slice == 0 && row == 0)
    for (int b = tid; b < a.nseq; b += kThreads) g.done[b] = 0;
  if (row >= a.rows) return;  // (a launch without rows only clears the counts)
  float v[kPer];
  load_slice<DT>(static_cast<const typename Logits<DT>::word*>(a.logits) + row * a.logits_row, s0, a.vocab, -INFINITY, v);
  const int seq = sequence_of(a, row);
  if (seq < 0) {
    if (slice == 0 && tid == 0) a.out_tokens[row] = -1;
    return;
  }
  const float t = temperature_of(a, seq);
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < kPer; ++j) m = fmaxf(m, v[j]);  // (NaN stays out)
  __shared__ float mx[4];
  __shared__ int ix[4];
  __shared__ double sums[4];
  m = wave_fold(m, [](float x, float y) { return fmaxf(x, y); });
  if (__lane_id() == 0) mx[tid >> 6] = m;
  __syncthreads();
  m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
  int best = INT32_MAX;
#pragma unroll
  for (int j = kPer - 1; j >= 0; --j) best = v[j] == m ? place<DT>(tid, j) : best;
  best = wave_fold(best, [](int x, int y) { return min(x, y); });
  if (__lane_id() == 0) ix[tid >> 6] = best;
  double s = 0.0;
  if (t > 0.f && m > -INFINITY) {
    const double inv_t = 1.0 / static_cast<double>(t);
    double s2[2] = {0.0, 0.0};
#pragma unroll 4
    for (int j = 0; j < kPer; ++j) s2[j & 1] += weight(fmaxf(v[j], -INFINITY), m, inv_t);
    s = s2[0] + s2[1];
  }
  s = block_sum(s, sums);
  if (tid == 0)
    g.stat[static_cast<int64_t>(row) * g.slices + slice] =
        SliceStat{s, m, static_cast<int>(s0) + min(min(ix[0], ix[1]), min(ix[2], ix[3]))};
}

// A row's maximum, its first place and its sum, from its slices' (by a wave).
struct RowStat {
  float max;
  int best;
  double sum;
};
__device__ __forceinline__ RowStat row_stat(const VerifyArgs& g, int row, double inv_t) {
  const SliceStat* st = g.stat + static_cast<int64_t>(row) * g.slices;
  const int lane = __lane_id();
  float m = -INFINITY;
  for (int s = lane; s < g.slices; s += 64) m = fmaxf(m, st[s].max);
  m = wave_fold(m, [](float x, float y) { return fmaxf(x, y); });
  int best = INT32_MAX;
  double sum = 0.0;
  for (int s = lane; s < g.slices; s += 64) {
    const SliceStat x = st[s];
    if (x.max == m) best = min(best, x.best);
    sum += x.sum * weight(x.max, m, inv_t);
  }
  best = wave_fold(best, [](int x, int y) { return min(x, y); });
  return RowStat{m, best, wave_fold(sum, add)};
}

// A drawing row: the weights max(p - q, 0) S, S the row's sum, so that
// nothing is divided (q is the draft's probabilities, one at x, or nothing).
struct Draw {
  int64_t row;
  float max;
  double sum, inv_t;
  const float* q;  // NULL: one at `hot` (-1: nothing)
  int hot;
};
__device__ __forceinline__ double draw_weight(const Draw& d, float l, float q, int64_t i) {
  const double w = weight(l, d.max, d.inv_t);
  const double take = d.q ? (q > 0.f ? static_cast<double>(q) * d.sum : 0.0) : i == d.hot ? d.sum : 0.0;
  return w > take ? w - take : 0.0;
}

// Inclusive running sum over the wave's lanes.
__device__ __forceinline__ double wave_scan(double v, int lane) {
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) {
    const double o = __shfl_up(v, k);
    v = lane >= k ? v + o : v;
  }
  return v;
}

// The token: the first whose running sum passes u times the total (by the
// whole workgroup).  plain: p itself, from the slices' sums.
template <int DT>
__device__ __forceinline__ int find_token(const VerifyArgs& g, int b, const Draw& d0, float u) {
  const qmv_verify_args& a = g.a;
  const int tid = threadIdx.x, lane = __lane_id(), wave = tid >> 6;
  __shared__ double sh_goal;
  __shared__ int sh_slice, sh_plain, sh_last[4];
  __shared__ double sh_sum[4];
  Draw d = d0;
  if (wave == 0) {
    bool plain = false;
    double total = 0.0;
    auto part = [&](int s) {
      if (s >= g.slices) return 0.0;
      if (!plain) return __hip_atomic_load(g.part + static_cast<int64_t>(b) * g.slices + s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      const SliceStat st = g.stat[d.row * g.slices + s];
      return st.sum * weight(st.max, d.max, d.inv_t);
    };
    for (;;) {
      total = 0.0;
      for (int s0 = 0; s0 < g.slices; s0 += 64) total += wave_fold(part(s0 + lane), add);
      if (total > 0.0 || plain) break;
      plain = true;  // nothing is left over q: the target's own probabilities
    }
    const double goal = static_cast<double>(u) * total;
    double before = 0.0;
    int slice = -1, last = 0;
    double base = 0.0;
    for (int s0 = 0; s0 < g.slices && slice < 0; s0 += 64) {
      const double v = part(s0 + lane), c = wave_scan(v, lane) + before;
      const uint64_t some = __ballot(v > 0.0), over = __ballot(c > goal && v > 0.0);
      if (some) last = s0 + 63 - __builtin_clzll(some);
      if (over) {
        const int l = __builtin_ctzll(over);
        slice = s0 + l;
        base = __shfl(c, l) - __shfl(v, l);
      }
      before = __shfl(c, 63);
    }
    if (lane == 0) {
      sh_slice = slice >= 0 ? slice : last;  // (rounding: the last slice of any weight, to its end)
      sh_goal = slice >= 0 ? goal - base : INFINITY;
      sh_plain = plain;
    }
  }
  __syncthreads();
  if (sh_plain) {
    d.q = nullptr;
    d.hot = -1;
  }
  // contiguous places to a thread
  const int64_t i0 = static_cast<int64_t>(sh_slice) * kSlice + tid * kPer;
  const void* row = static_cast<const typename Logits<DT>::word*>(a.logits) + d.row * a.logits_row;
  float v[kPer], q[kPer];
  load_row<DT, kPer>(row, i0, a.vocab, -INFINITY, v);
  if (d.q) load_row<QMV_F32, kPer>(d.q, i0, a.vocab, 0.f, q);
  double w[kPer], s = 0.0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    w[j] = i0 + j < a.vocab ? draw_weight(d, fmaxf(v[j], -INFINITY), d.q ? q[j] : 0.f, i0 + j) : 0.0;
    s += w[j];
  }
  double c = wave_scan(s, lane);
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
  __shared__ int sh_first[4];
  if (lane == 0) {
    sh_first[wave] = first;
    sh_last[wave] = last;
  }
  __syncthreads();
  first = min(min(sh_first[0], sh_first[1]), min(sh_first[2], sh_first[3]));
  last = max(max(sh_last[0], sh_last[1]), max(sh_last[2], sh_last[3]));
  return first == INT32_MAX ? last : first;
}

template <int DT>
__global__ void __launch_bounds__(kThreads) verify_draw_kernel(const VerifyArgs g) {
  const qmv_verify_args& a = g.a;
  const int slice = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r0 = min(max(a.row_start[b], 0), static_cast<int>(a.rows));
  const int end = min(max(a.row_start[b + 1], r0), static_cast<int>(a.rows));
  const int n = min(end - r0, a.max_rows);
  const float t = temperature_of(a, b), u = a.u_sample[b];
  const bool greedy = t == 0.f;
  const double inv_t = greedy ? 0.0 : 1.0 / static_cast<double>(t);

  // The first row whose draft is not accepted, four rows at a time.
  __shared__ int sh_ok[4];
  __shared__ RowStat sh_stat[4];
  int at = 0;
  RowStat rs{-INFINITY, 0, 0.0};
  for (int t0 = 0; t0 < n; t0 += 4) {
    const int i = t0 + wave;
    bool ok = false;
    if (i < n) {
      const int r = r0 + i;
      const RowStat x = row_stat(g, r, inv_t);
      if (i + 1 < n && x.max > -INFINITY) {
        const int draft = a.tokens[r + 1];
        if (draft >= 0 && draft < a.vocab) {
          if (greedy) {
            ok = draft == x.best;
          } else {
            const double q = a.draft_probs ? static_cast<double>(fmaxf(a.draft_probs[r * a.draft_row + draft], 0.f)) : 1.0;
            ok = static_cast<double>(a.u_accept[r]) * q * x.sum < weight(logit<DT>(a, r, draft), x.max, inv_t);
          }
        }
      }
      if (__lane_id() == 0) {
        sh_ok[wave] = ok;
        sh_stat[wave] = x;
      }
    }
    __syncthreads();
    int k = 0;
    while (k < 4 && t0 + k < n && sh_ok[k]) ++k;
    at = t0 + k;
    if (k < 4 && at < n) rs = sh_stat[k];
    __syncthreads();
    if (k < 4) break;
  }

  // (n > 0 here has a row that draws: the last row is never accepted)
  const bool draws = n > 0 && !greedy && rs.max > -INFINITY;
  int token = n > 0 && greedy && rs.max > -INFINITY ? rs.best : -1;
  if (draws) {
    const bool rejected = at + 1 < n;
    Draw d;
    d.row = r0 + at;
    d.max = rs.max;
    d.sum = rs.sum;
    d.inv_t = inv_t;
    d.q = rejected && a.draft_probs ? a.draft_probs + d.row * a.draft_row : nullptr;
    d.hot = rejected && !a.draft_probs ? a.tokens[d.row + 1] : -1;
    __shared__ double sums[4];
    const int64_t s0 = static_cast<int64_t>(slice) * kSlice;
    float v[kPer], q[kPer];
    load_slice<DT>(static_cast<const typename Logits<DT>::word*>(a.logits) + d.row * a.logits_row, s0, a.vocab, -INFINITY, v);
    double s = 0.0;
    if (d.q) {
      // (in the places that v holds)
      constexpr int kV = 16 / static_cast<int>(sizeof(typename Logits<DT>::word));
#pragma unroll
      for (int k = 0; k < kPer; k += kV) load_row<QMV_F32, kV>(d.q, s0 + place<DT>(tid, k), a.vocab, 0.f, q + k);
    }
#pragma unroll 4
    for (int j = 0; j < kPer; ++j) {
      const int64_t i = s0 + place<DT>(tid, j);
      s += i < a.vocab ? draw_weight(d, fmaxf(v[j], -INFINITY), d.q ? q[j] : 0.f, i) : 0.0;
    }
    s = block_sum(s, sums);
    // The last workgroup of the sequence to leave its sum draws the token.
    __shared__ int sh_last;
    if (tid == 0) {
      __hip_atomic_store(g.part + static_cast<int64_t>(b) * g.slices + slice, s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      sh_last = __hip_atomic_fetch_add(g.done + b, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) + 1 ==
                static_cast<uint32_t>(g.slices);
    }
    __syncthreads();
    if (!sh_last) return;
    token = find_token<DT>(g, b, d, u);
  } else if (slice != 0) {
    return;
  }
  if (tid == 0) a.accepted[b] = n > 0 ? at : 0;
  for (int r = r0 + tid; r < end; r += kThreads)
    a.out_tokens[r] = r < r0 + at ? a.tokens[r + 1] : r == r0 + at ? token : -1;
}

static int slices_of(const qmv_verify_args& a) { return static_cast<int>((a.vocab + kSlice - 1) / kSlice); }
static size_t up256(size_t n) { return (n + 255) / 256 * 256; }

size_t verify_workspace(const qmv_verify_args& a) {
  const size_t slices = slices_of(a);
  return up256(a.rows * slices * sizeof(SliceStat)) + up256(a.nseq * slices * sizeof(double)) + up256(a.nseq * 4);
}

template <int DT>
static hipError_t verify_typed(const VerifyArgs& g, hipStream_t s) {
  const unsigned rows = static_cast<unsigned>(std::max<int64_t>(1, g.a.rows));
  hipLaunchKernelGGL(verify_rows_kernel<DT>, dim3(g.slices, rows), dim3(kThreads), 0, s, g);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(verify_draw_kernel<DT>, dim3(g.slices, g.a.nseq), dim3(kThreads), 0, s, g);
  return hipGetLastError();
}

hipError_t verify(const qmv_verify_args& a, void* ws, hipStream_t s) {
  VerifyArgs g;
  g.a = a;
  g.slices = slices_of(a);
  uint8_t* p = static_cast<uint8_t*>(ws);
  g.stat = reinterpret_cast<SliceStat*>(p);
  p += up256(static_cast<size_t>(a.rows) * g.slices * sizeof(SliceStat));
  g.part = reinterpret_cast<double*>(p);
  p += up256(static_cast<size_t>(a.nseq) * g.slices * sizeof(double));
  g.done = reinterpret_cast<uint32_t*>(p);
  switch (a.logits_dtype) {
    case QMV_F32: return verify_typed<QMV_F32>(g, s);
    case QMV_F16: return verify_typed<QMV_F16>(g, s);
    default: return verify_typed<QMV_BF16>(g, s);
  }
}

}  // namespace qmv
