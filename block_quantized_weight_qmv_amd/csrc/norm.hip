// Norms around a block of a model, with the residual that joins them:
//   s = residual + scale * gate . post(block),   y = pre(s)
// norm(x) = (x - mean) / sqrt(mean((x - mean)^2) + eps) * weight + bias, with
// mean = 0 for RMS norms.
//
// Bound: HBM (each number is read and written once).  A row lives in the
// registers of its threads between the sums, so that the block's norm, the
// residual's sum and the next block's norm are one pass; sums are fp32, those
// of a layer norm around the row's mean.  Rows of up to 2048 numbers belong to
// one wave (no barrier, four rows to a workgroup), longer ones to a workgroup.
#include "launch.h"
#include "mx4.h"

namespace qmv {

struct NormArgs {
  const void *residual, *block, *gate, *pre_w, *pre_b, *post_w, *post_b;
  void *sum, *y;
  int64_t residual_row, block_row, gate_row, sum_row, y_row;
  int rows, cols, pre, post, y_dtype;
  float eps, scale;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(_Float16 v) { return static_cast<float>(v); }
__device__ __forceinline__ float to_f32(bf16_t v) { return bf16_to_f32(v.bits); }

// Numbers at(k) of a row, k = 0 .. 8 VPT: with VEC eight consecutive ones for
// each step of the row's threads (16-byte loads), else one (any alignment).
template <int VPT, bool VEC>
struct RowMap {
  int t, threads, cols;
  __device__ int at(int k) const { return VEC ? ((k >> 3) * threads + t) * 8 + (k & 7) : k * threads + t; }
  __device__ bool ok(int k) const { return at(k) < cols; }
};

// Raw numbers of a row (zero past its end), converted later, so that the loads
// of all the row's inputs are in flight together.
template <typename T, int VPT, bool VEC>
struct RawRow {
  static constexpr int kPer = 8 * static_cast<int>(sizeof(T)) / 16;
  uint4 raw[VEC ? VPT * kPer : 1];
  T one[VEC ? 1 : 8 * VPT];
  __device__ void load(const T* p, const RowMap<VPT, VEC>& m) {
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          raw[j * kPer + i] = m.ok(8 * j) ? reinterpret_cast<const uint4*>(p + m.at(8 * j))[i] : make_uint4(0, 0, 0, 0);
    } else {
#pragma unroll
      for (int k = 0; k < 8 * VPT; ++k) one[k] = m.ok(k) ? p[m.at(k)] : T{};
    }
  }
  __device__ void get(float* v) const {
    if constexpr (VEC) {
      x_to_f32<8 * VPT>(raw, v, static_cast<const T*>(nullptr));
    } else {
#pragma unroll
      for (int k = 0; k < 8 * VPT; ++k) v[k] = to_f32(one[k]);
    }
  }
};

template <int OUT, int VPT, bool VEC>
__device__ __forceinline__ void store_row(void* p, const float* v, const RowMap<VPT, VEC>& m) {
  if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (!m.ok(8 * j)) continue;
      const float* w = v + 8 * j;
      if constexpr (OUT == QMV_F32) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(p) + m.at(8 * j));
        o[0] = make_float4(w[0], w[1], w[2], w[3]);
        o[1] = make_float4(w[4], w[5], w[6], w[7]);
      } else {
        auto two = [&](int k) { return OUT == QMV_F16 ? pack_f16(w[k], w[k + 1]) : pack_bf16(w[k], w[k + 1]); };
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + m.at(8 * j)) = make_uint4(two(0), two(2), two(4), two(6));
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8 * VPT; ++k) {
      if (!m.ok(k)) continue;
      if constexpr (OUT == QMV_F32)
        static_cast<float*>(p)[m.at(k)] = v[k];
      else if constexpr (OUT == QMV_F16)
        static_cast<_Float16*>(p)[m.at(k)] = static_cast<_Float16>(v[k]);
      else
        static_cast<uint16_t*>(p)[m.at(k)] = static_cast<uint16_t>(pack_bf16(v[k], 0.f));
    }
  }
}

// The sum over a row's threads: its wave's lanes, then, where the row has a
// workgroup, the waves' sums in LDS (a slot of its own for each sum, so one
// barrier is enough).
template <bool WAVE>
__device__ __forceinline__ float row_sum(float v, float* slot) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  if constexpr (!WAVE) {
    const int waves = blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
    for (int w = 0; w < waves; ++w) v += slot[w];
  }
  return v;
}

// v = norm(v) of kind QMV_NORM_RMS or QMV_NORM_LAYER.
template <typename W, int VPT, bool VEC, bool WAVE>
__device__ __forceinline__ void norm_row(float* v, int kind, const RawRow<W, VPT, VEC>& w, const RawRow<W, VPT, VEC>& b,
                                         bool has_w, bool has_b, const RowMap<VPT, VEC>& m, float eps, float* slot) {
  constexpr int N = 8 * VPT;
  const float count = 1.0f / static_cast<float>(m.cols);
  if (kind == QMV_NORM_LAYER) {
    float a = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) a += v[k];  // zeros past the row's end
    const float mean = row_sum<WAVE>(a, slot) * count;
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = m.ok(k) ? v[k] - mean : 0.f;
  }
  float a = 0.f;
#pragma unroll
  for (int k = 0; k < N; ++k) a = fmaf(v[k], v[k], a);
  const float f = 1.0f / sqrtf(row_sum<WAVE>(a, slot + 16) * count + eps);
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] *= f;
  float u[N];
  if (has_w) {
    w.get(u);
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] *= u[k];
  }
  if (has_b) {
    b.get(u);
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += u[k];
  }
}

template <typename T, typename W, int VPT, bool VEC, bool WAVE>
__global__ void __launch_bounds__(WAVE ? 256 : 1024)
norm_kernel(const NormArgs a, int row0) {
  constexpr int N = 8 * VPT;
  __shared__ float slots[64];
  const RowMap<VPT, VEC> m{WAVE ? static_cast<int>(threadIdx.x & 63) : static_cast<int>(threadIdx.x),
                           WAVE ? 64 : static_cast<int>(blockDim.x), a.cols};
  const int64_t r = row0 + (WAVE ? static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6) : blockIdx.x);
  if (WAVE && r >= a.rows) return;
  typedef RawRow<T, VPT, VEC> Row;
  typedef RawRow<W, VPT, VEC> Weights;
  Row res, blk, gate;
  Weights pre_w, pre_b, post_w, post_b;
  res.load(static_cast<const T*>(a.residual) + r * a.residual_row, m);
  if (a.block) blk.load(static_cast<const T*>(a.block) + r * a.block_row, m);
  if (a.gate) gate.load(static_cast<const T*>(a.gate) + r * a.gate_row, m);
  if (a.post_w) post_w.load(static_cast<const W*>(a.post_w), m);
  if (a.post_b) post_b.load(static_cast<const W*>(a.post_b), m);
  if (a.pre_w) pre_w.load(static_cast<const W*>(a.pre_w), m);
  if (a.pre_b) pre_b.load(static_cast<const W*>(a.pre_b), m);
  float s[N];
  res.get(s);
  if (a.block) {
    float b[N];
    blk.get(b);
    if (a.post != QMV_NORM_NONE)
      norm_row<W, VPT, VEC, WAVE>(b, a.post, post_w, post_b, a.post_w, a.post_b, m, a.eps, slots);
    if (a.gate) {
      float g[N];
      gate.get(g);
#pragma unroll
      for (int k = 0; k < N; ++k) b[k] *= g[k];
    }
#pragma unroll
    for (int k = 0; k < N; ++k) s[k] = m.ok(k) ? fmaf(a.scale, b[k], s[k]) : 0.f;
  }
  if (a.sum) {
    constexpr int kOut = sizeof(T) == 4 ? QMV_F32 : __is_same(T, _Float16) ? QMV_F16 : QMV_BF16;
    store_row<kOut>(static_cast<T*>(a.sum) + r * a.sum_row, s, m);
  }
  if (!a.y) return;
  if (a.pre != QMV_NORM_NONE)
    norm_row<W, VPT, VEC, WAVE>(s, a.pre, pre_w, pre_b, a.pre_w, a.pre_b, m, a.eps, slots + 32);
  if (a.y_dtype == QMV_F32)
    store_row<QMV_F32>(static_cast<float*>(a.y) + r * a.y_row, s, m);
  else if (a.y_dtype == QMV_F16)
    store_row<QMV_F16>(static_cast<uint16_t*>(a.y) + r * a.y_row, s, m);
  else
    store_row<QMV_BF16>(static_cast<uint16_t*>(a.y) + r * a.y_row, s, m);
}

template <typename T, typename W, int VPT, bool VEC>
static hipError_t norm_launch(const NormArgs& a, hipStream_t s) {
  const bool wave = a.cols <= 64 * 8 * VPT;
  const int per = 8 * VPT, threads = wave ? 256 : ((a.cols + per - 1) / per + 63) / 64 * 64;
  // (a launch's work-items along x are counted in 32 bits)
  constexpr int most = 1 << 21;
  for (int r = 0; r < a.rows; r += most) {
    const int rows = a.rows - r < most ? a.rows - r : most;
    if (wave)
      hipLaunchKernelGGL((norm_kernel<T, W, VPT, VEC, true>), dim3((rows + 3) / 4), dim3(256), 0, s, a, r);
    else
      hipLaunchKernelGGL((norm_kernel<T, W, VPT, VEC, false>), dim3(rows), dim3(threads), 0, s, a, r);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Numbers to a thread: eight for rows that one wave holds so or that need no
// more than 1024 threads so, else 32.
template <typename T, typename W>
static hipError_t norm_typed(const NormArgs& a, bool vec, hipStream_t s) {
  const bool wide = a.cols > 512 && (a.cols <= 2048 || a.cols > 8192);
  if (vec) return wide ? norm_launch<T, W, 4, true>(a, s) : norm_launch<T, W, 1, true>(a, s);
  return wide ? norm_launch<T, W, 4, false>(a, s) : norm_launch<T, W, 1, false>(a, s);
}

template <typename T>
static hipError_t norm_weights(const NormArgs& a, int w_dtype, bool vec, hipStream_t s) {
  switch (w_dtype) {
    case QMV_F32: return norm_typed<T, float>(a, vec, s);
    case QMV_F16: return norm_typed<T, _Float16>(a, vec, s);
    default: return norm_typed<T, bf16_t>(a, vec, s);
  }
}

hipError_t norm(const qmv_norm_args& n, hipStream_t s) {
  NormArgs a;
  a.residual = n.residual, a.block = n.block, a.gate = n.gate;
  a.pre_w = n.pre_weight, a.pre_b = n.pre_bias, a.post_w = n.post_weight, a.post_b = n.post_bias;
  a.sum = n.sum, a.y = n.y;
  a.residual_row = n.residual_row, a.block_row = n.block_row, a.gate_row = n.gate_row;
  a.sum_row = n.sum_row, a.y_row = n.y_row;
  a.rows = static_cast<int>(n.rows), a.cols = static_cast<int>(n.cols);
  a.pre = n.pre, a.post = n.post, a.y_dtype = n.y_dtype, a.eps = n.eps, a.scale = n.scale;
  // 16-byte accesses where every row of everything starts on 16 bytes and ends
  // with a whole eight
  bool vec = n.cols % 8 == 0;
  auto check = [&](const void* p, int64_t row, int size) {
    if (p && ((reinterpret_cast<uintptr_t>(p) & 15) || (n.rows > 1 && row * size % 16))) vec = false;
  };
  const int xs = n.dtype == QMV_F32 ? 4 : 2;
  check(n.residual, n.residual_row, xs);
  check(n.block, n.block_row, xs);
  check(n.gate, n.gate_row, xs);
  check(n.sum, n.sum_row, xs);
  check(n.y, n.y_row, n.y_dtype == QMV_F32 ? 4 : 2);
  for (const void* p : {n.pre_weight, n.pre_bias, n.post_weight, n.post_bias}) check(p, 0, 0);
  switch (n.dtype) {
    case QMV_F32: return norm_weights<float>(a, n.weight_dtype, vec, s);
    case QMV_F16: return norm_weights<_Float16>(a, n.weight_dtype, vec, s);
    default: return norm_weights<bf16_t>(a, n.weight_dtype, vec, s);
  }
}

}  // namespace qmv
