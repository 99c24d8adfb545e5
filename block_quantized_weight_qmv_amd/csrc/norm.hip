// Norms around a block of a model, with the residual that joins them:
//   s = residual + scale * gate . post(block),   y = pre(s)
// norm(x) = (x - mean) / sqrt(mean((x - mean)^2) + eps) * weight + bias, with
// mean = 0 for RMS norms.
//
// Bound: HBM (each number is read and written once); a few rows take a launch and
// the latency of their loads.  A row lives in the registers of its threads between
// the sums, so that the block's norm, the residual's sum and the next block's norm
// are one pass; sums are fp32, those of a layer norm around the row's mean.  Rows of
// up to 2048 numbers belong to one wave (no barrier, four rows to a workgroup),
// longer ones to a workgroup.  A thread holds runs of eight numbers, loaded as 16
// bytes whatever the row's alignment; rows that do not end with a whole run pay a
// branch for each (bf16, both norms and the sum's store, 8 bytes a number: 16384
// rows of 3584 90 us, 5.2 TB/s; of 3590 126 us, 326 when loaded number by number;
// 65536 of 512 48 us, 5.5 TB/s).
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

// Numbers at(k) of a row, k = 0 .. 8 VPT: eight consecutive ones for each step of
// the row's threads.  WHOLE: the row is a number of whole eights.
template <int VPT, bool WHOLE>
struct RowMap {
  int t, threads, cols;
  __device__ int at(int k) const { return ((k >> 3) * threads + t) * 8 + (k & 7); }
  __device__ bool ok(int k) const { return at(k) < cols; }
};

// Sixteen bytes at any alignment of their elements.
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));

// Raw numbers of a row (zero past its end), converted later, so that the loads
// of all the row's inputs are in flight together.
template <typename T, int VPT, bool WHOLE>
struct RawRow {
  static constexpr int kPer = 8 * static_cast<int>(sizeof(T)) / 16;
  uint4 raw[VPT * kPer];
  __device__ void load(const T* p, const RowMap<VPT, WHOLE>& m) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const T* q = p + m.at(8 * j);
      const int left = m.cols - m.at(8 * j);
      if (left >= 8) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const u32x4_a2 v = reinterpret_cast<const u32x4_a2*>(q)[i];
          raw[j * kPer + i] = make_uint4(v.x, v.y, v.z, v.w);
        }
      } else if (WHOLE) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) raw[j * kPer + i] = make_uint4(0, 0, 0, 0);
      } else {  // the row's last few, by one thread
        T one[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) one[e] = e < left ? q[e] : T{};
        __builtin_memcpy(&raw[j * kPer], one, sizeof(one));
      }
    }
  }
  __device__ void get(float* v) const { x_to_f32<8 * VPT>(raw, v, static_cast<const T*>(nullptr)); }
};

template <int OUT, int VPT, bool WHOLE>
__device__ __forceinline__ void store_row(void* p, const float* v, const RowMap<VPT, WHOLE>& m) {
  constexpr int kSize = OUT == QMV_F32 ? 4 : 2, kPer = 8 * kSize / 16;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const float* w = v + 8 * j;
    uint32_t d[4 * kPer];
#pragma unroll
    for (int i = 0; i < 4 * kPer; ++i)
      d[i] = OUT == QMV_F32 ? __float_as_uint(w[i]) : OUT == QMV_F16 ? pack_f16(w[2 * i], w[2 * i + 1]) : pack_bf16(w[2 * i], w[2 * i + 1]);
    uint8_t* o = static_cast<uint8_t*>(p) + static_cast<int64_t>(m.at(8 * j)) * kSize;
    const int left = m.cols - m.at(8 * j);
    if (left >= 8) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        reinterpret_cast<u32x4_a2*>(o)[i] = u32x4_a2{d[4 * i], d[4 * i + 1], d[4 * i + 2], d[4 * i + 3]};
    } else if (!WHOLE) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e >= left) continue;
        if constexpr (OUT == QMV_F32)
          reinterpret_cast<uint32_t*>(o)[e] = d[e];
        else
          reinterpret_cast<uint16_t*>(o)[e] = static_cast<uint16_t>(d[e / 2] >> (16 * (e & 1)));
      }
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
template <typename W, int VPT, bool WHOLE, bool WAVE>
__device__ __forceinline__ void norm_row(float* v, int kind, const RawRow<W, VPT, WHOLE>& w, const RawRow<W, VPT, WHOLE>& b,
                                         bool has_w, bool has_b, const RowMap<VPT, WHOLE>& m, float eps, float* slot) {
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

template <typename T, typename W, int VPT, bool WHOLE, int MAXT, bool WAVE>
__global__ void __launch_bounds__(MAXT)
norm_kernel(const NormArgs a, int row0) {
  constexpr int N = 8 * VPT;
  __shared__ float slots[64];
  const RowMap<VPT, WHOLE> m{WAVE ? static_cast<int>(threadIdx.x & 63) : static_cast<int>(threadIdx.x),
                                  WAVE ? 64 : static_cast<int>(blockDim.x), a.cols};
  const int64_t r = row0 + (WAVE ? static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6) : blockIdx.x);
  if (WAVE && r >= a.rows) return;
  typedef RawRow<T, VPT, WHOLE> Row;
  typedef RawRow<W, VPT, WHOLE> Weights;
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
      norm_row<W, VPT, WHOLE, WAVE>(b, a.post, post_w, post_b, a.post_w, a.post_b, m, a.eps, slots);
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
    norm_row<W, VPT, WHOLE, WAVE>(s, a.pre, pre_w, pre_b, a.pre_w, a.pre_b, m, a.eps, slots + 32);
  if (a.y_dtype == QMV_F32)
    store_row<QMV_F32>(static_cast<float*>(a.y) + r * a.y_row, s, m);
  else if (a.y_dtype == QMV_F16)
    store_row<QMV_F16>(static_cast<uint16_t*>(a.y) + r * a.y_row, s, m);
  else
    store_row<QMV_BF16>(static_cast<uint16_t*>(a.y) + r * a.y_row, s, m);
}

// WAVE: a wave to a row, four rows to a workgroup; else a workgroup of up to MAXT.
template <typename T, typename W, int VPT, int MAXT, bool WAVE, bool WHOLE>
static hipError_t norm_launch(const NormArgs& a, hipStream_t s) {
  constexpr int per = 8 * VPT;
  const int threads = WAVE ? 256 : ((a.cols + per - 1) / per + 63) / 64 * 64;
  // (a launch's work-items along x are counted in 32 bits)
  constexpr int most = 1 << 21;
  for (int64_t r = 0; r < a.rows; r += most) {
    const int rows = static_cast<int>(a.rows - r < most ? a.rows - r : most);
    hipLaunchKernelGGL((norm_kernel<T, W, VPT, WHOLE, MAXT, WAVE>), dim3(WAVE ? (rows + 3) / 4 : rows), dim3(threads), 0, s,
                       a, static_cast<int>(r));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Numbers to a thread.  Eight for rows that one wave holds so, and for few longer
// rows, whose latency counts; sixteen for many rows of a workgroup (16384 rows of
// 3584 in bf16, both norms: 90 us, 108 with eight); else 32, whose workgroups of
// more than 512 threads spill registers (1024 rows of 16384 36 us, of 32768 119).
template <typename T, typename W, bool WHOLE>
static hipError_t norm_typed(const NormArgs& a, hipStream_t s) {
  if (a.cols <= 512) return norm_launch<T, W, 1, 256, true, WHOLE>(a, s);
  if (a.cols <= 2048) return norm_launch<T, W, 4, 256, true, WHOLE>(a, s);
  if (a.cols <= 8192 && a.rows < 1024) return norm_launch<T, W, 1, 1024, false, WHOLE>(a, s);
  if (a.cols <= 8192) return norm_launch<T, W, 2, 512, false, WHOLE>(a, s);
  if (a.cols <= 16384) return norm_launch<T, W, 4, 512, false, WHOLE>(a, s);
  return norm_launch<T, W, 4, 1024, false, WHOLE>(a, s);
}

template <typename T, typename W>
static hipError_t norm_whole(const NormArgs& a, hipStream_t s) {
  return a.cols % 8 ? norm_typed<T, W, false>(a, s) : norm_typed<T, W, true>(a, s);
}

template <typename T>
static hipError_t norm_weights(const NormArgs& a, int w_dtype, hipStream_t s) {
  switch (w_dtype) {
    case QMV_F32: return norm_whole<T, float>(a, s);
    case QMV_F16: return norm_whole<T, _Float16>(a, s);
    default: return norm_whole<T, bf16_t>(a, s);
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
  switch (n.dtype) {
    case QMV_F32: return norm_weights<float>(a, n.weight_dtype, s);
    case QMV_F16: return norm_weights<_Float16>(a, n.weight_dtype, s);
    default: return norm_weights<bf16_t>(a, n.weight_dtype, s);
  }
}

}  // namespace qmv
