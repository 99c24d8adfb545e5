// Attention of a step's rows over a prefix that the whole batch shares and
// their own sequences' paged suffixes:
//   o = sum_j p_j v_j / sum_j p_j,  p_j = e^(scale q.k_j - m),  m = max_j scale q.k_j,
// over the prefix tokens and the suffix tokens that the row sees.
#include "device_util.h"
#include "launch.h"

namespace qmv {

__device__ __forceinline__ float attn_elem(const uint16_t* p, int bf16) {
  return bf16 ? bf16_to_f32(*p) : f16_to_f32(*p);
}

// A row's place: its sequence (-1: none), index among the sequence's rows,
// the sequence's rows and suffix tokens.
struct RowPlace {
  int seq, i, n, len;
};

__device__ __forceinline__ RowPlace place_of(const qmv_attn_args& a, int row) {
  RowPlace p{-1, 0, 0, 0};
  int lo = 0, hi = a.nseq;  // the last sequence that starts at or before the row
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (mid < a.nseq + 0 && a.row_start[mid] <= row) lo = mid; else hi = mid - 1;
  }
  const int s = a.row_start[lo], e = a.row_start[lo + 1];
  if (row < s || row >= e) return p;
  p.seq = lo;
  p.i = row - s;
  p.n = e - s;
  p.len = a.max_suffix > 0 ? min(max(a.suffix_len[lo], 0), static_cast<int>(a.max_suffix)) : 0;
  return p;
}

// One workgroup per (row, query head), one thread per key of a chunk of 256.
__global__ void __launch_bounds__(256) attn_kernel(const qmv_attn_args a) {
  const int row = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  const int hk = h / (a.heads / a.kv_heads), D = a.head_dim, bf = a.dtype == QMV_BF16;
  const RowPlace pl = place_of(a, row);
  __shared__ float q[256], p[256], red[4];
  __shared__ int64_t at[256];
  __shared__ int from_pool[256];
  uint16_t* out = static_cast<uint16_t*>(a.out) + row * a.out_row + h * a.out_head;
  if (tid < D) q[tid] = attn_elem(static_cast<const uint16_t*>(a.q) + row * a.q_row + h * a.q_head + tid, bf) * a.scale;
  const uint64_t mask = a.tree_mask ? a.tree_mask[row] : 0;
  const int P = static_cast<int>(a.prefix_len), total = P + pl.len;
  float m = -INFINITY, l = 0.f, o = 0.f;
  __syncthreads();
  for (int j0 = 0; j0 < total; j0 += 256) {
    const int j = j0 + tid;
    float s = -INFINITY;
    int64_t off = -1;
    int pool = 0;
    if (j < total) {
      const int jj = j < P ? j : j - P;
      bool seen = true;
      const int32_t* table = j < P ? a.prefix_pages : a.block_table + static_cast<int64_t>(pl.seq) * a.table_stride;
      if (j >= P) {
        const int slot = jj - (pl.len - pl.n);
        seen = slot < 0 || (a.tree_mask ? slot < 64 && ((mask >> slot) & 1) : slot <= pl.i);
      }
      if (table) {
        pool = 1;
        const int page = table[jj / a.page_size];
        if (page < 0 || page >= a.num_pages) seen = false;
        off = page * a.page_stride + (jj % a.page_size) * a.page_row + hk * a.page_head;
      } else {
        off = jj * a.prefix_row + hk * a.prefix_head;
      }
      if (!seen) off = -1;
    }
    if (off >= 0) {
      const uint16_t* k = static_cast<const uint16_t*>(pool ? a.k_pages : a.k_prefix) + off;
      s = 0.f;
      for (int d = 0; d < D; ++d) s = fmaf(q[d], attn_elem(k + d, bf), s);
    }
    p[tid] = s;
    at[tid] = off;
    from_pool[tid] = pool;
    __syncthreads();
    float mx = m;
    for (int k = 0; k < 256; ++k) mx = fmaxf(mx, at[k] >= 0 ? p[k] : -INFINITY);
    const float base = mx == -INFINITY ? 0.f : mx;
    const float f = m == -INFINITY ? 0.f : expf(m - base);
    l *= f;
    o *= f;
    m = mx;
    for (int k = 0; k < 256; ++k) {
      if (at[k] < 0) continue;
      const float w = expf(p[k] - base);
      l += w;
      if (tid < D) o = fmaf(w, attn_elem(static_cast<const uint16_t*>(from_pool[k] ? a.v_pages : a.v_prefix) + at[k] + tid, bf), o);
    }
    __syncthreads();
  }
  const bool past = pl.seq >= 0 && pl.i >= a.max_rows;
  if (tid < D) {
    const float v = past ? __builtin_nanf("") : l == 0.f ? 0.f : o / l;
    out[tid] = bf ? __builtin_bit_cast(uint16_t, static_cast<__bf16>(v))
                  : __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
  }
  if (a.lse && tid == 0) a.lse[static_cast<size_t>(row) * a.heads + h] = past ? __builtin_nanf("") : l == 0.f ? -INFINITY : m + logf(l);
}

size_t attn_workspace(const qmv_attn_args&) { return 0; }

hipError_t attn(const qmv_attn_args& a, void*, hipStream_t s) {
  hipLaunchKernelGGL(attn_kernel, dim3(static_cast<unsigned>(a.rows), a.heads), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace qmv
