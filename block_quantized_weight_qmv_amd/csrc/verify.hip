// Verification of drafted tokens: one workgroup per sequence, row after row.
#include "device_util.h"
#include "launch.h"

namespace qmv {

struct VerifyArgs {
  qmv_verify_args a;
};

template <int DT>
__device__ __forceinline__ double logit_at(const qmv_verify_args& a, int row, int64_t i) {
  const int64_t k = row * a.logits_row + i;
  float v;
  if (DT == QMV_F32) v = static_cast<const float*>(a.logits)[k];
  else if (DT == QMV_F16) v = f16_to_f32(static_cast<const uint16_t*>(a.logits)[k]);
  else v = bf16_to_f32(static_cast<const uint16_t*>(a.logits)[k]);
  return v != v ? -INFINITY : v;
}

template <int DT>
__global__ void __launch_bounds__(1024) verify_kernel(const qmv_verify_args a) {
  const int b = blockIdx.x, tid = threadIdx.x, V = static_cast<int>(a.vocab);
  const int r0 = min(max(a.row_start[b], 0), static_cast<int>(a.rows));
  const int r1 = min(min(max(a.row_start[b + 1], r0), static_cast<int>(a.rows)), r0 + a.max_rows);
  __shared__ double sh[1024];
  __shared__ float mx[1024];
  __shared__ int ix[1024];
  float t = a.temperature ? a.temperature[b] : 1.f;
  const bool greedy = !(t > 0.f);
  int r = r0, token = -1;
  for (; r < r1; ++r) {
    float m = -INFINITY;
    int best = 0;
    for (int i = tid; i < V; i += 1024) {
      const float v = static_cast<float>(logit_at<DT>(a, r, i));
      if (v > m) m = v, best = i;
    }
    mx[tid] = m; ix[tid] = best;
    __syncthreads();
    for (int k = 0; k < 1024; ++k)
      if (mx[k] > m || (mx[k] == m && ix[k] < best)) m = mx[k], best = ix[k];
    __syncthreads();
    const bool last = r + 1 == r1;
    const int x = last ? -1 : a.tokens[r + 1];
    const bool known = x >= 0 && x < V;
    if (m == -INFINITY) break;
    auto weight = [&](int i) {
      const double v = logit_at<DT>(a, r, i);
      if (greedy) return i == best ? 1.0 : 0.0;
      if (m == INFINITY) return v == INFINITY ? 1.0 : 0.0;
      return exp((v - m) / t);
    };
    double s = 0;
    for (int i = tid; i < V; i += 1024) s += weight(i);
    sh[tid] = s;
    __syncthreads();
    double total = 0;
    for (int k = 0; k < 1024; ++k) total += sh[k];
    __syncthreads();
    const bool hot = greedy || !a.draft_probs;
    if (!last && known) {
      const double q = hot ? 1.0 : fmax(0.0, static_cast<double>(a.draft_probs[r * a.draft_row + x]));
      const bool good = greedy ? x == best : static_cast<double>(a.u_accept[r]) * q < weight(x) / total;
      if (good) {
        if (tid == 0) a.out_tokens[r] = x;
        continue;
      }
    }
    // contiguous chunks keep the order of the sum the order of the tokens
    const int per = (V + 1023) / 1024, i0 = min(tid * per, V), i1 = min(i0 + per, V);
    auto residual = [&](int i, bool plain) {
      const double p = weight(i) / total;
      if (last || plain) return p;
      const double q = hot ? (i == x ? 1.0 : 0.0) : a.draft_probs[r * a.draft_row + i];
      return q > 0 ? (p > q ? p - q : 0.0) : p;
    };
    bool plain = false;
    double sum;
    for (;;) {
      s = 0;
      for (int i = i0; i < i1; ++i) s += residual(i, plain);
      sh[tid] = s;
      __syncthreads();
      sum = 0;
      for (int k = 0; k < 1024; ++k) sum += sh[k];
      if (sum > 0 || plain) break;
      plain = true;
      __syncthreads();
    }
    const double goal = a.u_sample[b] * sum;
    double before = 0;
    for (int k = 0; k < tid; ++k) before += sh[k];
    int mine = V, nonzero = -1;
    for (int i = i0; i < i1; ++i) {
      const double w = residual(i, plain);
      before += w;
      if (w > 0) {
        nonzero = i;
        if (before > goal && mine == V) mine = i;
      }
    }
    ix[tid] = mine;
    mx[tid] = nonzero;
    __syncthreads();
    token = V;
    for (int k = 0; k < 1024; ++k) token = min(token, ix[k]);
    if (token == V)
      for (int k = 0; k < 1024; ++k) if (mx[k] >= 0) token = static_cast<int>(mx[k]);
    break;
  }
  if (b == 0) {  // rows outside every sequence
    const int64_t first = r0, end = max(min(static_cast<int64_t>(a.row_start[a.nseq]), a.rows), int64_t{0});
    for (int64_t k = tid; k < a.rows; k += 1024)
      if (k < first || k >= end) a.out_tokens[k] = -1;
  }
  if (tid == 0) {
    a.accepted[b] = min(r, max(r1 - 1, r0)) - r0;
    const int end = min(max(a.row_start[b + 1], r0), static_cast<int>(a.rows));
    for (int k = r; k < end; ++k) a.out_tokens[k] = k == r && r < r1 ? token : -1;
  }
}

size_t verify_workspace(const qmv_verify_args&) { return 0; }

hipError_t verify(const qmv_verify_args& a, void*, hipStream_t s) {
  const dim3 g(a.nseq);
  switch (a.logits_dtype) {
    case QMV_F32: hipLaunchKernelGGL(verify_kernel<QMV_F32>, g, dim3(1024), 0, s, a); break;
    case QMV_F16: hipLaunchKernelGGL(verify_kernel<QMV_F16>, g, dim3(1024), 0, s, a); break;
    default: hipLaunchKernelGGL(verify_kernel<QMV_BF16>, g, dim3(1024), 0, s, a); break;
  }
  return hipGetLastError();
}

}  // namespace qmv
