// Losses through a stored vocabulary projection, z = W_hat h / T, with the
// logits never kept: the statistics of the softmax and the few logits that the
// targets name come from the product's own tiles (launch_head_partials), and
// the gradient takes the softmax one piece of the vocabulary at a time.
//
//   labels        loss = lse(z) - z_y
//   distillation  p = softmax(teacher / T) over the K entries given,
//                 loss = sum_k p_k (log p_k - z_k + lse(z))
//   gradient      dz_v = softmax(z)_v - sum_{k: index_k = v} p_k
//
// An entry takes part if its index lies in [0, rows) and its teacher logit is
// not -inf; a token without entries has loss and gradient 0.
#include "common.h"

namespace gptq {
namespace {

__device__ inline bool takes_part(const HeadTargets& tg, int64_t t, int k, int64_t rows) {
  const int v = tg.index[t * tg.top + k];
  if (v < 0 || v >= rows) return false;
  return tg.logits == nullptr || tg.logits[t * tg.top + k] != -INFINITY;
}

__device__ inline float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}

__device__ inline float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// log of the teacher's normalisation over the entries that take part: the
// entry's log probability is logit * inv_t - this (labels: 0).  *any: whether
// one does.
__device__ inline float teacher_lse(const HeadTargets& tg, int64_t t, int64_t rows, bool* any) {
  const int lane = threadIdx.x & 63;
  bool mine = false;
  float top = -INFINITY;
  for (int k = lane; k < tg.top; k += 64)
    if (takes_part(tg, t, k, rows)) {
      mine = true;
      if (tg.logits != nullptr) top = fmaxf(top, tg.logits[t * tg.top + k] * tg.inv_t);
    }
  *any = __ballot(mine) != 0;
  if (tg.logits == nullptr || !*any) return 0.f;
  top = wave_max(top);
  float sum = 0.f;
  for (int k = lane; k < tg.top; k += 64)
    if (takes_part(tg, t, k, rows)) sum += __expf(tg.logits[t * tg.top + k] * tg.inv_t - top);
  return top + __logf(wave_sum(sum));
}

__device__ inline float log_p(const HeadTargets& tg, int64_t t, int k, float tlse) {
  return tg.logits == nullptr ? 0.f : tg.logits[t * tg.top + k] * tg.inv_t - tlse;
}

// One token per wave.
__global__ __launch_bounds__(256) void head_finish_kernel(int64_t m, int64_t rows, HeadTargets tg,
                                                          const float2* __restrict__ part,
                                                          int64_t tiles, float* __restrict__ loss,
                                                          float* __restrict__ lse_out,
                                                          float* __restrict__ zk) {
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (t >= m) return;
  float top = -INFINITY;
  for (int64_t i = lane; i < tiles; i += 64) top = fmaxf(top, part[i * m + t].x);
  top = wave_max(top);
  const float base = top == -INFINITY ? 0.f : top;
  float sum = 0.f;
  for (int64_t i = lane; i < tiles; i += 64) {
    const float2 p = part[i * m + t];
    sum += p.x == -INFINITY ? p.y : p.y * __expf(p.x - base);
  }
  const float lse = base + __logf(wave_sum(sum));
  bool any;
  const float tlse = teacher_lse(tg, t, rows, &any);
  float l = 0.f;
  for (int k = lane; k < tg.top; k += 64) {
    if (takes_part(tg, t, k, rows)) {
      const float lp = log_p(tg, t, k, tlse);
      l += __expf(lp) * (lp - zk[t * tg.top + k] + lse);
    } else {
      zk[t * tg.top + k] = 0.f;
    }
  }
  l = wave_sum(l);
  if (lane == 0) {
    loss[t] = any ? l : 0.f;
    lse_out[t] = lse;
  }
}

__global__ __launch_bounds__(256) void head_rows_kernel(HeadTargets tg, int64_t m, int64_t rows,
                                                        const float* __restrict__ lse,
                                                        const float* __restrict__ dloss,
                                                        float* __restrict__ lse_eff,
                                                        float* __restrict__ gscale) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= m) return;
  bool any = false;
  for (int k = 0; k < tg.top && !any; ++k) any = takes_part(tg, t, k, rows);
  lse_eff[t] = any ? lse[t] : INFINITY;
  gscale[t] = any ? dloss[t] * tg.inv_t : 0.f;
}

// An index named by several entries gets their sum from each of them (the
// same value, written more than once).
__global__ __launch_bounds__(64) void head_scatter_kernel(HeadTargets tg, int64_t rows, int64_t v0,
                                                          int64_t width,
                                                          const float* __restrict__ zk,
                                                          const float* __restrict__ lse,
                                                          _Float16* __restrict__ P, int64_t ldp) {
  __shared__ int idx[kMaxTop];
  __shared__ float prob[kMaxTop];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x;
  bool any;
  const float tlse = teacher_lse(tg, t, rows, &any);
  for (int k = lane; k < tg.top; k += 64) {
    const bool in = takes_part(tg, t, k, rows);
    idx[k] = in ? tg.index[t * tg.top + k] : -1;
    prob[k] = in ? __expf(log_p(tg, t, k, tlse)) : 0.f;
  }
  __syncthreads();
  for (int k = lane; k < tg.top; k += 64) {
    const int v = idx[k];
    if (v < v0 || v >= v0 + width) continue;  // v0 >= 0: not an entry that is out
    float p = 0.f;
    for (int o = 0; o < tg.top; ++o) p += idx[o] == v ? prob[o] : 0.f;
    P[t * ldp + v - v0] = (_Float16)(__expf(zk[t * tg.top + k] - lse[t]) - p);
  }
}

}  // namespace

hipError_t launch_head_finish(int64_t m, int64_t rows, const HeadTargets& tg, const float2* part,
                              int64_t tiles, float* loss, float* lse, float* zk, hipStream_t s) {
  hipLaunchKernelGGL(head_finish_kernel, dim3((unsigned)ceil_div(m, 4)), dim3(256), 0, s, m, rows,
                     tg, part, tiles, loss, lse, zk);
  return hipGetLastError();
}

hipError_t launch_head_rows(const HeadTargets& tg, int64_t m, int64_t rows, const float* lse,
                            const float* dloss, float* lse_eff, float* gscale, hipStream_t s) {
  hipLaunchKernelGGL(head_rows_kernel, dim3((unsigned)ceil_div(m, 256)), dim3(256), 0, s, tg, m,
                     rows, lse, dloss, lse_eff, gscale);
  return hipGetLastError();
}

hipError_t launch_head_scatter(const HeadTargets& tg, int64_t m, int64_t rows, int64_t v0,
                               int64_t width, const float* zk, const float* lse, _Float16* P,
                               int64_t ldp, hipStream_t s) {
  hipLaunchKernelGGL(head_scatter_kernel, dim3((unsigned)m), dim3(64), 0, s, tg, rows, v0, width,
                     zk, lse, P, ldp);
  return hipGetLastError();
}

}  // namespace gptq
