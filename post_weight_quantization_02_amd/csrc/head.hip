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

// The gradient at the named entries, dz_k = exp(z_k - lse) - sum of their
// probabilities (an index named by several entries gets the sum from each of
// them), in fp32; one token per wave.  dz16 is what the product takes, rest =
// dz - dz16 what its rounding leaves (0 for a repeated index but the first,
// and for entries under 1/32 of the token's largest, whose roundings are as
// much smaller).  Also lse_eff = lse or +inf and gscale = dloss inv_t or 0, for
// tokens with and without entries.
__global__ __launch_bounds__(256) void head_entries_kernel(
    HeadTargets tg, int64_t m, int64_t rows, const float* __restrict__ zk,
    const float* __restrict__ lse, const float* __restrict__ dloss, float* __restrict__ lse_eff,
    float* __restrict__ gscale, _Float16* __restrict__ dz16, float* __restrict__ rest) {
  __shared__ int idx[4][kMaxTop];
  __shared__ float prob[4][kMaxTop];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t t = min((int64_t)blockIdx.x * 4 + wave, m - 1);  // (the last ones again)
  bool any;
  const float tlse = teacher_lse(tg, t, rows, &any);
  for (int k = lane; k < tg.top; k += 64) {
    const bool in = takes_part(tg, t, k, rows);
    idx[wave][k] = in ? tg.index[t * tg.top + k] : -1;
    prob[wave][k] = in ? __expf(log_p(tg, t, k, tlse)) : 0.f;
  }
  __syncthreads();
  const float l = lse[t];
  float dz[kMaxTop / 64], top = 0.f;
  bool mine[kMaxTop / 64];
#pragma unroll
  for (int u = 0; u < kMaxTop / 64; ++u) {
    const int k = lane + 64 * u;
    dz[u] = 0.f;
    mine[u] = false;
    if (k >= tg.top || idx[wave][k] < 0) continue;
    const int v = idx[wave][k];
    float p = 0.f;
    bool first = true;
    for (int o = 0; o < tg.top; ++o)
      if (idx[wave][o] == v) {
        p += prob[wave][o];
        first = first && o >= k;
      }
    dz[u] = __expf(zk[t * tg.top + k] - l) - p;
    mine[u] = first;
    top = fmaxf(top, __builtin_fabsf(dz[u]));
  }
  top = wave_max(top);
#pragma unroll
  for (int u = 0; u < kMaxTop / 64; ++u) {
    const int k = lane + 64 * u;
    if (k >= tg.top) continue;
    const _Float16 h = (_Float16)dz[u];
    dz16[t * tg.top + k] = h;
    rest[t * tg.top + k] =
        mine[u] && __builtin_fabsf(dz[u]) * 32.f >= top ? dz[u] - (float)h : 0.f;
  }
  if (lane == 0) {
    lse_eff[t] = any ? l : INFINITY;
    gscale[t] = any ? dloss[t] * tg.inv_t : 0.f;
  }
}

// The named entries' dz16 into one piece of the probabilities.
__global__ __launch_bounds__(256) void head_scatter_kernel(HeadTargets tg, int64_t m, int64_t rows,
                                                           int64_t v0, int64_t width,
                                                           const _Float16* __restrict__ dz16,
                                                           _Float16* __restrict__ P, int64_t ldp) {
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= m * tg.top) return;
  const int64_t t = e / tg.top;
  const int64_t v = tg.index[e];
  if (v >= v0 && v < v0 + width && takes_part(tg, t, (int)(e % tg.top), rows))
    P[t * ldp + v - v0] = dz16[e];
}

// sums[t] = sum_k rest[t][k] W_hat[index[t][k]] in fp32, what the entries'
// rounding leaves out of the product (their dz are the gradient's largest
// terms, and W_hat and dh are rounded already: without this dh is 1.65 times a
// single rounding off).  One token per workgroup, a word (4 bits) or two (8)
// of the rows per thread and turn; bound by the rows' reads from the caches.
template <int BITS>
__global__ __launch_bounds__(256) void head_rest_kernel(
    HeadTargets tg, const uint32_t* __restrict__ packed, int64_t nw, int64_t cols,
    const float* __restrict__ scales, const float* __restrict__ zeros, int64_t ngroups,
    int groupsize, const float* __restrict__ rest, float* __restrict__ sums) {
  constexpr int W = BITS / 4;  // words of 8 codes
  constexpr uint32_t MASK = (1u << BITS) - 1u;
  __shared__ int64_t row[kMaxTop];
  __shared__ float weight[kMaxTop];
  __shared__ int count;
  const int64_t t = blockIdx.x;
  if (threadIdx.x < 64) {  // the entries that have something, in order
    int n = 0;
    for (int k0 = 0; k0 < tg.top; k0 += 64) {
      const int k = k0 + threadIdx.x;
      const float r = k < tg.top ? rest[t * tg.top + k] : 0.f;
      const unsigned long long b = __ballot(r != 0.f);  // (true for NaN)
      if (r != 0.f) {
        const int at = n + __popcll(b & ((1ull << threadIdx.x) - 1));
        row[at] = tg.index[t * tg.top + k];
        weight[at] = r;
      }
      n += __popcll(b);
    }
    if (threadIdx.x == 0) count = n;
  }
  __syncthreads();
  const int n = count;
  for (int64_t c = (int64_t)threadIdx.x * 8; c < cols; c += 256 * 8) {
    const int64_t g = c / groupsize;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const int64_t r = row[i];
      uint32_t q[W];
#pragma unroll
      for (int w = 0; w < W; ++w) q[w] = packed[r * nw + c * BITS / 32 + w];
      const float s = scales[r * ngroups + g] * weight[i], z = zeros[r * ngroups + g];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        acc[j] = __builtin_fmaf(
            s, (float)((q[j * BITS / 32] >> (j * BITS % 32)) & MASK) - z, acc[j]);
    }
    float4* out = reinterpret_cast<float4*>(sums + t * cols + c);
    out[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    out[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
  }
}

}  // namespace

hipError_t launch_head_finish(int64_t m, int64_t rows, const HeadTargets& tg, const float2* part,
                              int64_t tiles, float* loss, float* lse, float* zk, hipStream_t s) {
  hipLaunchKernelGGL(head_finish_kernel, dim3((unsigned)ceil_div(m, 4)), dim3(256), 0, s, m, rows,
                     tg, part, tiles, loss, lse, zk);
  return hipGetLastError();
}

hipError_t launch_head_entries(const HeadTargets& tg, int64_t m, int64_t rows, const float* zk,
                               const float* lse, const float* dloss, float* lse_eff,
                               float* gscale, _Float16* dz16, float* rest, hipStream_t s) {
  hipLaunchKernelGGL(head_entries_kernel, dim3((unsigned)ceil_div(m, 4)), dim3(256), 0, s, tg, m,
                     rows, zk, lse, dloss, lse_eff, gscale, dz16, rest);
  return hipGetLastError();
}

hipError_t launch_head_scatter(const HeadTargets& tg, int64_t m, int64_t rows, int64_t v0,
                               int64_t width, const _Float16* dz16, _Float16* P, int64_t ldp,
                               hipStream_t s) {
  hipLaunchKernelGGL(head_scatter_kernel, dim3((unsigned)ceil_div(m * tg.top, 256)), dim3(256), 0, s,
                     tg, m, rows, v0, width, dz16, P, ldp);
  return hipGetLastError();
}

hipError_t launch_head_rest(int bits, const HeadTargets& tg, int64_t m, const uint32_t* packed,
                            int64_t cols, const float* scales, const float* zeros, int groupsize,
                            const float* rest, float* sums, hipStream_t s) {
  const int64_t nw = packed_words(cols, bits), ng = ceil_div(cols, groupsize);
  if (bits == 4)
    hipLaunchKernelGGL(head_rest_kernel<4>, dim3((unsigned)m), dim3(256), 0, s, tg, packed, nw, cols,
                       scales, zeros, ng, groupsize, rest, sums);
  else
    hipLaunchKernelGGL(head_rest_kernel<8>, dim3((unsigned)m), dim3(256), 0, s, tg, packed, nw, cols,
                       scales, zeros, ng, groupsize, rest, sums);
  return hipGetLastError();
}

}  // namespace gptq
