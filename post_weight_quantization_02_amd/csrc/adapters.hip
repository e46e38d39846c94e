// Low-rank adapters of many requests beside one stored layer:
//   y_t  = W_hat x_t + s_a B_a (A_a x_t),       a = index[t]
// and the adapters' gradients, with dv_t = s_a B_a^T dy_t:
//   dA_a = sum_{t: index[t] = a} dv_t x_t^T,    dB_a = sum dy_t v_t^T,
// v_t = s_a A_a x_t.  A_a is rank x cols, B_a rows x rank (fp16); v and dv are
// fp32, and every product below is exact in fp32 and summed in fp32.
#include "adapters_dev.h"

namespace gptq {
namespace {

// 8 values of a row of K values from k on, zero past its end.
template <bool VEC>
__device__ inline half8 load8(const _Float16* row, int64_t k, int64_t K) {
  half8 v = {};
  if (VEC) {  // K % 8 == 0, 16-byte aligned rows
    if (k < K) v = *reinterpret_cast<const half8*>(row + k);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (k + e < K) v[e] = row[k + e];
  }
  return v;
}

__device__ inline int valid_id(const int* index, int64_t t, int count) {
  const int d = index[t];
  return (d >= 0 && d < count) ? d : -1;
}

// Token t's row into its place in xp (see launch_pack_x).
__device__ inline void pack_row(const _Float16* x, int64_t t, int64_t K, _Float16* xp) {
  for (int64_t p = threadIdx.x; p < K / 8; p += 256)  // p: chunk, step, piece
    *reinterpret_cast<half8*>(xp + ((t / 16) * (K / 8) + p) * 128 + (t % 16) * 8) =
        *reinterpret_cast<const half8*>(x + 8 * p);
}

__global__ __launch_bounds__(256) void pack_x_kernel(const _Float16* __restrict__ x, int64_t ldx,
                                                     int64_t K, _Float16* __restrict__ xp) {
  pack_row(x + (int64_t)blockIdx.x * ldx, blockIdx.x, K, xp);
}

// v[t][j] for one token and four j per workgroup: a few tokens, each with an
// adapter of its own (decode).  Bound by the read of the adapters' rows.
template <bool VEC>
__global__ __launch_bounds__(256) void shrink_rows_kernel(ShrinkJob first, ShrinkJob second) {
  __shared__ float red[4][4];
  const ShrinkJob& job = blockIdx.z == 0 ? first : second;
  const int64_t t = blockIdx.x;
  const int j0 = 4 * blockIdx.y;
  const int a = valid_id(job.index, t, job.count);
  float* out = job.v + t * job.ldv + j0;
  if (job.xp != nullptr && blockIdx.y == 0) pack_row(job.x + t * job.ldx, t, job.K, job.xp);
  if (a < 0) {  // the whole workgroup
    if (threadIdx.x < 4) out[threadIdx.x] = 0.f;
    return;
  }
  const _Float16* x = job.x + t * job.ldx;
  const _Float16* down = job.down + a * job.stride;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int64_t k = (int64_t)threadIdx.x * 8; k < job.K; k += 256 * 8) {
    const half8 xv = load8<VEC>(x, k, job.K);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (j0 + u >= job.rank) continue;
      const half8 av = load8<VEC>(down + (j0 + u) * job.ldd, k, job.K);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[u] = __builtin_fmaf((float)xv[e], (float)av[e], acc[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < 4; ++u)
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) acc[u] += __shfl_xor(acc[u], o, 64);
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int u = 0; u < 4; ++u) red[wave][u] = acc[u];
  __syncthreads();
  if (threadIdx.x < 4) {
    const int u = threadIdx.x;
    const float sum = (red[0][u] + red[1][u]) + (red[2][u] + red[3][u]);
    out[u] = j0 + u < job.rank ? job.scaling[a] * sum : 0.f;
  }
}

// v for 16 T tokens per workgroup on v_mfma_f32_16x16x32_f16 (tokens x rank
// tiles of 16), the eight waves taking every eighth run of 32 of K and their
// sums added in wave order.  One pass per adapter found among the tokens, the
// passes dealt out to gridDim.z workgroups, the second ones first: a tile where
// one request ends and the next begins has two, and one workgroup for both
// ends the launch late (8192 tokens, 4096 and 11008 columns: 97 us instead of
// 64; 417 tokens, 1024 and 7791 columns: 33 instead of 19).  Bound by the reads
// from the L2, x once and the adapter's rows for every tile (16 tokens of 4096
// columns at rank 32: 390 KB): U runs are in flight per wave, and twice as many
// take as long.
constexpr int kShrinkWaves = 8;
template <bool VEC, int NB, int U, int T>
__global__ __launch_bounds__(64 * kShrinkWaves) void shrink_tile_kernel(ShrinkJob j0, ShrinkJob j1,
                                                                        int64_t m) {
  constexpr int W = kShrinkWaves;
  __shared__ float red[W][16 * T][16 * NB + 1];
  const ShrinkJob& job = blockIdx.y == 0 ? j0 : j1;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, li = lane & 15, kg = lane >> 4;
  const int64_t t0 = (int64_t)blockIdx.x * 16 * T;
  int id[T];
  const _Float16* x[T];
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const int64_t tok = t0 + 16 * t + li;
    id[t] = tok < m ? valid_id(job.index, tok, job.count) : -1;
    x[t] = job.x + min(tok, m - 1) * job.ldx;
  }
  // zeros where a token has no adapter, and behind the rank
  for (int o = tid; o < 16 * T * job.ldv && blockIdx.z == 0; o += 64 * W) {
    const int tok = o / job.ldv, j = o % job.ldv;
    if (t0 + tok < m && (j >= job.rank || valid_id(job.index, t0 + tok, job.count) < 0))
      job.v[(t0 + tok) * job.ldv + j] = 0.f;
  }
  int cur = -1;
  unsigned pass = 0;
  while (true) {
    int next = 0x7fffffff;
#pragma unroll
    for (int t = 0; t < T; ++t)
      if (id[t] > cur) next = min(next, id[t]);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) next = min(next, __shfl_xor(next, o, 64));
    cur = __builtin_amdgcn_readfirstlane(next);
    if (cur == 0x7fffffff) break;  // the same in all the waves
    if (pass++ % gridDim.z != gridDim.z - 1 - blockIdx.z) continue;
    const _Float16* down = job.down + cur * job.stride;
    f32x4 acc[T][NB];
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[t][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    // workgroups start at different columns: rows whose pitch is a multiple of
    // 2 KB would have all of them read from the same memory channels
    const int64_t turns = ceil_div(job.K, 32 * W * U);
    int64_t turn = blockIdx.x % turns;
    for (int64_t i = 0; i < turns; ++i, turn = turn + 1 == turns ? 0 : turn + 1) {
      const int64_t k0 = 32 * wave + 32 * W * U * turn;
      half8 xv[U][T], dv[U][NB];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t k = k0 + 32 * W * u + 8 * kg;
#pragma unroll
        for (int t = 0; t < T; ++t) xv[u][t] = load8<VEC>(x[t], k, job.K);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const int j = 16 * b + li;  // a row of the adapter, zero behind the rank
          dv[u][b] = load8<VEC>(down + min(j, job.rank - 1) * job.ldd, j < job.rank ? k : job.K,
                                job.K);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
          for (int b = 0; b < NB; ++b)
            acc[t][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(xv[u][t], dv[u][b], acc[t][b], 0, 0, 0);
    }
    __syncthreads();  // the previous turn's reads of red
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[wave][16 * t + 4 * kg + i][16 * b + li] = acc[t][b][i];
    __syncthreads();
    const float s = job.scaling[cur];
    for (int o = tid; o < 16 * T * 16 * NB; o += 64 * W) {
      const int tok = o / (16 * NB), j = o % (16 * NB);
      if (t0 + tok < m && job.index[t0 + tok] == cur && j < job.rank) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) sum += red[w][tok][j];
        job.v[(t0 + tok) * job.ldv + j] = s * sum;
      }
    }
  }
}

// One chunk's sum_t left[t][j] right[t][c] for 64 j x 512 c per workgroup, on
// v_mfma_f32_16x16x4_f32: lane (li, kg) brings token kg of four, left's
// column 16 b + li and eight of right's columns, 8 li .. 8 li + 7 (their
// order inside a tile is free).
template <bool VEC, int NB>
__global__ __launch_bounds__(256) void grad_chunk_kernel(GradJob g0, GradJob g1,
                                                         const int* __restrict__ list,
                                                         const GradChunk* __restrict__ chunks,
                                                         int ldv, int rank, int jblocks) {
  const GradJob& job = blockIdx.z < (unsigned)jblocks ? g0 : g1;
  const int jb = (blockIdx.z % jblocks) * NB;
  const GradChunk ch = chunks[blockIdx.y];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15, kg = lane >> 4;
  const int64_t c0 = (int64_t)blockIdx.x * 512 + 128 * wave + 8 * li;
  if (ch.adapter < 0 || (int64_t)blockIdx.x * 512 + 128 * wave >= job.N) return;
  f32x4 acc[NB][8];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[b][e] = f32x4{0.f, 0.f, 0.f, 0.f};
  // the chunk's tokens, 64 a register: no load of an index before a load of a row
  static_assert(kGradChunk % 64 == 0, "token registers");
  int tok[kGradChunk / 64];
#pragma unroll
  for (int q = 0; q < kGradChunk / 64; ++q)
    tok[q] = list[ch.begin + min(64 * q + lane, ch.count - 1)];
  // U steps of four tokens are loaded while the U before them are used
  constexpr int U = VEC ? (NB <= 2 ? 4 : 2) : 1;
  half8 r[U];
  float l[U][NB];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + 4 * u + kg;
      const bool in = k < ch.count;
      const int q = (k0 + 4 * u) >> 6;  // uniform: 4 | k0
      int mine = tok[0];
#pragma unroll
      for (int i = 1; i < kGradChunk / 64; ++i) mine = q == i ? tok[i] : mine;
      const int64_t t = __shfl(mine, k & 63, 64);
      r[u] = load8<VEC>(job.right + t * job.ldr, in ? c0 : job.R, job.R);
#pragma unroll
      for (int b = 0; b < NB; ++b)
        l[u][b] = in && 16 * (jb + b) < ldv ? job.left[t * ldv + 16 * (jb + b) + li] : 0.f;
    }
  };
  fetch(0);
  for (int k = 0; k < ch.count; k += 4 * U) {
    half8 rc[U];
    float lc[U][NB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rc[u] = r[u];
#pragma unroll
      for (int b = 0; b < NB; ++b) lc[u][b] = l[u][b];
    }
    if (k + 4 * U < ch.count) fetch(k + 4 * U);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int b = 0; b < NB; ++b)
          acc[b][e] =
              __builtin_amdgcn_mfma_f32_16x16x4f32(lc[u][b], (float)rc[u][e], acc[b][e], 0, 0, 0);
  }
  float* out = job.part + (int64_t)blockIdx.y * rank * job.N;
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = 16 * (jb + b) + 4 * kg + i;
      if (j >= rank) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c0 + e < job.N) out[j * job.N + c0 + e] = acc[b][e][i];
    }
}

// The chunks of an adapter added in order.  out[a][j][c] (js = N, cs = 1) or
// out[a][c][j] (js = 1, cs = rank).
__global__ __launch_bounds__(256) void grad_reduce_kernel(GradJob g0, GradJob g1,
                                                          const int2* __restrict__ ranges,
                                                          int rank) {
  const GradJob& job = blockIdx.z == 0 ? g0 : g1;
  const int a = blockIdx.y;
  const int64_t o = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (o >= job.N * rank) return;
  const int2 r = ranges[a];
  float sum = 0.f;
  for (int c = 0; c < r.y; ++c) sum += job.part[(int64_t)(r.x + c) * rank * job.N + o];
  const int64_t j = o / job.N, n = o % job.N;
  job.out[a * job.N * rank + j * job.js + n * job.cs] = sum;
}

__global__ __launch_bounds__(256) void fill_zero_kernel(float* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    p[i] = 0.f;
}

bool vec_ok(const void* p, int64_t ld, int64_t K) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0 && K % 8 == 0;
}

bool vec_job(const ShrinkJob& j) { return vec_ok(j.x, j.ldx, j.K) && vec_ok(j.down, j.ldd, j.K); }

template <bool VEC, int NB>
void shrink_tiles(const ShrinkJob& j0, const ShrinkJob* j1, int64_t m, hipStream_t s) {
  constexpr int U = !VEC ? 1 : NB <= 2 ? 4 : 2;
  // 32 tokens share an adapter row's load where that still fills the CUs
  if constexpr (VEC && NB <= 2) {
    if (m >= 32 * 256) {
      hipLaunchKernelGGL((shrink_tile_kernel<VEC, NB, U, 2>),
                         dim3((unsigned)ceil_div(m, 32), j1 ? 2 : 1, 2), dim3(64 * kShrinkWaves), 0, s,
                         j0, j1 ? *j1 : j0, m);
      return;
    }
  }
  hipLaunchKernelGGL((shrink_tile_kernel<VEC, NB, U, 1>),
                     dim3((unsigned)ceil_div(m, 16), j1 ? 2 : 1, 2),
                     dim3(64 * kShrinkWaves), 0, s, j0, j1 ? *j1 : j0, m);
}

}  // namespace

hipError_t launch_pack_x(const _Float16* x, int64_t ldx, int64_t m, int64_t K, _Float16* xp,
                         hipStream_t s) {
  hipLaunchKernelGGL(pack_x_kernel, dim3((unsigned)m), dim3(256), 0, s, x, ldx, K, xp);
  return hipGetLastError();
}

static hipError_t launch_shrink_rows(const ShrinkJob& j0, const ShrinkJob* j1, int64_t m,
                                     hipStream_t s) {
  const dim3 grid((unsigned)m, (unsigned)(j0.ldv / 4), j1 ? 2 : 1);
  if (vec_job(j0) && (j1 == nullptr || vec_job(*j1)))
    hipLaunchKernelGGL(shrink_rows_kernel<true>, grid, dim3(256), 0, s, j0, j1 ? *j1 : j0);
  else
    hipLaunchKernelGGL(shrink_rows_kernel<false>, grid, dim3(256), 0, s, j0, j1 ? *j1 : j0);
  return hipGetLastError();
}

static hipError_t launch_shrink_tiles(const ShrinkJob& j0, const ShrinkJob* j1, int64_t m, hipStream_t s) {
  const bool vec = vec_job(j0) && (j1 == nullptr || vec_job(*j1));
  const int nb = j0.ldv / 16;
#define GPTQ_SHRINK(V)                        \
  if (nb == 1) shrink_tiles<V, 1>(j0, j1, m, s);      \
  else if (nb == 2) shrink_tiles<V, 2>(j0, j1, m, s); \
  else if (nb <= 4) shrink_tiles<V, 4>(j0, j1, m, s); \
  else shrink_tiles<V, 8>(j0, j1, m, s);
  if (vec) {
    GPTQ_SHRINK(true)
  } else {
    GPTQ_SHRINK(false)
  }
#undef GPTQ_SHRINK
  return hipGetLastError();
}

// A few tokens have workgroups of their own: 16-token tiles leave CUs idle.
// Per token that reads every adapter row again (rank + rank / 4 rows of K from
// the L2), so the limit falls with the rank.
hipError_t launch_shrink(const ShrinkJob& j0, const ShrinkJob* j1, int64_t m, hipStream_t s) {
  if (m * j0.ldv <= 8192) return launch_shrink_rows(j0, j1, m, s);
  const hipError_t e = launch_shrink_tiles(j0, j1, m, s);
  if (e != hipSuccess || j0.xp == nullptr) return e;
  return launch_pack_x(j0.x, j0.ldx, m, j0.K, j0.xp, s);
}

int64_t grad_chunks(int64_t m, int64_t count) { return ceil_div(m, grad_chunk(m)) + count; }

hipError_t launch_grads(const GradJob& g0, const GradJob& g1, int64_t m, int64_t count, int rank,
                        int ldv, const int* list, const GradChunk* chunks, const int2* ranges,
                        hipStream_t s) {
  const int64_t N = g0.N > g1.N ? g0.N : g1.N;
  const bool vec = vec_ok(g0.right, g0.ldr, g0.R) && vec_ok(g1.right, g1.ldr, g1.R);
  const int tiles = ldv / 16, nb = tiles == 1 ? 1 : tiles == 2 ? 2 : 4;
  const int jblocks = (int)ceil_div(tiles, nb);
  const dim3 grid((unsigned)ceil_div(N, 512), (unsigned)grad_chunks(m, count),
                  (unsigned)(2 * jblocks));
#define GPTQ_GRAD(V, B)                                                                    \
  hipLaunchKernelGGL((grad_chunk_kernel<V, B>), grid, dim3(256), 0, s, g0, g1, list, chunks, \
                     ldv, rank, jblocks)
  if (vec) {
    if (nb == 1) GPTQ_GRAD(true, 1);
    else if (nb == 2) GPTQ_GRAD(true, 2);
    else GPTQ_GRAD(true, 4);
  } else {
    if (nb == 1) GPTQ_GRAD(false, 1);
    else if (nb == 2) GPTQ_GRAD(false, 2);
    else GPTQ_GRAD(false, 4);
  }
#undef GPTQ_GRAD
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(grad_reduce_kernel, dim3((unsigned)ceil_div(N * rank, 256), (unsigned)count, 2),
                     dim3(256), 0, s, g0, g1, ranges, rank);
  return hipGetLastError();
}

hipError_t launch_fill_zero(float* p, int64_t n, hipStream_t s) {
  if (n == 0) return hipSuccess;
  const int64_t blocks = ceil_div(n, 256) < 65536 ? ceil_div(n, 256) : 65536;
  hipLaunchKernelGGL(fill_zero_kernel, dim3((unsigned)blocks), dim3(256), 0, s, p, n);
  return hipGetLastError();
}

}  // namespace gptq
