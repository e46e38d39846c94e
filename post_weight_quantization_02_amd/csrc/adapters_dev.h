// Low-rank adapters as the kernels see them, and their part of an output tile.
//
// A token t with adapter a = index[t] adds v_t up_a to its output row, v_t
// (rank values, fp32, the adapter's scale already in it) formed beforehand:
// forward v = s x A^T and up[j][n] = B[n][j]; backward v = s dy B and
// up[j][c] = A[j][c].  Tokens with an index outside [0, count) have none.
#pragma once

#include "common.h"

namespace gptq {

struct AdapterTile {
  const float* v;        // tokens x ldv
  int ldv;               // a multiple of 16; columns from rank on hold zeros
  const int* index;      // one per token
  const _Float16* up;    // up[a * stride + n * ns + j]
  int64_t stride, ns;
  int rank, count;
};

#ifdef __HIPCC__
// 8 values of a row of up from j on, zeros from the rank on.  vec: 16-byte
// aligned rows, whose values behind the rank, up to ns, are zeros.
__device__ inline half8 load_up(const AdapterTile& ad, const _Float16* row, int j, bool vec) {
  half8 u = {};
  if (vec) {
    if (j < ad.rank) u = *reinterpret_cast<const half8*>(row + j);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (j + e < ad.rank) u[e] = row[j + e];
  }
  return u;
}

__device__ inline bool vec_up(const AdapterTile& ad) {
  return ad.ns % 8 == 0 && ad.stride % 8 == 0 && (reinterpret_cast<uintptr_t>(ad.up) & 15) == 0;
}

// Adds the adapters' part to a wave's AT x BT tiles of 16 x 16 outputs (lane
// (li, kg) holds rows 4 kg + i, column li of each): tokens t0.., columns n0..
// (read clamped to m - 1 and n - 1).
//
// 16 of the rank's values at a time: v = 2^e (hi + lo), both fp16, 2^e the size
// of the largest of the 16, which keeps 23 bits below it.  hi and lo are the
// two halves of one operand of v_mfma_f32_16x16x32_f16 against [up | up], whose
// products are exact in fp32; the sum is scaled by 2^e (exact) and added.
// (On v_mfma_f32_16x16x4_f32, with loads of single values, the 4096 x 11008
// outputs of a 4096-token prompt at rank 32 took 711 us instead of 538.)
//
// The tile's adapters are taken in increasing order, each over all of the
// tile's rows, and a row takes only its own adapter's sum, so an infinity or
// NaN in one adapter never reaches another one's tokens.
template <int AT, int BT>
__device__ inline void add_adapters(f32x4 (&acc)[AT][BT], const AdapterTile& ad, int64_t t0,
                                    int64_t m, int64_t n0, int64_t n) {
  const int lane = threadIdx.x & 63, li = lane & 15, kg = lane >> 4;
  const bool vec = vec_up(ad);
  int id[AT];  // of token 16 a + li
#pragma unroll
  for (int a = 0; a < AT; ++a) {
    const int64_t t = t0 + 16 * a + li;
    const int d = t < m ? ad.index[t] : -1;
    id[a] = (d >= 0 && d < ad.count) ? d : -1;
  }
  int cur = -1;
  while (true) {
    int next = 0x7fffffff;
#pragma unroll
    for (int a = 0; a < AT; ++a)
      if (id[a] > cur && id[a] < next) next = id[a];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) next = min(next, __shfl_xor(next, o, 64));
    cur = __builtin_amdgcn_readfirstlane(next);
    if (cur == 0x7fffffff) break;  // every wave ends: cur grows each turn
    for (int j0 = 0; j0 < ad.rank; j0 += 16) {
      const int j = j0 + 8 * (kg & 1);
      half8 u[BT];
#pragma unroll
      for (int b = 0; b < BT; ++b)
        u[b] = load_up(ad, ad.up + cur * ad.stride + min(n0 + 16 * b + li, n - 1) * ad.ns, j, vec);
#pragma unroll
      for (int a = 0; a < AT; ++a) {
        if (__ballot(id[a] == cur) == 0) continue;
        int row = 16 * a + li;
        asm volatile("" : "+v"(row));  // the AT row addresses not before they are needed
        const float* vrow = ad.v + min(t0 + row, m - 1) * ad.ldv + j;
        const float4 v0 = *reinterpret_cast<const float4*>(vrow);
        const float4 v1 = *reinterpret_cast<const float4*>(vrow + 4);
        const float w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, __builtin_fabsf(w[e]));
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        const int ex = top < INFINITY ? __builtin_amdgcn_frexp_expf(top) : 0;
        half8 f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = __builtin_ldexpf(w[e], -ex);
          const _Float16 hi = (_Float16)x;
          const float rest = x - (float)hi;  // not a number where hi is infinite
          f[e] = kg < 2 ? hi : __builtin_fabsf(x) < 2.f ? (_Float16)rest : (_Float16)0.f;
        }
        f32x4 part[BT];
#pragma unroll
        for (int b = 0; b < BT; ++b)
          part[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f, u[b], f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool mine = __shfl(id[a], 4 * kg + i, 64) == cur;
          const int up = __shfl(ex, 4 * kg + i, 64);
#pragma unroll
          for (int b = 0; b < BT; ++b)
            if (mine) acc[a][b][i] += __builtin_ldexpf(part[b][i], up);
        }
      }
    }
  }
}

// sum_j v[t][j] up[a][r][j] of one token and output in fp32, 0 without an
// adapter.
__device__ inline float low_rank(const AdapterTile& ad, int64_t t, int64_t r, bool vec) {
  const int a = ad.index[t];
  if (a < 0 || a >= ad.count) return 0.f;
  const _Float16* up = ad.up + a * ad.stride + r * ad.ns;
  const float* v = ad.v + t * ad.ldv;
  float sum = 0.f;
  for (int j = 0; j < ad.rank; j += 8) {
    const half8 u = load_up(ad, up, j, vec);
    const float4 v0 = *reinterpret_cast<const float4*>(v + j);
    const float4 v1 = *reinterpret_cast<const float4*>(v + j + 4);
    sum = __builtin_fmaf(v0.x, (float)u[0], sum);
    sum = __builtin_fmaf(v0.y, (float)u[1], sum);
    sum = __builtin_fmaf(v0.z, (float)u[2], sum);
    sum = __builtin_fmaf(v0.w, (float)u[3], sum);
    sum = __builtin_fmaf(v1.x, (float)u[4], sum);
    sum = __builtin_fmaf(v1.y, (float)u[5], sum);
    sum = __builtin_fmaf(v1.z, (float)u[6], sum);
    sum = __builtin_fmaf(v1.w, (float)u[7], sum);
  }
  return sum;
}
#endif

}  // namespace gptq
