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
  const _Float16* up;    // up[a * stride + j * js + n * ns]
  int64_t stride, js, ns;
  int rank, count;
};

#ifdef __HIPCC__
// Adds the adapters' part to a wave's AT x BT tiles of 16 x 16 outputs
// (lane (li, kg) holds rows 4 kg + i, column li of each): tokens t0.., columns
// n0.. (read clamped to m - 1 and n - 1).  Products run on
// v_mfma_f32_16x16x4_f32, exact in fp32.  The tile's adapters are taken in
// increasing order, each over all of the tile's rows, and a row takes only
// its own adapter's sum, so an infinity or NaN in one adapter never reaches
// another one's tokens.
template <int AT, int BT>
__device__ inline void add_adapters(f32x4 (&acc)[AT][BT], const AdapterTile& ad, int64_t t0,
                                    int64_t m, int64_t n0, int64_t n) {
  const int lane = threadIdx.x & 63, li = lane & 15, kg = lane >> 4;
  int id[AT];  // of token 16 a + li
#pragma unroll
  for (int a = 0; a < AT; ++a) {
    const int64_t t = t0 + 16 * a + li;
    const int d = t < m ? ad.index[t] : -1;
    id[a] = (d >= 0 && d < ad.count) ? d : -1;
  }
  const int steps = (ad.rank + 3) / 4;
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
    const _Float16* up = ad.up + cur * ad.stride;
#pragma unroll
    for (int a = 0; a < AT; ++a) {
      if (__ballot(id[a] == cur) == 0) continue;
      int row = 16 * a + li;
      asm volatile("" : "+v"(row));  // keeps the AT row addresses out of the registers till here
      const float* vrow = ad.v + min(t0 + row, m - 1) * ad.ldv + kg;
      f32x4 part[BT];
#pragma unroll
      for (int b = 0; b < BT; ++b) part[b] = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int s = 0; s < steps; ++s) {
        const float av = vrow[4 * s];
        const int j = 4 * s + kg;
#pragma unroll
        for (int b = 0; b < BT; ++b) {
          const int64_t c = min(n0 + 16 * b + li, n - 1);
          const float bv = j < ad.rank ? (float)up[j * ad.js + c * ad.ns] : 0.f;
          part[b] = __builtin_amdgcn_mfma_f32_16x16x4f32(av, bv, part[b], 0, 0, 0);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool mine = __shfl(id[a], 4 * kg + i, 64) == cur;
#pragma unroll
        for (int b = 0; b < BT; ++b)
          if (mine) acc[a][b][i] += part[b][i];
      }
    }
  }
}
#endif

}  // namespace gptq
