// The layer's product from its stored form and what the calls do with its sums
// (linear_mfma.hip, linear_wide.hip).
#pragma once

#include "adapters_dev.h"
#include "store_tile.h"
#include "tile_grid.h"

namespace gptq {

// What becomes of a tile's sums:
//   kStore     fp16 outputs, the layer's own product
//   kAdapters  the adapters' part added first (adapters_dev.h)
//   kSplit     fp32 sums of one split of the input columns
//   kPartials  z = sum * inv_t: per token the tile's max and sum exp(z - max),
//              the pieces of the softmax statistics of a vocabulary whose
//              logits are not kept, and the logits that the targets name
//   kProbs     exp(z - lse) in fp16, the softmax of one piece of it
enum TailMode { kStore = 0, kAdapters = 1, kSplit = 2, kPartials = 3, kProbs = 4 };
struct Tail {
  AdapterTile ad;
  float* sums;       // splits x m x rows
  float inv_t;
  float2* part;      // output tiles x m
  const float* lse;  // m
  const int* index;  // m x top
  int top;
  float* zk;         // m x top
};

// One product: y = x W_hat^T for m tokens.
struct LinearCall {
  const _Float16* x;
  int64_t ldx, m;
  const uint32_t* packed;
  int64_t rows, cols;
  const float *scales, *zeros;
  int groupsize;
  _Float16* y;
  int64_t ldy;
  const float *scales_t, *zeros_t;  // groups x pitch_t (launch_scales), for the wide shape
  int64_t pitch_t;
};

template <bool RELU, int TAIL>
hipError_t launch_linear_wide(int bits, const LinearCall& c, const Tail& tail, hipStream_t s);

// An XCD takes 4 token tiles x 8 output tiles at once (at 128 x 256 outputs,
// 32 KB and 16 KB per stage: the split that minimises its misses).  With fewer
// than 32 token tiles xm falls below 8, so that an XCD still has 4 of them and
// the weights are read by fewer XCDs.
constexpr int kGroupM = 4;
inline TileGrid linear_grid(int64_t ntm, int64_t ntn) {
  TileGrid g{ntm, ntn, kXcds, kGroupM};
  while (g.xm > 1 && ntm < g.xm * kGroupM) g.xm /= 2;
  const int64_t mine = ceil_div(ntm, g.xm);
  if (mine < g.gm) g.gm = (int)mine;
  return g;
}

#ifdef __HIPCC__
// Below, a workgroup of WM x WN waves holds 16 AT WM tokens x 16 BT WN outputs
// from (t0, n0) on; this wave is (wm, wn).

// (max, sum exp(z - max)) of two sets of values as one's.
__device__ inline void join(float& top, float& sum, float top2, float sum2) {
  const float t = fmaxf(top, top2), base = t == -INFINITY ? 0.f : t;
  sum = sum * __expf(top - base) + sum2 * __expf(top2 - base);
  top = t;
}

// (max, sum exp(z - max)) of the tile's outputs for each of its tokens.  Every
// lane takes its own BT outputs of 16 rows; four exchanges over its 16 lanes,
// each halving the rows a lane keeps (8 + 4 + 2 + 1 pairs, where a butterfly
// for every row takes 64), leave one row to a lane; the waves' are joined
// through LDS.  Outputs past the matrix count as -inf.
template <int AT, int BT, int WM, int WN>
__device__ inline void tile_partials(const f32x4 (&acc)[AT][BT], const Tail& tail, float2* red,
                                     int64_t t0, int64_t m, int64_t tn, int64_t n0, int64_t rows,
                                     int wm, int wn) {
  constexpr int TM = 16 * AT * WM;
  const int tid = threadIdx.x, lane = tid & 63, li = lane & 15, kg = lane >> 4;
  const int64_t nw = n0 + 16 * BT * wn;
#pragma unroll
  for (int c = 0; c < AT / 4; ++c) {
    float top[16], sum[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float z[BT];
      top[r] = -INFINITY;
#pragma unroll
      for (int b = 0; b < BT; ++b) {
        z[b] = nw + 16 * b + li < rows ? acc[4 * c + r / 4][b][r % 4] * tail.inv_t : -INFINITY;
        top[r] = fmaxf(top[r], z[b]);
      }
      const float base = top[r] == -INFINITY ? 0.f : top[r];
      sum[r] = 0.f;
#pragma unroll
      for (int b = 0; b < BT; ++b) sum[r] += __expf(z[b] - base);
    }
#pragma unroll
    for (int half = 8; half > 0; half >>= 1) {  // also the lanes' distance
      const bool up = (li & half) != 0;
#pragma unroll
      for (int r = 0; r < half; ++r) {
        const float t = __shfl_xor(up ? top[r] : top[r + half], half, 64);
        const float s = __shfl_xor(up ? sum[r] : sum[r + half], half, 64);
        if (up) {
          top[r] = top[r + half];
          sum[r] = sum[r + half];
        }
        join(top[r], sum[r], t, s);
      }
    }
    // row li of the 16: tile 4 c + li / 4, row 4 kg + li % 4 of it
    red[wn * TM + 16 * (AT * wm + 4 * c + li / 4) + 4 * kg + li % 4] = make_float2(top[0], sum[0]);
  }
  __syncthreads();
  if (tid < TM && t0 + tid < m) {
    float2 p = red[tid];
#pragma unroll
    for (int w = 1; w < WN; ++w) {
      const float2 q = red[w * TM + tid];
      join(p.x, p.y, q.x, q.y);
    }
    tail.part[tn * m + t0 + tid] = p;
  }
}

// zk[t][k] = z[t][index[t][k]] for the named outputs inside the tile: 16
// tokens' sums of every wave row at a time go through LDS, and every thread
// looks its share of their entries up, the entries of the next 16 tokens being
// loaded meanwhile.
template <int AT, int BT, int WM, int WN>
__device__ inline void tile_targets(const f32x4 (&acc)[AT][BT], const Tail& tail, float* zs,
                                    int64_t t0, int64_t m, int64_t n0, int64_t rows, int wm,
                                    int wn) {
  constexpr int TN = 16 * BT * WN, PITCH = TN + 4;  // rows 4 banks apart
  constexpr int THREADS = 64 * WM * WN, U = 4;      // entries per thread that are loaded ahead
  const int tid = threadIdx.x, lane = tid & 63, li = lane & 15, kg = lane >> 4;
  const int64_t end = min(n0 + TN, rows);
  const int each = 16 * tail.top, n = WM * each;
  // entry e of step a: wave row e / each, token (e % each) / top of its 16
  auto place = [&](int a, int e, int& row) -> int64_t {
    const int w = e / each, r = e % each;
    row = 16 * w + r / tail.top;
    const int64_t t = t0 + 16 * (AT * w + a) + r / tail.top;
    return e < n && t < m ? t * tail.top + r % tail.top : -1;
  };
  int next[U];
  auto load = [&](int a) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      int row;
      const int64_t at = place(a, tid + THREADS * u, row);
      next[u] = at >= 0 ? tail.index[at] : -1;
    }
  };
  load(0);
#pragma unroll
  for (int a = 0; a < AT; ++a) {
    int now[U];
#pragma unroll
    for (int u = 0; u < U; ++u) now[u] = next[u];
    if (a + 1 < AT) load(a + 1);
    __syncthreads();
#pragma unroll
    for (int b = 0; b < BT; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        zs[(16 * wm + 4 * kg + i) * PITCH + 16 * (BT * wn + b) + li] = acc[a][b][i];
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (now[u] >= n0 && now[u] < end) {
        int row;
        const int64_t at = place(a, tid + THREADS * u, row);
        tail.zk[at] = zs[row * PITCH + (now[u] - n0)] * tail.inv_t;
      }
    for (int e = tid + THREADS * U; e < n; e += THREADS) {
      int row;
      const int64_t at = place(a, e, row);
      const int v = at >= 0 ? tail.index[at] : -1;
      if (v >= n0 && v < end) tail.zk[at] = zs[row * PITCH + (v - n0)] * tail.inv_t;
    }
  }
}

// s0 and s1: LDS that the product is done with (behind a barrier, taken here).
template <bool RELU, int TAIL, int AT, int BT, int WM, int WN>
__device__ inline void tile_tail(f32x4 (&acc)[AT][BT], const Tail& tail, const LinearCall& c,
                                 int64_t t0, int64_t n0, int64_t tn, int wm, int wn, char* s0,
                                 char* s1) {
  const int lane = threadIdx.x & 63, li = lane & 15, kg = lane >> 4;
  const int64_t tw = t0 + 16 * AT * wm, nw = n0 + 16 * BT * wn, m = c.m, rows = c.rows;
  if constexpr (TAIL == kAdapters) add_adapters<AT, BT>(acc, tail.ad, tw, m, nw, rows);
  if constexpr (TAIL == kPartials) {
    __syncthreads();
    tile_partials<AT, BT, WM, WN>(acc, tail, reinterpret_cast<float2*>(s0), t0, m, tn, n0, rows, wm,
                                  wn);
    tile_targets<AT, BT, WM, WN>(acc, tail, reinterpret_cast<float*>(s1), t0, m, n0, rows, wm, wn);
    return;
  }
  // lane holds rows 4 * kg + i of each 16 x 16 tile, column li
  if constexpr (TAIL == kAdapters || TAIL == kProbs) {
    static_assert(StoreTile<BT>::kBytes * WM * WN <= 32 * 1024, "LDS of a stage");
    __syncthreads();  // the stages are free
    char* lds = s0 + StoreTile<BT>::kBytes * (threadIdx.x >> 6);
    const bool wide = wide_rows(c.y, c.ldy);
    // probabilities go on in zeros to the end of the piece's rows
    const int64_t end = TAIL == kProbs ? min(c.ldy, n0 + 16 * BT * WN) : rows;
#pragma unroll
    for (int a = 0; a < AT; ++a) {
      f32x4 v[BT];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t t = tw + 16 * a + 4 * kg + i;
        const float lse = TAIL == kProbs && t < m ? tail.lse[t] : 0.f;
#pragma unroll
        for (int b = 0; b < BT; ++b) {
          float x = acc[a][b][i];
          if constexpr (TAIL == kProbs) {
            const bool in = nw + 16 * b + li < rows && lse != INFINITY;
            x = in ? __expf(x * tail.inv_t - lse) : 0.f;
          } else if (RELU) {
            x = x > 0.f ? x : 0.f;
          }
          v[b][i] = x;
        }
      }
      store_rows<BT>(v, lds, c.y, c.ldy, tw + 16 * a, m, nw, end, wide);
    }
    return;
  }
#pragma unroll
  for (int a = 0; a < AT; ++a)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t t = tw + 16 * a + 4 * kg + i;
      if (t >= m) continue;
#pragma unroll
      for (int b = 0; b < BT; ++b) {
        const int64_t r = nw + 16 * b + li;
        if (r >= rows) continue;
        float v = acc[a][b][i];
        if constexpr (TAIL == kSplit) {
          tail.sums[((int64_t)blockIdx.y * m + t) * rows + r] = v;
          continue;
        }
        if (RELU) v = v > 0.f ? v : 0.f;
        c.y[t * c.ldy + r] = (_Float16)v;
      }
    }
}
#endif

}  // namespace gptq
