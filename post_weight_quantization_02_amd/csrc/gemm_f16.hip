// The gradient through a stored layer, dx = dy W_hat, and the products of the
// vocabulary losses' gradient: the stored weights are written once in fp16
// with the layer's outputs along the fast axis (launch_prepare), and a dense
// fp16 product C = A B^T over that axis follows; few tokens take the weights
// straight from the packed words instead.
//
// W_hat = (code - zero) * scale is formed in fp32 and rounded to fp16 once
// (at most 2^-11 of its size, 2^-25 below 2^-14); the products are exact in
// fp32 and summed there.
#include "adapters_dev.h"
#include "store_tile.h"
#include "tile_grid.h"

namespace gptq {
namespace {

// ------------------------------------------------------- what goes before
// One launch writes the transposed weights and, for the adapters' gradients,
// A and B the other way round and the tokens grouped by adapter: workgroups of
// one kind after another, the grouping (a few long ones) first.
struct Prepare {
  // the layer
  const uint32_t* packed;
  int bits;
  int64_t nw, rows, cols, kp;
  const float *scales, *zeros;
  int64_t ngroups;
  int groupsize;
  const int* g_idx;
  int64_t ldt;
  _Float16* wt;
  // adapters (count 0: none)
  const _Float16* B;
  int64_t count;
  int rank;
  int64_t ldb;
  _Float16* bt;
  const _Float16* A;
  int lda;
  _Float16* at;
  const int* index;
  int64_t m;
  int chunk, max_chunks;
  int* list;
  GradChunk* chunks;
  int2* ranges;
  int64_t bt_blocks, at_blocks, wt_x, wt_blocks;  // workgroups of each kind (wt_x per row of them)
};

// 4 and 8 bits, every word inside a group.  A lane takes one word of eight
// adjacent rows (4 or 8 columns x 8 rows), so its outputs are whole 16-byte
// pieces of the transposed rows; the lanes of a wave are eight such row groups
// x eight words, which makes 128 adjacent bytes of eight rows per store.
// Bound by the store: 90 MB at 11008 x 4096, 34 us.
template <int BITS>
__device__ inline void transpose_words(const Prepare& p, int64_t bx, int64_t by) {
  constexpr int K = 32 / BITS;
  constexpr uint32_t MASK = (1u << BITS) - 1u;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t r0 = bx * 64 + 8 * (lane & 7);
  const int64_t w = by * 32 + 8 * wave + (lane >> 3);
  if (w >= p.nw || r0 >= p.kp) return;
  const int64_t g = w * K / p.groupsize;
  uint32_t q[8];
  float s[8], z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = min(r0 + i, p.rows - 1);
    q[i] = p.packed[r * p.nw + w];
    s[i] = p.scales[r * p.ngroups + g];
    z[i] = p.zeros[r * p.ngroups + g];
  }
#pragma unroll
  for (int j = 0; j < K; ++j) {
    half8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float f = ((float)((q[i] >> (BITS * j)) & MASK) - z[i]) * s[i];
      v[i] = (_Float16)(r0 + i < p.rows ? f : 0.f);
    }
    if (w * K + j < p.cols) *reinterpret_cast<half8*>(p.wt + (w * K + j) * p.ldt + r0) = v;
  }
}

// Any bits and groups: 64 rows x 64 columns per workgroup through LDS.
typedef _Float16 TransposeTile[64][64 + 8];
__device__ inline void transpose_tile(const Prepare& p, int64_t bx, int64_t by,
                                      TransposeTile& tile) {
  const int64_t r0 = bx * 64, c0 = by * 64;
  const int tid = threadIdx.x, k = 32 / p.bits;
  const uint32_t mask = (1u << p.bits) - 1u;
  {
    const int64_t c = c0 + (tid & 63);
    const int64_t cc = min(c, p.cols - 1);
    int64_t g = p.g_idx != nullptr ? (int64_t)p.g_idx[cc] : cc / p.groupsize;
    g = g < 0 ? 0 : g >= p.ngroups ? p.ngroups - 1 : g;
    const int64_t w = cc / k;
    const int sh = p.bits * (int)(cc % k);
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
      const int row = (tid >> 6) * 16 + i;
      const int64_t r = r0 + row;
      float v = 0.f;
      if (r < p.rows && c < p.cols) {
        const float q = (float)((p.packed[r * p.nw + w] >> sh) & mask);
        v = (q - p.zeros[r * p.ngroups + g]) * p.scales[r * p.ngroups + g];
      }
      tile[tid & 63][row] = (_Float16)v;
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int o = tid + 256 * u, c = o >> 3, q = o & 7;
    if (c0 + c < p.cols)
      *reinterpret_cast<uint4*>(p.wt + (c0 + c) * p.ldt + r0 + 8 * q) =
          *reinterpret_cast<const uint4*>(&tile[c][8 * q]);
  }
}

// B_a (rows x rank) -> rank x ldb, the rows' order along the fast axis, zeros
// from rows to ldb: the layout that v's kernels read.
__device__ inline void transpose_up(const Prepare& p, int64_t bid) {
  const int64_t per = ceil_div(p.ldb, 256);
  const int64_t a = bid / per, n = (bid % per) * 256 + threadIdx.x;
  if (n >= p.ldb) return;
  for (int j = 0; j < p.rank; ++j)
    p.bt[(a * p.rank + j) * p.ldb + n] =
        n < p.rows ? p.B[(a * p.rows + n) * p.rank + j] : (_Float16)0.f;
}

// A_a (rank x cols) -> cols x lda, zeros behind the rank: what add_adapters
// reads.
__device__ inline void transpose_down(const Prepare& p, int64_t bid) {
  const int64_t per = ceil_div(p.cols, 256);
  const int64_t a = bid / per, c = (bid % per) * 256 + threadIdx.x;
  if (c >= p.cols) return;
  for (int j0 = 0; j0 < p.lda; j0 += 8) {
    half8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = j0 + e < p.rank ? p.A[(a * p.rank + j0 + e) * p.cols + c] : (_Float16)0.f;
    *reinterpret_cast<half8*>(p.at + (a * p.cols + c) * p.lda + j0) = v;
  }
}

// Tokens grouped by adapter, in token order inside each (so the gradients'
// sums have one order), and cut into chunks of at most `chunk` tokens of one
// adapter.  One workgroup per adapter: it counts every adapter's tokens
// (integer LDS atomics), finds its own places and writes its own tokens, 16
// adjacent ones a thread at a time.
struct GroupShared {
  int hist[kMaxGradAdapters];
  int wsum[4], base;
};
constexpr int kPerThread = 16;

__device__ inline void group_tokens(const Prepare& p, int a, GroupShared& sh) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, count = (int)p.count;
  for (int i = tid; i < count; i += 256) sh.hist[i] = 0;
  __syncthreads();
#pragma unroll 8
  for (int64_t t = tid; t < p.m; t += 256) {
    const int d = p.index[t];
    if (d >= 0 && d < count) atomicAdd(&sh.hist[d], 1);
  }
  __syncthreads();
  if (wave == 0) {  // tokens and chunks of the adapters before this one
    int tokens = 0, before = 0, total = 0;
    for (int i = lane; i < count; i += 64) {
      const int c = (sh.hist[i] + p.chunk - 1) / p.chunk;
      total += c;
      if (i < a) {
        tokens += sh.hist[i];
        before += c;
      }
    }
    for (int o = 32; o > 0; o >>= 1) {
      tokens += __shfl_xor(tokens, o, 64);
      before += __shfl_xor(before, o, 64);
      total += __shfl_xor(total, o, 64);
    }
    const int mine = (sh.hist[a] + p.chunk - 1) / p.chunk;
    if (lane == 0) {
      sh.base = tokens;
      p.ranges[a] = make_int2(before, mine);
    }
    for (int c = lane; c < mine; c += 64)
      p.chunks[before + c] =
          GradChunk{a, tokens + c * p.chunk, min(p.chunk, sh.hist[a] - c * p.chunk)};
    if (a == 0)
      for (int c = total + lane; c < p.max_chunks; c += 64) p.chunks[c] = GradChunk{-1, 0, 0};
  }
  __syncthreads();
  int at = sh.base;
  for (int64_t t0 = 0; t0 < p.m; t0 += 256 * kPerThread) {
    const int64_t first = t0 + tid * kPerThread;
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i)
      if (first + i < p.m && p.index[first + i] == a) mine |= 1u << i;
    int pre = __popc(mine);  // inclusive over the wave's lanes, then exclusive
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(pre, o, 64);
      if (lane >= o) pre += v;
    }
    if (lane == 63) sh.wsum[wave] = pre;
    __syncthreads();
    int all = 0;
    pre -= __popc(mine);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (w < wave) pre += sh.wsum[w];
      all += sh.wsum[w];
    }
    for (int i = 0, n = 0; i < kPerThread; ++i)
      if (mine >> i & 1) p.list[at + pre + n++] = (int)(first + i);
    at += all;
    __syncthreads();
  }
}

// WORDS: 4 or 8, the bits of the layer's word-wise transposition, else 0
template <int WORDS>
__global__ __launch_bounds__(256) void prepare_kernel(Prepare p) {
  __shared__ union {
    GroupShared group;
    TransposeTile tile;
  } sh;
  int64_t bid = blockIdx.x;
  if (bid < p.count) return group_tokens(p, (int)bid, sh.group);
  bid -= p.count;
  if (bid < p.bt_blocks) return transpose_up(p, bid);
  bid -= p.bt_blocks;
  if (bid < p.at_blocks) return transpose_down(p, bid);
  bid -= p.at_blocks;
  if constexpr (WORDS > 0) transpose_words<WORDS>(p, bid % p.wt_x, bid / p.wt_x);
  else transpose_tile(p, bid % p.wt_x, bid / p.wt_x, sh.tile);
}

__global__ __launch_bounds__(256) void pad_rows_kernel(const _Float16* __restrict__ src,
                                                       int64_t lds, int64_t K, int64_t kp,
                                                       int64_t ldd, _Float16* __restrict__ dst) {
  const int64_t t = blockIdx.x, c = ((int64_t)blockIdx.y * 256 + threadIdx.x) * 8;
  if (c >= kp) return;
  half8 v;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = c + e < K ? src[t * lds + c + e] : (_Float16)0.f;
  *reinterpret_cast<half8*>(dst + t * ldd + c) = v;
}

// ------------------------------------------------------------ C = A B^T
// 32 AT tokens x 64 BT outputs per workgroup of eight waves (two by four),
// each AT x BT tiles of v_mfma_f32_16x16x32_f16.  64 columns of K of both
// operands go straight into a stage of LDS by global_load_lds_dwordx4; a row
// of a stage is 128 bytes, its eight 16-byte pieces permuted by (row >> 1) & 7
// so the 16 rows that a fragment read touches use 16 distinct bank groups.
// Rows past the operands are read clamped and not stored.
//
// Measured at 8192 x 4096 outputs, K = 11008 (8192: 4096 x 4096 outputs):
// 256 x 256 with two stages of 64 columns 1213 TF/s (1273); four stages of 32
// columns 1146 (1158); four waves of 128 x 128 1026 (1119); 128 x 256 1068
// (1096); with both pitches a multiple of 2 KB 256 x 256 falls to 1065 (1263).
// The library's fp16 product reaches 1060-1090.  Bound by the matrix units'
// clock under load and the wait at each stage.  128 x 128 with three stages is
// the shape where 256 x 256 leaves CUs idle (1000 x 4096, K = 8192: 85 us
// against 105 with four waves and 32 columns).
constexpr int KC = 64;

typedef __attribute__((address_space(3))) void lds_void;

template <int N>
__device__ inline void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

__device__ inline void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// What becomes of the sums: fp16 (with adapters first, or scaled row by row on
// top of c32: the last of several products), fp32 on top of c32 (the others),
// or the fp32 sums of one split of K.
enum GemmMode { kStore = 0, kStoreAdapters = 1, kAccumulate = 2, kFinish = 3, kSplit = 4 };

struct GemmOut {
  AdapterTile ad;
  _Float16* c16;
  int64_t ldc;
  float* c32;          // m x n
  const float* scale;  // m
  float* sums;         // splits x m x n
};

template <int AT, int BT, int NST, int MODE>
__global__ __launch_bounds__(512, 1) void gemm_nt_kernel(const _Float16* __restrict__ A,
                                                         int64_t lda, int64_t m,
                                                         const _Float16* __restrict__ B,
                                                         int64_t ldb, int64_t n, int64_t K,
                                                         TileGrid grid, GemmOut o) {
  constexpr int TM = 32 * AT, TN = 64 * BT;
  constexpr int ABYTES = TM * KC * 2, STAGE = (TM + TN) * KC * 2;
  constexpr int AU = TM / 64, BU = TN / 64, LPS = AU + BU;  // 8-row loads per wave and stage
  __shared__ __attribute__((aligned(1024))) char ring[NST * STAGE];
  int64_t tm, tn;
  if (!tile_of(grid, blockIdx.x, tm, tn)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3, li = lane & 15, kg = lane >> 4;
  const int64_t t0 = tm * TM, n0 = tn * TN;
  const int all = (int)(K / KC);
  const int kb = MODE == kSplit ? (int)((int64_t)all * blockIdx.y / gridDim.y) : 0;
  const int ke = MODE == kSplit ? (int)((int64_t)all * (blockIdx.y + 1) / gridDim.y) : all;

  // this lane's 16 bytes of each load, from the tile's first row (64-bit: a
  // row pitch may be any user's)
  const char* asrc[AU];
  const char* bsrc[BU];
#pragma unroll
  for (int u = 0; u < AU; ++u) {
    const int row = 8 * (wave + 8 * u) + (lane >> 3);
    asrc[u] = reinterpret_cast<const char*>(A + min(t0 + row, m - 1) * lda) +
              16 * ((lane & 7) ^ ((row >> 1) & 7));
  }
#pragma unroll
  for (int u = 0; u < BU; ++u) {
    const int row = 8 * (wave + 8 * u) + (lane >> 3);
    bsrc[u] = reinterpret_cast<const char*>(B + min(n0 + row, n - 1) * ldb) +
              16 * ((lane & 7) ^ ((row >> 1) & 7));
  }
  auto issue = [&](int k) {
    char* st = ring + ((k - kb) % NST) * STAGE;
    const uint32_t off = (uint32_t)k * (KC * 2);
#pragma unroll
    for (int u = 0; u < AU; ++u)
      __builtin_amdgcn_global_load_lds((const void*)(asrc[u] + off),
                                       (lds_void*)(st + 1024 * (wave + 8 * u)), 16, 0, 0);
#pragma unroll
    for (int u = 0; u < BU; ++u)
      __builtin_amdgcn_global_load_lds((const void*)(bsrc[u] + off),
                                       (lds_void*)(st + ABYTES + 1024 * (wave + 8 * u)), 16, 0, 0);
  };
  f32x4 acc[AT][BT];
#pragma unroll
  for (int a = 0; a < AT; ++a)
#pragma unroll
    for (int b = 0; b < BT; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};

  for (int k = kb; k < kb + NST - 1 && k < ke; ++k) issue(k);
  for (int k = kb; k < ke; ++k) {
    // stage k has landed for this wave, the later ones may be in flight; the
    // barrier publishes it, and behind it nobody reads the stage before
    if (NST == 3 && k + 1 < ke) wait_vm<LPS>();
    else wait_vm<0>();
    lds_barrier();
    if (k + NST - 1 < ke) issue(k + NST - 1);
    const char* st = ring + ((k - kb) % NST) * STAGE;
#pragma unroll
    for (int s = 0; s < KC / 32; ++s) {
      const int frag = 2 * KC * li + 16 * ((4 * s + kg) ^ ((li >> 1) & 7));
      const char* as = st + wm * (16 * AT * 2 * KC) + frag;
      const char* bs = st + ABYTES + wn * (16 * BT * 2 * KC) + frag;
      half8 bf[BT];
#pragma unroll
      for (int b = 0; b < BT; ++b) bf[b] = *reinterpret_cast<const half8*>(bs + 32 * KC * b);
#pragma unroll
      for (int a = 0; a < AT; ++a) {
        const half8 af = *reinterpret_cast<const half8*>(as + 32 * KC * a);
#pragma unroll
        for (int b = 0; b < BT; ++b)
          acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(af, bf[b], acc[a][b], 0, 0, 0);
      }
    }
  }

  const int64_t tw = t0 + 16 * AT * wm, nw = n0 + 16 * BT * wn;  // this wave's corner
  if constexpr (MODE == kStoreAdapters) add_adapters<AT, BT>(acc, o.ad, tw, m, nw, n);
  if constexpr (MODE == kStore || MODE == kStoreAdapters || MODE == kFinish) {
    lds_barrier();  // the stages are free: every wave's reads are in its products
    char* lds = ring + StoreTile<BT>::kBytes * wave;
    const bool wide = wide_rows(o.c16, o.ldc);
#pragma unroll
    for (int a = 0; a < AT; ++a) {
      if constexpr (MODE == kFinish) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t t = tw + 16 * a + 4 * kg + i;
          if (t >= m) continue;
#pragma unroll
          for (int b = 0; b < BT; ++b) {
            const int64_t c = nw + 16 * b + li;
            if (c < n) acc[a][b][i] += o.c32[t * n + c];
            acc[a][b][i] *= o.scale[t];
          }
        }
      }
      store_rows<BT>(acc[a], lds, o.c16, o.ldc, tw + 16 * a, m, nw, n, wide);
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
        const int64_t c = nw + 16 * b + li;
        if (c >= n) continue;
        const float v = acc[a][b][i];
        if constexpr (MODE == kSplit) {
          o.sums[((int64_t)blockIdx.y * m + t) * n + c] = v;
        } else {
          o.c32[t * n + c] += v;
        }
      }
    }
}

// The splits added in order, then as the modes above.
template <int MODE>
__global__ __launch_bounds__(256) void gemm_reduce_kernel(int splits, int64_t m, int64_t n,
                                                          GemmOut o) {
  const int64_t t = blockIdx.x, c = (int64_t)blockIdx.y * 256 + threadIdx.x;
  if (c >= n) return;
  float v = 0.f;
#pragma unroll 8
  for (int k = 0; k < splits; ++k) v += o.sums[(k * m + t) * n + c];
  if constexpr (MODE == kStoreAdapters) v += low_rank(o.ad, t, c, vec_up(o.ad));
  if constexpr (MODE == kAccumulate || MODE == kFinish)
    v += o.c32[t * n + c];
  if constexpr (MODE == kAccumulate) o.c32[t * n + c] = v;
  else o.c16[t * o.ldc + c] = (_Float16)(MODE == kFinish ? o.scale[t] * v : v);
}

// ------------------------------------------------------- few tokens
// The same product straight from the packed words, for the few tokens that
// would not pay for a transposed copy of the weights: 64 WM tokens x 128
// columns per workgroup and split of the rows (the product's K), 64 rows a
// stage.  A thread takes the words of two adjacent rows, so that a code of
// each makes the adjacent pair that a fragment wants: a byte of both words by
// one v_perm_b32, 1024 + q by bit operations, q by one packed addition
// (exact), and (q - z) * s in fp32, rounded to fp16 once: the transposed copy's
// values, for any z.
// Words, scales and A are loaded two stages ahead into registers, and a stage
// is written to LDS while the one before is multiplied.
//
// 160 tokens x 4096 x 4096 at 8 bits: 24 us, where the transposition (19) and
// the product from the copy (16) took 35; with the pieces in their own order
// 34, with branches around the loads of the last stages 27.  Bound by latency: a split has 8
// stages.
typedef _Float16 h2 __attribute__((ext_vector_type(2)));

template <int BITS, int WM>
__global__ __launch_bounds__(512, 2) void gemm_words_kernel(
    const _Float16* __restrict__ A, int64_t lda, int64_t m, const uint32_t* __restrict__ packed,
    int64_t nw, int64_t rows, int64_t n, int64_t K, const float* __restrict__ scales,
    const float* __restrict__ zeros, int64_t ngroups, int groupsize, float* __restrict__ sums) {
  constexpr int WN = 8 / WM, BT = 8 / WN, TM = 64 * WM, P = KC + 8;
  constexpr int AU = TM / 64;          // 16-byte pieces of A per thread and stage
  constexpr int W = BITS / 4;          // words per row and thread (8 columns)
  __shared__ __attribute__((aligned(16))) _Float16 sa[2][TM * P];
  __shared__ __attribute__((aligned(16))) _Float16 sb[2][128 * KC];
  // 16-byte piece p of column c: the pieces move so that neither the writes
  // (8 columns apart) nor the reads (16 adjacent columns) share banks
  auto piece = [](int c, int p) { return c * KC + 8 * (p ^ ((c ^ (c >> 3)) & 7)); };
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / WN, wn = wave % WN, li = lane & 15, kg = lane >> 4;
  const int64_t c0 = (int64_t)blockIdx.x * 128, t0 = (int64_t)blockIdx.z * TM;
  const int64_t g = c0 / groupsize;
  const int all = (int)(K / KC);
  const int kb = (int)((int64_t)all * blockIdx.y / gridDim.y);
  const int ke = (int)((int64_t)all * (blockIdx.y + 1) / gridDim.y);
  const int pair = tid >> 4, col = 8 * (tid & 15);  // this thread's rows 2 pair, and columns

  struct Stage {
    half8 a[AU];
    uint32_t w[2][W];
    float s[2], z[2];
  };
  auto fetch = [&](Stage& st, int k) {
    k = min(k, ke - 1);  // (no branch: it would hold up the loads in flight)
#pragma unroll
    for (int u = 0; u < AU; ++u)  // rows past the tokens read the last one
      st.a[u] = *reinterpret_cast<const half8*>(
          A + min(t0 + 64 * u + (tid >> 3), m - 1) * lda + (int64_t)k * KC + 8 * (tid & 7));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t r = (int64_t)k * KC + 2 * pair + i, rr = min(r, rows - 1);
#pragma unroll
      for (int v = 0; v < W; ++v)
        st.w[i][v] = packed[rr * nw + (c0 + col) * BITS / 32 + v];
      const float s = scales[rr * ngroups + g], z = zeros[rr * ngroups + g];
      st.s[i] = r < rows ? s : 0.f;  // (A holds zeros behind the rows)
      st.z[i] = r < rows ? z : 0.f;
    }
  };
  auto store = [&](const Stage& st, int buf) {
#pragma unroll
    for (int u = 0; u < AU; ++u)
      *reinterpret_cast<half8*>(&sa[buf][(64 * u + (tid >> 3)) * P + 8 * (tid & 7)]) = st.a[u];
    const h2 base = {(_Float16)-1024.f, (_Float16)-1024.f};
    auto put = [&](int j, uint32_t bits) {  // column col + j: 1024 + q of both rows
      const h2 q = __builtin_bit_cast(h2, bits) + base;
      h2 v;
      v[0] = (_Float16)(((float)q[0] - st.z[0]) * st.s[0]);
      v[1] = (_Float16)(((float)q[1] - st.z[1]) * st.s[1]);
      *reinterpret_cast<h2*>(&sb[buf][piece(col + j, pair >> 2) + 2 * (pair & 3)]) = v;
    };
#pragma unroll
    for (int v = 0; v < W; ++v)
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        // 0x00bb00bb: byte p of the first row's word below, of the second's above
        const uint32_t b = __builtin_amdgcn_perm(st.w[1][v], st.w[0][v],
                                                 0x0c000c00u | ((uint32_t)(4 + p) << 16) | p);
        if constexpr (BITS == 4) {
          put(2 * p, (b & 0x000F000Fu) | 0x64006400u);
          put(2 * p + 1, ((b >> 4) & 0x000F000Fu) | 0x64006400u);
        } else {
          put(4 * v + p, b | 0x64006400u);
        }
      }
  };
  f32x4 acc[4][BT];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < BT; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](int buf) {
#pragma unroll
    for (int s = 0; s < KC / 32; ++s) {
      half8 bf[BT];
#pragma unroll
      for (int b = 0; b < BT; ++b)
        bf[b] = *reinterpret_cast<const half8*>(
            &sb[buf][piece(16 * (BT * wn + b) + li, 4 * s + kg)]);
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const half8 af = *reinterpret_cast<const half8*>(
            &sa[buf][(64 * wm + 16 * a + li) * P + 32 * s + 8 * kg]);
#pragma unroll
        for (int b = 0; b < BT; ++b)
          acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(af, bf[b], acc[a][b], 0, 0, 0);
      }
    }
  };
  Stage s0, s1;
  fetch(s0, kb);
  fetch(s1, kb + 1);
  store(s0, 0);  // kb < ke: every split has a stage
  fetch(s0, kb + 2);
  __syncthreads();
  for (int k = kb; k < ke; k += 2) {
    if (k + 1 < ke) store(s1, 1);
    fetch(s1, k + 3);
    multiply(0);
    __syncthreads();
    if (k + 1 >= ke) break;
    if (k + 2 < ke) store(s0, 0);
    fetch(s0, k + 4);
    multiply(1);
    __syncthreads();
  }
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t t = t0 + 64 * wm + 16 * a + 4 * kg + i;
      if (t >= m) continue;
#pragma unroll
      for (int b = 0; b < BT; ++b)
        sums[((int64_t)blockIdx.y * m + t) * n + c0 + 16 * (BT * wn + b) + li] = acc[a][b][i];
    }
}

// A block of tiles per XCD that is as near a square as 1, 2, 4 or 8 XCDs along
// the tokens make it.
TileGrid gemm_grid(int64_t ntm, int64_t ntn) {
  TileGrid g{ntm, ntn, kXcds, 1};
  while (g.xm > 1 && ceil_div(ntm, g.xm) < ceil_div(ntn, kXcds / g.xm)) g.xm /= 2;
  const int64_t mine = ceil_div(ntm, g.xm);
  g.gm = mine < 8 ? (int)mine : 8;
  return g;
}

// A round of 256 large tiles takes 2.5 times one of small tiles.
bool large_tiles(int64_t m, int64_t n) {
  const int64_t large = ceil_div(ceil_div(m, 256) * ceil_div(n, 256), 256);
  const int64_t small = ceil_div(ceil_div(m, 128) * ceil_div(n, 128), 256);
  return 5 * large <= 2 * small;
}

hipError_t launch_words(const _Float16* A, int64_t lda, int64_t m, const StoredWeights& w,
                        int64_t K, int splits, float* sums, hipStream_t s) {
  const int wm = m <= 64 ? 1 : 2;
  const dim3 grid((unsigned)(w.cols / 128), (unsigned)splits, (unsigned)ceil_div(m, 64 * wm));
#define GPTQ_WORDS(BITS, WM)                                                                     \
  hipLaunchKernelGGL((gemm_words_kernel<BITS, WM>), grid, dim3(512), 0, s, A, lda, m, w.packed,  \
                     packed_words(w.cols, w.bits), w.rows, w.cols, K, w.scales, w.zeros,         \
                     ceil_div(w.cols, w.groupsize), w.groupsize, sums)
  if (w.bits == 4 && wm == 1) GPTQ_WORDS(4, 1);
  else if (w.bits == 4) GPTQ_WORDS(4, 2);
  else if (wm == 1) GPTQ_WORDS(8, 1);
  else GPTQ_WORDS(8, 2);
#undef GPTQ_WORDS
  return hipGetLastError();
}

template <int MODE>
hipError_t launch_gemm(const _Float16* A, int64_t lda, int64_t m, const _Float16* B, int64_t ldb,
                       int64_t n, int64_t K, const StoredWeights* w, const GemmOut& o,
                       hipStream_t s) {
  const int splits = w != nullptr ? words_splits(m, n, K) : gemm_splits(m, n, K);
  if (w != nullptr) {
    const hipError_t e = launch_words(A, lda, m, *w, K, splits, o.sums, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(gemm_reduce_kernel<MODE>, dim3((unsigned)m, (unsigned)ceil_div(n, 256)),
                       dim3(256), 0, s, splits, m, n, o);
  } else if (splits > 1) {
    const TileGrid g = gemm_grid(ceil_div(m, 128), ceil_div(n, 128));
    hipLaunchKernelGGL((gemm_nt_kernel<4, 2, 3, kSplit>),
                       dim3((unsigned)g.blocks(), (unsigned)splits), dim3(512), 0, s, A, lda, m, B,
                       ldb, n, K, g, o);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(gemm_reduce_kernel<MODE>, dim3((unsigned)m, (unsigned)ceil_div(n, 256)),
                       dim3(256), 0, s, splits, m, n, o);
  } else if (large_tiles(m, n)) {
    const TileGrid g = gemm_grid(ceil_div(m, 256), ceil_div(n, 256));
    hipLaunchKernelGGL((gemm_nt_kernel<8, 4, 2, MODE>), dim3((unsigned)g.blocks()), dim3(512), 0, s,
                       A, lda, m, B, ldb, n, K, g, o);
  } else {
    const TileGrid g = gemm_grid(ceil_div(m, 128), ceil_div(n, 128));
    hipLaunchKernelGGL((gemm_nt_kernel<4, 2, 3, MODE>), dim3((unsigned)g.blocks()), dim3(512), 0, s,
                       A, lda, m, B, ldb, n, K, g, o);
  }
  return hipGetLastError();
}

}  // namespace

// One tile of tokens (128): straight from the words, 15 to 43 us instead of 28
// to 70 for the layers 4096 x 4096 to 32000 x 2048 at 4 bits, 15 to 46 instead
// of 29 to 87 at 8.  Two tiles round the weights twice: 27 instead of 33 us at
// 160 tokens x 4096 x 4096 and 68 instead of 76 at 32000 x 2048, but 69 instead
// of 60 at 4096 x 11008, whose 172 workgroups leave a third of the CUs idle
// (the copy's tiles are finer), so they have to fill three quarters of them.
bool words_ok(int64_t m, int bits, int64_t cols, int groupsize, const int* g_idx) {
  if ((bits != 4 && bits != 8) || g_idx != nullptr || cols % 128 != 0 ||
      (groupsize % 128 != 0 && groupsize < cols))
    return false;
  if (m <= 128) return true;
  const int64_t tiles = 2 * (cols / 128), wgs = tiles < 256 ? 256 / tiles * tiles : tiles;
  return m <= 256 && 4 * wgs >= 3 * round_up(wgs, 256);
}

int words_splits(int64_t m, int64_t n, int64_t K) {
  const int64_t tiles = ceil_div(m, m <= 64 ? 64 : 128) * (n / 128);
  int64_t s = 256 / (tiles > 0 ? tiles : 1);
  if (s > K / KC / 4) s = K / KC / 4;
  return s < 1 ? 1 : (int)s;
}

int gemm_splits(int64_t m, int64_t n, int64_t K) {
  const int64_t tiles = ceil_div(m, 128) * ceil_div(n, 128);
  int64_t s = 256 / tiles;
  if (s > K / KC / 4) s = K / KC / 4;
  return s < 2 ? 1 : (int)s;
}

hipError_t launch_prepare(const uint32_t* packed, int bits, int64_t rows, int64_t cols,
                          const float* scales, const float* zeros, int groupsize, const int* g_idx,
                          int64_t kp, int64_t ldt, _Float16* wt, const PrepareAdapters* ad,
                          hipStream_t s) {
  Prepare p{};
  p.packed = packed;
  p.bits = bits;
  p.nw = packed_words(cols, bits);
  p.rows = rows;
  p.cols = cols;
  p.kp = kp;
  p.scales = scales;
  p.zeros = zeros;
  p.ngroups = ceil_div(cols, groupsize);
  p.groupsize = groupsize;
  p.g_idx = g_idx;
  p.ldt = ldt;
  p.wt = wt;
  if (ad != nullptr) {
    p.B = ad->B;
    p.count = ad->count;
    p.rank = ad->rank;
    p.ldb = ad->ldb;
    p.bt = ad->bt;
    p.A = ad->A;
    p.lda = ad->lda;
    p.at = ad->at;
    p.at_blocks = ad->count * ceil_div(cols, 256);
    p.index = ad->index;
    p.m = ad->m;
    p.chunk = grad_chunk(ad->m);
    p.max_chunks = (int)grad_chunks(ad->m, ad->count);
    p.list = ad->list;
    p.chunks = ad->chunks;
    p.ranges = ad->ranges;
    p.bt_blocks = ad->count * ceil_div(ad->ldb, 256);
  }
  const bool words = g_idx == nullptr && (bits == 4 || bits == 8) &&
                     (groupsize % (32 / bits) == 0 || groupsize >= cols);
  p.wt_x = kp / 64;
  p.wt_blocks = wt == nullptr ? 0 : p.wt_x * (words ? ceil_div(p.nw, 32) : ceil_div(cols, 64));
  const dim3 grid((unsigned)(p.count + p.bt_blocks + p.at_blocks + p.wt_blocks));
  if (grid.x == 0) return hipSuccess;
  if (words && bits == 4) hipLaunchKernelGGL(prepare_kernel<4>, grid, dim3(256), 0, s, p);
  else if (words) hipLaunchKernelGGL(prepare_kernel<8>, grid, dim3(256), 0, s, p);
  else hipLaunchKernelGGL(prepare_kernel<0>, grid, dim3(256), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_pad_rows(const _Float16* src, int64_t lds, int64_t m, int64_t K, int64_t kp,
                           int64_t ldd, _Float16* dst, hipStream_t s) {
  hipLaunchKernelGGL(pad_rows_kernel, dim3((unsigned)m, (unsigned)ceil_div(kp, 2048)), dim3(256),
                     0, s, src, lds, K, kp, ldd, dst);
  return hipGetLastError();
}

hipError_t launch_gemm_nt_f16(const _Float16* A, int64_t lda, int64_t m, const _Float16* B,
                              int64_t ldb, int64_t n, int64_t K, const StoredWeights* w,
                              const AdapterTile* ad,
                              float* sums, _Float16* C, int64_t ldc, hipStream_t s) {
  GemmOut o{};
  o.sums = sums;
  o.c16 = C;
  o.ldc = ldc;
  if (ad == nullptr) return launch_gemm<kStore>(A, lda, m, B, ldb, n, K, w, o, s);
  o.ad = *ad;
  return launch_gemm<kStoreAdapters>(A, lda, m, B, ldb, n, K, w, o, s);
}

hipError_t launch_gemm_nt_acc(const _Float16* A, int64_t lda, int64_t m, const _Float16* B,
                              int64_t ldb, int64_t n, int64_t K, const StoredWeights* w,
                              float* C32,
                              const float* scale, float* sums, _Float16* C16, int64_t ldc,
                              hipStream_t s) {
  GemmOut o{};
  o.sums = sums;
  o.c16 = C16;
  o.ldc = ldc;
  o.c32 = C32;
  o.scale = scale;
  if (C16 == nullptr) return launch_gemm<kAccumulate>(A, lda, m, B, ldb, n, K, w, o, s);
  return launch_gemm<kFinish>(A, lda, m, B, ldb, n, K, w, o, s);
}

}  // namespace gptq
