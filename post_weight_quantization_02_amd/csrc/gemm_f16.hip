// The gradient through a stored layer, dx = dy W_hat, and the products of the
// vocabulary losses' gradient: the stored weights are written once in fp16
// with the layer's outputs along the fast axis (launch_dequant_transposed),
// and a dense fp16 product C = A B^T over that axis follows.
//
// W_hat = (code - zero) * scale is formed in fp32 and rounded to fp16 once
// (at most 2^-11 of its size, 2^-25 below 2^-14); the products are exact in
// fp32 and summed there.
#include "adapters_dev.h"
#include "tile_grid.h"

namespace gptq {
namespace {

// ------------------------------------------------------- transposed weights
// 4 and 8 bits, every word inside a group.  A lane takes one word of eight
// adjacent rows (4 or 8 columns x 8 rows), so its outputs are whole 16-byte
// pieces of the transposed rows; the lanes of a wave are eight such row groups
// x eight words, which makes 128 adjacent bytes of eight rows per store.
// Bound by the store: 90 MB at 11008 x 4096.
template <int BITS>
__global__ __launch_bounds__(256) void dequant_transposed_words_kernel(
    const uint32_t* __restrict__ packed, int64_t nw, int64_t rows, int64_t cols, int64_t kp,
    const float* __restrict__ scales, const float* __restrict__ zeros, int64_t ngroups,
    int groupsize, int64_t ldt, _Float16* __restrict__ Wt) {
  constexpr int K = 32 / BITS;
  constexpr uint32_t MASK = (1u << BITS) - 1u;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t r0 = (int64_t)blockIdx.x * 64 + 8 * (lane & 7);
  const int64_t w = (int64_t)blockIdx.y * 32 + 8 * wave + (lane >> 3);
  if (w >= nw || r0 >= kp) return;
  const int64_t g = w * K / groupsize;
  uint32_t q[8];
  float s[8], z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = min(r0 + i, rows - 1);
    q[i] = packed[r * nw + w];
    s[i] = scales[r * ngroups + g];
    z[i] = zeros[r * ngroups + g];
  }
#pragma unroll
  for (int j = 0; j < K; ++j) {
    half8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float f = ((float)((q[i] >> (BITS * j)) & MASK) - z[i]) * s[i];
      v[i] = (_Float16)(r0 + i < rows ? f : 0.f);
    }
    if (w * K + j < cols) *reinterpret_cast<half8*>(Wt + (w * K + j) * ldt + r0) = v;
  }
}

// Any bits and groups: 64 rows x 64 columns per workgroup through LDS.
__global__ __launch_bounds__(256) void dequant_transposed_kernel(
    const uint32_t* __restrict__ packed, int bits, int64_t nw, int64_t rows, int64_t cols,
    const float* __restrict__ scales, const float* __restrict__ zeros, int64_t ngroups,
    int groupsize, const int* __restrict__ g_idx, int64_t ldt, _Float16* __restrict__ Wt) {
  // (blockIdx.x covers the padded rows)
  __shared__ __attribute__((aligned(16))) _Float16 tile[64][64 + 8];
  const int64_t r0 = (int64_t)blockIdx.x * 64, c0 = (int64_t)blockIdx.y * 64;
  const int tid = threadIdx.x, k = 32 / bits;
  const uint32_t mask = (1u << bits) - 1u;
  {
    const int64_t c = c0 + (tid & 63);
    const int64_t cc = c < cols ? c : cols - 1;
    int64_t g = g_idx != nullptr ? (int64_t)g_idx[cc] : cc / groupsize;
    g = g < 0 ? 0 : g >= ngroups ? ngroups - 1 : g;
    const int64_t w = cc / k;
    const int sh = bits * (int)(cc % k);
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
      const int row = (tid >> 6) * 16 + i;
      const int64_t r = r0 + row;
      float v = 0.f;
      if (r < rows && c < cols) {
        const float q = (float)((packed[r * nw + w] >> sh) & mask);
        v = (q - zeros[r * ngroups + g]) * scales[r * ngroups + g];
      }
      tile[tid & 63][row] = (_Float16)v;
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int o = tid + 256 * u, c = o >> 3, p = o & 7;
    if (c0 + c < cols)
      *reinterpret_cast<uint4*>(Wt + (c0 + c) * ldt + r0 + 8 * p) =
          *reinterpret_cast<const uint4*>(&tile[c][8 * p]);
  }
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
  bool first;          // c32 holds nothing yet
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
#pragma unroll
  for (int a = 0; a < AT; ++a)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t t = tw + 16 * a + 4 * kg + i;
      if (t >= m) continue;
      const float scale = MODE == kFinish ? o.scale[t] : 1.f;
#pragma unroll
      for (int b = 0; b < BT; ++b) {
        const int64_t c = nw + 16 * b + li;
        if (c >= n) continue;
        float v = acc[a][b][i];
        if constexpr (MODE == kSplit) {
          o.sums[((int64_t)blockIdx.y * m + t) * n + c] = v;
          continue;
        }
        if constexpr (MODE == kAccumulate || MODE == kFinish)
          if (!o.first) v += o.c32[t * n + c];
        if constexpr (MODE == kAccumulate) o.c32[t * n + c] = v;
        else o.c16[t * o.ldc + c] = (_Float16)(MODE == kFinish ? scale * v : v);
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
  if constexpr (MODE == kStoreAdapters) {
    const int a = o.ad.index[t];
    if (a >= 0 && a < o.ad.count) {
      const _Float16* up = o.ad.up + a * o.ad.stride + c * o.ad.ns;
      float low = 0.f;
#pragma unroll 8
      for (int j = 0; j < o.ad.rank; ++j)
        low = __builtin_fmaf(o.ad.v[t * o.ad.ldv + j], (float)up[j * o.ad.js], low);
      v += low;
    }
  }
  if constexpr (MODE == kAccumulate || MODE == kFinish)
    if (!o.first) v += o.c32[t * n + c];
  if constexpr (MODE == kAccumulate) o.c32[t * n + c] = v;
  else o.c16[t * o.ldc + c] = (_Float16)(MODE == kFinish ? o.scale[t] * v : v);
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

template <int MODE>
hipError_t launch_gemm(const _Float16* A, int64_t lda, int64_t m, const _Float16* B, int64_t ldb,
                       int64_t n, int64_t K, const GemmOut& o, hipStream_t s) {
  const int splits = gemm_splits(m, n, K);
  if (splits > 1) {
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

int gemm_splits(int64_t m, int64_t n, int64_t K) {
  const int64_t tiles = ceil_div(m, 128) * ceil_div(n, 128);
  int64_t s = 256 / tiles;
  if (s > K / KC / 4) s = K / KC / 4;
  return s < 2 ? 1 : (int)s;
}

hipError_t launch_dequant_transposed(const uint32_t* packed, int bits, int64_t rows, int64_t cols,
                                     const float* scales, const float* zeros, int groupsize,
                                     const int* g_idx, int64_t kp, int64_t ldt, _Float16* Wt,
                                     hipStream_t s) {
  const int64_t nw = packed_words(cols, bits), ng = ceil_div(cols, groupsize);
  const dim3 words((unsigned)(kp / 64), (unsigned)ceil_div(nw, 32));
  if (bits == 4 && g_idx == nullptr && (groupsize % 8 == 0 || groupsize >= cols))
    hipLaunchKernelGGL(dequant_transposed_words_kernel<4>, words, dim3(256), 0, s, packed, nw, rows,
                       cols, kp, scales, zeros, ng, groupsize, ldt, Wt);
  else if (bits == 8 && g_idx == nullptr && (groupsize % 4 == 0 || groupsize >= cols))
    hipLaunchKernelGGL(dequant_transposed_words_kernel<8>, words, dim3(256), 0, s, packed, nw, rows,
                       cols, kp, scales, zeros, ng, groupsize, ldt, Wt);
  else
    hipLaunchKernelGGL(dequant_transposed_kernel,
                       dim3((unsigned)(kp / 64), (unsigned)ceil_div(cols, 64)), dim3(256), 0, s,
                       packed, bits, nw, rows, cols, scales, zeros, ng, groupsize, g_idx, ldt, Wt);
  return hipGetLastError();
}

hipError_t launch_pad_rows(const _Float16* src, int64_t lds, int64_t m, int64_t K, int64_t kp,
                           int64_t ldd, _Float16* dst, hipStream_t s) {
  hipLaunchKernelGGL(pad_rows_kernel, dim3((unsigned)m, (unsigned)ceil_div(kp, 2048)), dim3(256),
                     0, s, src, lds, K, kp, ldd, dst);
  return hipGetLastError();
}

hipError_t launch_gemm_nt_f16(const _Float16* A, int64_t lda, int64_t m, const _Float16* B,
                              int64_t ldb, int64_t n, int64_t K, const AdapterTile* ad,
                              float* sums, _Float16* C, int64_t ldc, hipStream_t s) {
  GemmOut o{};
  o.sums = sums;
  o.c16 = C;
  o.ldc = ldc;
  if (ad == nullptr) return launch_gemm<kStore>(A, lda, m, B, ldb, n, K, o, s);
  o.ad = *ad;
  return launch_gemm<kStoreAdapters>(A, lda, m, B, ldb, n, K, o, s);
}

hipError_t launch_gemm_nt_acc(const _Float16* A, int64_t lda, int64_t m, const _Float16* B,
                              int64_t ldb, int64_t n, int64_t K, bool first, float* C32,
                              const float* scale, float* sums, _Float16* C16, int64_t ldc,
                              hipStream_t s) {
  GemmOut o{};
  o.sums = sums;
  o.c16 = C16;
  o.ldc = ldc;
  o.c32 = C32;
  o.scale = scale;
  o.first = first;
  if (C16 == nullptr) return launch_gemm<kAccumulate>(A, lda, m, B, ldb, n, K, o, s);
  return launch_gemm<kFinish>(A, lda, m, B, ldb, n, K, o, s);
}

}  // namespace gptq
