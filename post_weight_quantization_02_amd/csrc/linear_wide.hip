// The layer's product from its stored form for many tokens with what the
// training and scoring calls do with its sums (linear_tails.h): 256 tokens x
// 256 outputs per workgroup.
//
// Eight waves, two along the tokens by four along the outputs, each 8 x 4
// tiles of v_mfma_f32_16x16x32_f16.  A wave reads 8 x-fragments per 32 MFMAs
// from LDS, half of what a wave of 128 tokens x 32 outputs needs (there the
// LDS is as busy as the matrix units), at the price of building every B
// fragment twice.  B is (q - z), exact in fp16, as in linear_mfma.hip.
//
// Group scales: there is no room for a second set of sums, so the running sums
// are kept in units of the current group's scale: when a group begins they
// are multiplied by (last scale / its scale), and by the last scale at the
// end.  Each change costs two roundings (the quotient's and the product's),
// so an output is within (cols + 2 ngroups + 2) 2^-24 sum |x| |q - z| s of
// the exact sum.  A group whose scale is 0 (or so small that the quotient
// leaves fp32) adds nothing: its B is zero and the sums keep their unit.
//
// 64 columns per stage, three stages in LDS (126 KB at 4 bits, 150 KB at 8)
// by direct loads; rows of x swizzled as in the fp16 product (gemm_f16.hip).
// The scales and zeros come group by group from a copy with the outputs along
// the fast axis (launch_scales): from the stored order every one of a stage's
// 512 values is a cache line of its own, twice the lines that x takes.
#include "linear_tails.h"

namespace gptq {
namespace {

constexpr int KC = 64;  // input columns per stage
constexpr int TM = 256, TN = 256, NWAVE = 8, AT = 8, BT = 4;
constexpr int X_BYTES = TM * KC * 2;  // 32 KB
constexpr float kTinyScale = 0x1p-60f;

template <int BITS>
struct Wide {
  static constexpr int RB = KC * BITS / 8;       // packed bytes of one output row per stage
  static constexpr int PPR = RB / 16;            // 16-byte pieces of it
  static constexpr int W_BYTES = TN * RB;        // 8 or 16 KB
  static constexpr int WU = W_BYTES / 1024 / NWAVE;
  static constexpr int STAGE = X_BYTES + W_BYTES + 2 * TN * 4;
  static constexpr int LPS = 4 + WU + 1;         // direct loads per wave and stage
  static constexpr int NW = BITS / 2;            // words per lane, output and stage
  // The 16-byte pieces of a packed row change places with the row, so that a
  // fragment read meets every bank once: 8 bytes of 32 lanes (rows of 32
  // bytes, 4 bits), 16 bytes of 16 lanes (rows of 64 bytes, 8 bits).
  __device__ static int piece(int row, int p) {
    return BITS == 4 ? p ^ ((row >> 3) & 1) : p ^ ((row >> 2) & 3);
  }
};

// The 16-byte pieces of a row of x (128 bytes) are permuted by the row: the
// fp16 product's (row >> 1) & 7 with its bits turned, since here lane group kg
// reads piece 2 kg + s and not 4 s + kg.
__device__ inline int x_swizzle(int row) {
  const int r = (row >> 1) & 7;
  return ((r << 1) | (r >> 2)) & 7;
}

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
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

// (q - z) for 8 codes: of one 4-bit word (1024 + q and 1024 + 16 q by bit
// operations, one packed FMA), or of two 8-bit words (1024 + q by bytes of
// 0x64).  mul = off = 0 makes it 0.
__device__ inline half8 minus_zero4(uint32_t w, half2_t mul, half2_t off) {
  half8 r;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const uint32_t b =
        __builtin_amdgcn_perm(w, w, (12u << 24) | ((uint32_t)p << 16) | (12u << 8) | p);
    const half2_t h = __builtin_bit_cast(half2_t, (b & 0x00F0000Fu) | 0x64006400u) * mul + off;
    r[2 * p] = h[0];
    r[2 * p + 1] = h[1];
  }
  return r;
}

__device__ inline half8 minus_zero8(uint32_t w0, uint32_t w1, half2_t mul, half2_t off) {
  const uint32_t words[2] = {w0, w1};
  half8 r;
#pragma unroll
  for (int v = 0; v < 2; ++v)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const uint32_t sel = 0x04000400u | ((uint32_t)(2 * p + 1) << 16) | (uint32_t)(2 * p);
      const half2_t h =
          __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, words[v], sel)) * mul + off;
      r[4 * v + 2 * p] = h[0];
      r[4 * v + 2 * p + 1] = h[1];
    }
  return r;
}

// The chunk of 64 columns of a stage and its place in its scale group (gk
// chunks long), going around at the row's end.
struct Cursor {
  int chunk, in, grp;
  __device__ void advance(int gk, int end) {
    ++chunk;
    if (++in == gk) {
      in = 0;
      ++grp;
    }
    if (chunk == end) chunk = in = grp = 0;
  }
};

template <int BITS>
struct Loads {
  uint32_t x[4], w[Wide<BITS>::WU], sz;
};

template <int BITS>
__device__ inline void issue(const char* xb, const char* wb, const char* szb, int64_t szp,
                             const Loads<BITS>& l, const Cursor& c, char* st, int wave) {
  using L = Wide<BITS>;
  const uint32_t cx = (uint32_t)c.chunk * (KC * 2), cw = (uint32_t)c.chunk * L::RB;
#pragma unroll
  for (int u = 0; u < 4; ++u)
    __builtin_amdgcn_global_load_lds((const void*)(xb + (l.x[u] + cx)),
                                     (lds_void*)(st + 1024 * (wave + NWAVE * u)), 16, 0, 0);
#pragma unroll
  for (int u = 0; u < L::WU; ++u)
    __builtin_amdgcn_global_load_lds((const void*)(wb + (l.w[u] + cw)),
                                     (lds_void*)(st + X_BYTES + 1024 * (wave + NWAVE * u)), 16, 0,
                                     0);
  __builtin_amdgcn_global_load_lds((const void*)(szb + (int64_t)c.grp * szp + l.sz),
                                   (lds_void*)(st + X_BYTES + L::W_BYTES + 256 * wave), 4, 0, 0);
}

// One stage: wait for it, publish it, start the loads of the stage two further
// on, then the two K steps of its 64 columns.  Lane group kg takes columns
// 16 kg + 8 s .. of step s, so its codes of both steps are adjacent words.
template <int BITS>
__device__ inline void stage_step(int k, int nk, const char* cur, char* nxt, const char* xb,
                                  const char* wb, const char* szb, int64_t szp,
                                  const Loads<BITS>& l, int gk, Cursor& use, Cursor& iss,
                                  int wave, int xo, int wo, int so,
                                  f32x4 (&acc)[AT][BT], float (&unit)[BT], half2_t (&mul)[BT],
                                  half2_t (&off)[BT]) {
  using L = Wide<BITS>;
  if (k + 1 < nk) wait_vm<L::LPS>();
  else wait_vm<0>();
  lds_barrier();
  const char* ws = cur + X_BYTES + wo;
  uint32_t w[BT][L::NW];
#pragma unroll
  for (int b = 0; b < BT; ++b) {
    if constexpr (BITS == 4) {
      const uint2 v = *reinterpret_cast<const uint2*>(ws + 16 * L::RB * b);
      w[b][0] = v.x;
      w[b][1] = v.y;
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(ws + 16 * L::RB * b);
      w[b][0] = v.x;
      w[b][1] = v.y;
      w[b][2] = v.z;
      w[b][3] = v.w;
    }
  }
  if (use.in == 0) {  // a group begins
    const char* ss = cur + X_BYTES + L::W_BYTES + so;
#pragma unroll
    for (int b = 0; b < BT; ++b) {
      const float s = *reinterpret_cast<const float*>(ss + 64 * b);
      const float z = *reinterpret_cast<const float*>(ss + TN * 4 + 64 * b);
      const bool none = __builtin_fabsf(s) < kTinyScale;
      const float ratio = none ? 1.f : unit[b] / s;
      unit[b] = none ? unit[b] : s;
      const _Float16 lo = BITS == 4 ? (_Float16)0.0625f : (_Float16)1.f;
      const float zhi = BITS == 4 ? -64.f - z : -1024.f - z;
      mul[b] = none ? half2_t{(_Float16)0.f, (_Float16)0.f} : half2_t{(_Float16)1.f, lo};
      off[b] = none ? half2_t{(_Float16)0.f, (_Float16)0.f}
                    : half2_t{(_Float16)(-1024.f - z), (_Float16)zhi};
#pragma unroll
      for (int a = 0; a < AT; ++a)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[a][b][i] *= ratio;
    }
  }
  use.advance(gk, nk);
  if (k + 2 < nk) {
    issue<BITS>(xb, wb, szb, szp, l, iss, nxt, wave);
    iss.advance(gk, nk);
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    half8 bf[BT];
#pragma unroll
    for (int b = 0; b < BT; ++b) {
      if constexpr (BITS == 4) bf[b] = minus_zero4(w[b][s], mul[b], off[b]);
      else bf[b] = minus_zero8(w[b][2 * s], w[b][2 * s + 1], mul[b], off[b]);
    }
#pragma unroll
    for (int a = 0; a < AT; ++a) {
      const half8 af = *reinterpret_cast<const half8*>(cur + (xo ^ (16 * s)) + 2048 * a);
#pragma unroll
      for (int b = 0; b < BT; ++b)
        acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(af, bf[b], acc[a][b], 0, 0, 0);
    }
  }
}

template <int BITS, bool RELU, int TAIL>
__global__ __launch_bounds__(64 * NWAVE, 1) void linear_wide_kernel(LinearCall c, int64_t nw,
                                                                    int64_t ngroups, int gk,
                                                                    TileGrid grid, Tail tail) {
  using L = Wide<BITS>;
  __shared__ __attribute__((aligned(1024))) char st0[L::STAGE];
  __shared__ __attribute__((aligned(1024))) char st1[L::STAGE];
  __shared__ __attribute__((aligned(1024))) char st2[L::STAGE];
  int64_t tm, tn;
  if (!tile_of(grid, blockIdx.x, tm, tn)) return;
  const int xcd = (int)(blockIdx.x % kXcds);
  const int64_t t0 = tm * TM, n0 = tn * TN, m = c.m, rows = c.rows;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3, li = lane & 15, kg = lane >> 4;

  // byte offsets of this lane's direct loads (256 rows of at most 2^24 bytes)
  Loads<BITS> l;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int row = 8 * (wave + NWAVE * u) + (lane >> 3);
    l.x[u] = (uint32_t)((min(t0 + row, m - 1) - t0) * c.ldx * 2 +
                        16 * ((lane & 7) ^ x_swizzle(row)));
  }
#pragma unroll
  for (int u = 0; u < L::WU; ++u) {
    const int row = (64 / L::PPR) * (wave + NWAVE * u) + lane / L::PPR;
    l.w[u] = (uint32_t)((min(n0 + row, rows - 1) - n0) * nw * 4 +
                        16 * L::piece(row, lane % L::PPR));
  }
  l.sz = (uint32_t)((min(n0 + 64 * (wave & 3) + lane, rows - 1) - n0) * 4);
  const char* xb = reinterpret_cast<const char*>(c.x + t0 * c.ldx);
  const char* wb = reinterpret_cast<const char*>(c.packed + n0 * nw);
  const char* szb = reinterpret_cast<const char*>((wave < 4 ? c.scales_t : c.zeros_t) + n0);
  const int64_t szp = c.pitch_t * 4;

  // LDS offsets of this lane's fragments (a-tile a: + 2048 a, step s: ^ 16 s)
  const int xo = (128 * wm + li) * 128 + 16 * ((2 * kg) ^ x_swizzle(li));
  const int wo = (64 * wn + li) * L::RB +
                 (BITS == 4 ? 16 * L::piece(li, kg >> 1) + 8 * (kg & 1) : 16 * L::piece(li, kg));
  const int so = 4 * (64 * wn + li);

  f32x4 acc[AT][BT];
#pragma unroll
  for (int a = 0; a < AT; ++a)
#pragma unroll
    for (int b = 0; b < BT; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  float unit[BT];
  half2_t mul[BT], off[BT];
#pragma unroll
  for (int b = 0; b < BT; ++b) unit[b] = 1.f;

  const int nk = (int)(c.cols / KC);
  const int g0 = grid.xm == kXcds ? 0 : (int)(ngroups * xcd / kXcds);  // see linear_mfma.hip
  Cursor use{g0 * gk, 0, g0}, iss = use;
  issue<BITS>(xb, wb, szb, szp, l, iss, st0, wave);
  iss.advance(gk, nk);
  if (nk > 1) {
    issue<BITS>(xb, wb, szb, szp, l, iss, st1, wave);
    iss.advance(gk, nk);
  }
  for (int k = 0; k < nk; k += 3) {
    stage_step<BITS>(k, nk, st0, st2, xb, wb, szb, szp, l, gk, use, iss, wave, xo, wo, so, acc, unit, mul,
                     off);
    if (k + 1 < nk)
      stage_step<BITS>(k + 1, nk, st1, st0, xb, wb, szb, szp, l, gk, use, iss, wave, xo, wo, so, acc,
                       unit, mul, off);
    if (k + 2 < nk)
      stage_step<BITS>(k + 2, nk, st2, st1, xb, wb, szb, szp, l, gk, use, iss, wave, xo, wo, so, acc,
                       unit, mul, off);
  }
#pragma unroll
  for (int a = 0; a < AT; ++a)
#pragma unroll
    for (int b = 0; b < BT; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[a][b][i] *= unit[b];

  tile_tail<RELU, TAIL, AT, BT, 2, 4>(acc, tail, c, t0, n0, tn, wm, wn, st0, st1);
}

template <int BITS, bool RELU, int TAIL>
hipError_t launch_bits(const LinearCall& c, const Tail& tail, hipStream_t s) {
  const int64_t g = c.groupsize >= c.cols ? c.cols : c.groupsize;
  const TileGrid grid = linear_grid(ceil_div(c.m, TM), ceil_div(c.rows, TN));
  hipLaunchKernelGGL((linear_wide_kernel<BITS, RELU, TAIL>), dim3((unsigned)grid.blocks()),
                     dim3(64 * NWAVE), 0, s, c, c.cols * BITS / 32, ceil_div(c.cols, g),
                     (int)(g / KC), grid, tail);
  return hipGetLastError();
}

// (rows x groups) -> (groups x pitch), scales then zeros
__global__ __launch_bounds__(256) void scales_kernel(const float* __restrict__ scales,
                                                     const float* __restrict__ zeros, int64_t rows,
                                                     int64_t ngroups, float* __restrict__ scales_t,
                                                     float* __restrict__ zeros_t, int64_t pitch) {
  __shared__ float tile[32][33];
  const float* src = blockIdx.z == 0 ? scales : zeros;
  float* dst = blockIdx.z == 0 ? scales_t : zeros_t;
  const int64_t r0 = (int64_t)blockIdx.x * 32, g0 = (int64_t)blockIdx.y * 32;
  const int lo = threadIdx.x & 31, hi = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    if (r0 + hi + i < rows && g0 + lo < ngroups) tile[hi + i][lo] = src[(r0 + hi + i) * ngroups + g0 + lo];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    if (g0 + hi + i < ngroups && r0 + lo < rows) dst[(g0 + hi + i) * pitch + r0 + lo] = tile[lo][hi + i];
}

}  // namespace

hipError_t launch_scales(const float* scales, const float* zeros, int64_t rows, int64_t ngroups,
                         float* scales_t, float* zeros_t, int64_t pitch, hipStream_t s) {
  hipLaunchKernelGGL(scales_kernel,
                     dim3((unsigned)ceil_div(rows, 32), (unsigned)ceil_div(ngroups, 32), 2),
                     dim3(256), 0, s, scales, zeros, rows, ngroups, scales_t, zeros_t, pitch);
  return hipGetLastError();
}

template <bool RELU, int TAIL>
hipError_t launch_linear_wide(int bits, const LinearCall& c, const Tail& tail, hipStream_t s) {
  return bits == 4 ? launch_bits<4, RELU, TAIL>(c, tail, s) : launch_bits<8, RELU, TAIL>(c, tail, s);
}
template hipError_t launch_linear_wide<true, kAdapters>(int, const LinearCall&, const Tail&,
                                                        hipStream_t);
template hipError_t launch_linear_wide<false, kAdapters>(int, const LinearCall&, const Tail&,
                                                         hipStream_t);
template hipError_t launch_linear_wide<false, kPartials>(int, const LinearCall&, const Tail&,
                                                         hipStream_t);
template hipError_t launch_linear_wide<false, kProbs>(int, const LinearCall&, const Tail&,
                                                      hipStream_t);

}  // namespace gptq
