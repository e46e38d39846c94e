// The decode product of many requests, y_t = W_hat x_t + s_a B_a (A_a x_t),
// a = index[t], for a few tokens (fp32 y): the stored weights streamed once
// for all of them, each token's low-rank part (v = s A x formed beforehand)
// added where the sums end.  One token with 2, 4 or 8 bits stays with the
// product of infer.hip.
#include "adapters_dev.h"

namespace gptq {
namespace {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));

// ------------------------------------------------------------- MFMA, 4 and 8 bits
// 16 TT tokens x 16 BT outputs per workgroup; its eight waves take every
// eighth chunk of 128 columns (so together 1024 adjacent columns of each row
// at a time) and their sums are added in wave order.  Per chunk
// v_mfma_f32_16x16x32_f16 adds the exact products x * q, a second one against
// ones sum x, and the chunk enters as s * (sum x q - z sum x), for any fp32
// zero.
//
// x comes from the L2 for every workgroup (8 times the weights' bytes at 32
// tokens), so it is laid out first (with v) as the fragments read it: 1 KB per
// instruction, where rows of x would put 16 lanes' 64-byte pieces on one L2
// channel (8 KB apart at 4096 columns; 31 against 26 us at 11008 x 4096, 32
// tokens), and the packed words' own order, lane group kg on columns 32 kg..,
// every lane on a segment of its own (37 us).  The 4-bit words arrive as one
// 16-byte load per lane, word j of lane group kg, and two exchanges between
// lane groups transpose them to word kg of step j; four chunks' words are in
// flight per wave, and one load brings four chunks' scales (a load each cost
// 4 of 17 us at 2 tokens).  Bound by the latency of the weights: 4096 x 4096
// takes 8.3 us at 32 tokens, one round of workgroups.
constexpr int kWaves = 8;
constexpr int kDeep = 4;  // chunks of weights in flight per wave

// 8 codes of one 4-bit word as exact fp16, in column order (1024 + q and
// 1024 + 16 q by bit operations, then one packed FMA).
__device__ inline half8 codes4(uint32_t w) {
  const h2 mul = {(_Float16)1.f, (_Float16)0.0625f};
  const h2 off = {(_Float16)-1024.f, (_Float16)-64.f};
  half8 r;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const uint32_t b =
        __builtin_amdgcn_perm(w, w, (12u << 24) | ((uint32_t)p << 16) | (12u << 8) | p);
    const h2 h = __builtin_bit_cast(h2, (b & 0x00F0000Fu) | 0x64006400u) * mul + off;
    r[2 * p] = h[0];
    r[2 * p + 1] = h[1];
  }
  return r;
}

// 8 codes of two 8-bit words as exact fp16 (0x64 bytes beside the codes').
__device__ inline half8 codes8(uint32_t w0, uint32_t w1) {
  const h2 off = {(_Float16)-1024.f, (_Float16)-1024.f};
  const uint32_t words[2] = {w0, w1};
  half8 r;
#pragma unroll
  for (int v = 0; v < 2; ++v)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const uint32_t sel = 0x04000400u | ((uint32_t)(2 * p + 1) << 16) | (uint32_t)(2 * p);
      const h2 h =
          __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, words[v], sel)) + off;
      r[4 * v + 2 * p] = h[0];
      r[4 * v + 2 * p + 1] = h[1];
    }
  return r;
}

// Words w[j] of lane group kg -> word kg of lane group j's.
__device__ inline void transpose_groups(uint32_t (&w)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto p = __builtin_amdgcn_permlane32_swap(w[i], w[i + 2], false, false);
    w[i] = p[0];
    w[i + 2] = p[1];
  }
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const auto p = __builtin_amdgcn_permlane16_swap(w[i], w[i + 1], false, false);
    w[i] = p[0];
    w[i + 1] = p[1];
  }
}

template <int BITS, int TT, int BT>
__global__ __launch_bounds__(64 * kWaves, 2) void decode_mfma_kernel(
    const _Float16* __restrict__ xp, int m, const uint32_t* __restrict__ packed, int64_t nw,
    int64_t rows, int64_t cols, const float* __restrict__ scales,
    const float* __restrict__ zeros, int64_t ngroups, int groupsize, float* __restrict__ y,
    int64_t ldy, AdapterTile ad) {
  constexpr int WPC = 4 * BITS;          // words per chunk and row
  constexpr int NW = BITS == 4 ? 4 : 8;  // words per lane, row and chunk
  constexpr int OUT = TT * BT * 256;
  constexpr int PER = (OUT + 64 * kWaves - 1) / (64 * kWaves);
  __shared__ float part[kWaves][TT * 16][16 * BT + 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = lane & 15, kg = lane >> 4;
  const int64_t r0 = (int64_t)blockIdx.x * 16 * BT;
  const int nch = (int)(cols / 128);
  const int cb = nch * wave / kWaves, ce = nch * (wave + 1) / kWaves;  // this wave's chunks
  const uint32_t* wrow[BT];
  const float *srow[BT], *zrow[BT];
#pragma unroll
  for (int b = 0; b < BT; ++b) {
    const int64_t rr = min(r0 + 16 * b + n, rows - 1);
    wrow[b] = packed + rr * nw + (BITS == 4 ? 4 * kg : 2 * kg);
    srow[b] = scales + rr * ngroups;
    zrow[b] = zeros + rr * ngroups;
  }
  uint32_t wv[kDeep][BT][NW];
  float sv[BT], zv[BT];  // lane group kg: the block's chunk kg
  half8 xv[2][TT][4];
  auto fetch_w = [&](int slot, int c) {  // chunks past the end read the last one
    const int64_t cc = min(c, nch - 1);
#pragma unroll
    for (int b = 0; b < BT; ++b) {
      if constexpr (BITS == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(wrow[b] + WPC * cc);
        wv[slot][b][0] = v.x;
        wv[slot][b][1] = v.y;
        wv[slot][b][2] = v.z;
        wv[slot][b][3] = v.w;
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint2 v = *reinterpret_cast<const uint2*>(wrow[b] + WPC * cc + 8 * q);
          wv[slot][b][2 * q] = v.x;
          wv[slot][b][2 * q + 1] = v.y;
        }
      }
    }
  };
  auto fetch_sz = [&](int c) {
    const int64_t g = (int64_t)min(c + kg, nch - 1) * 128 / groupsize;
#pragma unroll
    for (int b = 0; b < BT; ++b) {
      sv[b] = srow[b][g];
      zv[b] = zrow[b][g];
    }
  };
  auto fetch_x = [&](int slot, int c) {
    const int64_t cc = min(c, nch - 1);
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        xv[slot][t][q] = *reinterpret_cast<const half8*>(xp + ((t * nch + cc) * 4 + q) * 512 + 8 * lane);
  };
#pragma unroll
  for (int i = 0; i < kDeep; ++i) fetch_w(i, cb + i);
  fetch_sz(cb);
  fetch_x(0, cb);
  fetch_x(1, cb + 1);
  // this thread's outputs' low-rank part, its loads beside the first chunks'
  const bool vec = vec_up(ad);
  float low[PER];
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int o = tid + 64 * kWaves * u, tok = o / (16 * BT);
    const int64_t r = r0 + o % (16 * BT);
    low[u] = (o < OUT && tok < m && r < rows) ? low_rank(ad, tok, r, vec) : 0.f;
  }
  const half8 ones = {(_Float16)1.f, (_Float16)1.f, (_Float16)1.f, (_Float16)1.f,
                      (_Float16)1.f, (_Float16)1.f, (_Float16)1.f, (_Float16)1.f};
  f32x4 acc[TT][BT];
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int b = 0; b < BT; ++b) acc[t][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int c0 = cb; c0 < ce; c0 += 4) {
    float sc[BT], zc[BT];
#pragma unroll
    for (int b = 0; b < BT; ++b) {
      sc[b] = sv[b];
      zc[b] = zv[b];
    }
    if (c0 + 4 < ce) fetch_sz(c0 + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = c0 + i;
      if (c < ce) {
        f32x4 d[TT][BT], dx[TT];
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          dx[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int b = 0; b < BT; ++b) d[t][b] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        if constexpr (BITS == 4) {
#pragma unroll
          for (int b = 0; b < BT; ++b) transpose_groups(wv[i % kDeep][b]);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
          for (int t = 0; t < TT; ++t)
            dx[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(xv[i & 1][t][q], ones, dx[t], 0, 0, 0);
#pragma unroll
          for (int b = 0; b < BT; ++b) {
            half8 qv;
            if constexpr (BITS == 4) qv = codes4(wv[i % kDeep][b][q]);
            else qv = codes8(wv[i % kDeep][b][2 * q], wv[i % kDeep][b][2 * q + 1]);
#pragma unroll
            for (int t = 0; t < TT; ++t)
              d[t][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(xv[i & 1][t][q], qv, d[t][b], 0, 0, 0);
          }
        }
        if (c + kDeep < ce) fetch_w(i % kDeep, c + kDeep);
        if (c + 2 < ce) fetch_x(i & 1, c + 2);
#pragma unroll
        for (int b = 0; b < BT; ++b) {
          const float s = __shfl(sc[b], n + 16 * i, 64), z = __shfl(zc[b], n + 16 * i, 64);
#pragma unroll
          for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[t][b][e] =
                  __builtin_fmaf(s, __builtin_fmaf(-z, dx[t][e], d[t][b][e]), acc[t][b][e]);
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int b = 0; b < BT; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) part[wave][16 * t + 4 * kg + e][16 * b + n] = acc[t][b][e];
  __syncthreads();
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int o = tid + 64 * kWaves * u, tok = o / (16 * BT), rw = o % (16 * BT);
    if (o >= OUT || tok >= m || r0 + rw >= rows) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += part[w][tok][rw];
    y[(int64_t)tok * ldy + r0 + rw] = v + low[u];
  }
}

// ------------------------------------------------------------ any bits, any groups
// One output row per wave, up to MT tokens; x of 4096 columns or so at a time
// sits in LDS (zeros past the row's end), a lane takes every 64th packed word,
// and W_hat is formed in fp32.  Bound by latency and the unpacking: 5 tokens x
// 1003 x 2000 at 3 bits take 10.6 us (12.9 with one load of x in flight).
template <int BITS, int MT>
__global__ __launch_bounds__(256) void decode_rows_kernel(
    const _Float16* __restrict__ x, int64_t ldx, int m, const uint32_t* __restrict__ packed,
    int64_t nw, int64_t rows, int64_t cols, const float* __restrict__ scales,
    const float* __restrict__ zeros, int64_t ngroups, int groupsize, const int* __restrict__ g_idx,
    float* __restrict__ y, int64_t ldy, AdapterTile ad) {
  constexpr int K = 32 / BITS;
  constexpr uint32_t MASK = (1u << BITS) - 1u;
  constexpr int TW = 4096 / K;  // words per pass
  constexpr int U = 16 / MT;
  __shared__ _Float16 xs[MT][TW * K];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t r = (int64_t)blockIdx.x * 4 + wave;
  const int64_t rr = min(r, rows - 1);
  float acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = 0.f;
  for (int64_t w0 = 0; w0 < nw; w0 += TW) {
    const int words = (int)min((int64_t)TW, nw - w0);
    __syncthreads();
    for (int c0 = tid; c0 < words * K; c0 += 256 * U) {  // 16 loads in flight
      _Float16 v[U][MT];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const int64_t col = w0 * K + c0 + 256 * u;
          v[u][t] = t < m && col < cols ? x[t * ldx + col] : (_Float16)0.f;
        }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int t = 0; t < MT; ++t)
          if (t < m && c0 + 256 * u < words * K) xs[t][c0 + 256 * u] = v[u][t];
    }
    __syncthreads();
    for (int w = lane; w < words; w += 64) {
      const uint32_t q = packed[rr * nw + w0 + w];
      const int c0 = (int)((w0 + w) * K);
      float wv[K];
      if (g_idx == nullptr && groupsize >= K) {  // a word meets at most two groups
        const int g = c0 / groupsize;
        const int g1 = (int)min((int64_t)g + 1, ngroups - 1);
        const int64_t edge = (int64_t)(g + 1) * groupsize;
        const float s0 = scales[rr * ngroups + g], z0 = zeros[rr * ngroups + g];
        const float s1 = scales[rr * ngroups + g1], z1 = zeros[rr * ngroups + g1];
#pragma unroll
        for (int j = 0; j < K; ++j) {
          const bool next = c0 + j >= edge;
          wv[j] = ((float)((q >> (BITS * j)) & MASK) - (next ? z1 : z0)) * (next ? s1 : s0);
        }
      } else {
#pragma unroll
        for (int j = 0; j < K; ++j) {
          const int64_t c = min((int64_t)c0 + j, cols - 1);
          int64_t g = g_idx != nullptr ? (int64_t)g_idx[c] : c / groupsize;
          g = g < 0 ? 0 : g >= ngroups ? ngroups - 1 : g;
          wv[j] = ((float)((q >> (BITS * j)) & MASK) - zeros[rr * ngroups + g]) *
                  scales[rr * ngroups + g];
        }
      }
#pragma unroll
      for (int t = 0; t < MT; ++t)
        if (t < m)
#pragma unroll
          for (int j = 0; j < K; ++j)
            acc[t] = __builtin_fmaf((float)xs[t][w * K + j], wv[j], acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    if (t >= m) break;
    const int a = ad.index[t];
    if (a >= 0 && a < ad.count) {
      const _Float16* up = ad.up + a * ad.stride + rr * ad.ns;
      for (int j = lane; j < ad.rank; j += 64)
        acc[t] = __builtin_fmaf(ad.v[(int64_t)t * ad.ldv + j], (float)up[j], acc[t]);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) acc[t] += __shfl_xor(acc[t], o, 64);
    if (lane == 0 && r < rows) y[t * ldy + r] = acc[t];
  }
}

AdapterTile from_token(const AdapterTile& ad, int64_t t0) {
  AdapterTile b = ad;
  b.v += t0 * b.ldv;
  b.index += t0;
  return b;
}

struct DecodeCall {
  const _Float16 *x, *xp;
  int64_t ldx, m;
  const uint32_t* packed;
  int64_t rows, cols;
  const float *scales, *zeros;
  int groupsize;
  const int* g_idx;
  float* y;
  int64_t ldy;
};

template <int BITS, int TT, int BT>
void decode_mfma(const DecodeCall& c, const AdapterTile& ad, int64_t t0, int mt, hipStream_t s) {
  hipLaunchKernelGGL((decode_mfma_kernel<BITS, TT, BT>), dim3((unsigned)ceil_div(c.rows, 16 * BT)),
                     dim3(64 * kWaves), 0, s, c.xp + t0 * c.cols, mt, c.packed,
                     packed_words(c.cols, BITS), c.rows, c.cols, c.scales, c.zeros,
                     ceil_div(c.cols, c.groupsize), c.groupsize, c.y + t0 * c.ldy, c.ldy,
                     from_token(ad, t0));
}

template <int BITS>
hipError_t decode_mfma_passes(const DecodeCall& c, const AdapterTile& ad, hipStream_t s) {
  for (int64_t t0 = 0; t0 < c.m; t0 += 64) {
    const int mt = (int)(c.m - t0 < 64 ? c.m - t0 : 64);
    // 16 outputs per workgroup, one workgroup per CU at a time: 8.3 us a round
    // of 4096 outputs at 32 tokens; 48 outputs take 19 us a round of 12288
    const bool wide = c.rows > 8192;
    if (mt <= 16) {
      if (wide) decode_mfma<BITS, 1, 3>(c, ad, t0, mt, s);
      else decode_mfma<BITS, 1, 1>(c, ad, t0, mt, s);
    } else if (mt <= 32) {
      bool done = false;
      if constexpr (BITS == 4) {  // 8 bits: the registers do not hold 48 outputs
        if (wide) decode_mfma<BITS, 2, 3>(c, ad, t0, mt, s);
        done = wide;
      }
      if (!done) decode_mfma<BITS, 2, 1>(c, ad, t0, mt, s);
    } else {
      decode_mfma<BITS, 4, 1>(c, ad, t0, mt, s);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int BITS>
hipError_t decode_rows(const DecodeCall& c, const AdapterTile& ad, hipStream_t s) {
  const dim3 grid((unsigned)ceil_div(c.rows, 4));
  for (int64_t t0 = 0; t0 < c.m; t0 += 8) {
    const int mt = (int)(c.m - t0 < 8 ? c.m - t0 : 8);
#define GPTQ_ROWS(MT)                                                                           \
  hipLaunchKernelGGL((decode_rows_kernel<BITS, MT>), grid, dim3(256), 0, s, c.x + t0 * c.ldx,   \
                     c.ldx, mt, c.packed, packed_words(c.cols, BITS), c.rows, c.cols, c.scales, \
                     c.zeros, ceil_div(c.cols, c.groupsize), c.groupsize, c.g_idx,              \
                     c.y + t0 * c.ldy, c.ldy, from_token(ad, t0))
    if (mt <= 2) GPTQ_ROWS(2);
    else GPTQ_ROWS(8);
#undef GPTQ_ROWS
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

// two tokens or more, 4 or 8 bits, whole 128-column chunks inside groups,
// 16-byte aligned rows
bool decode_mfma_ok(const _Float16* x, int64_t ldx, int64_t m, const uint32_t* packed, int bits,
                    int64_t cols, int groupsize, const int* g_idx) {
  return m >= 2 && (bits == 4 || bits == 8) && g_idx == nullptr && cols % 128 == 0 &&
         (groupsize % 128 == 0 || groupsize >= cols) && ldx % 8 == 0 &&
         (reinterpret_cast<uintptr_t>(x) & 15) == 0 &&
         (reinterpret_cast<uintptr_t>(packed) & 15) == 0;
}

hipError_t launch_decode_adapters(const _Float16* x, const _Float16* xp, int64_t ldx, int64_t m,
                                  const uint32_t* packed, int bits, int64_t rows, int64_t cols,
                                  const float* scales, const float* zeros, int groupsize,
                                  const int* g_idx, const AdapterTile& ad, float* y, int64_t ldy,
                                  hipStream_t s) {
  const DecodeCall c{x, xp, ldx, m, packed, rows, cols, scales, zeros, groupsize, g_idx, y, ldy};
  if (decode_mfma_ok(x, ldx, m, packed, bits, cols, groupsize, g_idx))
    return bits == 4 ? decode_mfma_passes<4>(c, ad, s) : decode_mfma_passes<8>(c, ad, s);
  if (gemv_fast_ok(bits, cols, groupsize, g_idx, packed))
    return launch_gemv_adapters(x, ldx, m, packed, bits, rows, cols, scales, zeros, groupsize, ad, y,
                                ldy, s);
  switch (bits) {
    case 2: return decode_rows<2>(c, ad, s);
    case 3: return decode_rows<3>(c, ad, s);
    case 4: return decode_rows<4>(c, ad, s);
    case 5: return decode_rows<5>(c, ad, s);
    case 6: return decode_rows<6>(c, ad, s);
    case 7: return decode_rows<7>(c, ad, s);
    case 8: return decode_rows<8>(c, ad, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace gptq
