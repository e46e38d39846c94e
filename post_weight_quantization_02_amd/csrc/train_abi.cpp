// Host side of the adapters', the backward and the vocabulary-loss entry
// points of include/gptq.h: argument validation, workspace carving and the
// launch order of the gfx950 kernels.
#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "adapters_dev.h"

using namespace gptq;

namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxDim = 1 << 20;
constexpr int64_t kMaxElems = (int64_t)1 << 40;
constexpr int64_t kMaxTokens = (int64_t)1 << 23;  // token lists hold ints, grids 2^16 chunks
constexpr int64_t kMaxAdapters = 1 << 20;
constexpr int64_t kMaxGroups = 1 << 24;    // workgroups of 256 in a launch
constexpr int64_t kHeadTokens = 8192;      // tokens per pass of the loss's gradient

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Consecutive 256-byte aligned pieces of the workspace.
struct Carve {
  size_t at = 0;
  size_t take(int64_t n, size_t each) {
    const size_t off = at;
    at += align_up((size_t)n * each);
    return off;
  }
};

int64_t most(int64_t a, int64_t b) { return a > b ? a : b; }

int64_t scales_copy(int64_t m, int64_t rows, int64_t cols) {  // of either number of bits
  return most(linear_scales(4, m, rows, cols), linear_scales(8, m, rows, cols));
}

int rank_pitch(int rank) { return (int)round_up(rank, 16); }

// the sums of a split product
int64_t split_sums(int64_t m, int64_t n, int64_t K) {
  const int splits = gemm_splits(m, n, K);
  const int64_t copy = splits > 1 ? splits * m * n : 0;
  const int64_t words = words_ok(m, 4, n, 128, nullptr) ? words_splits(m, n, K) * m * n : 0;
  return copy > words ? copy : words;
}

// The pitch of a matrix of the workspace whose rows the fp16 product reads 64
// bytes at a time: 256 bytes more than a multiple of 128, so the rows of a
// tile start on different memory channels.
int64_t gemm_pitch(int64_t k) { return k + 128; }

struct BackwardLayout {
  int64_t kp;   // rows padded to the fp16 product's K
  int64_t ldt;  // pitch of the transposed weights and of dy's copy
  size_t wt, dyp, sums, v, dv, bt, at, list, chunks, ranges, part_a, part_b, total;
};

BackwardLayout backward_layout(int64_t m, int64_t rows, int64_t cols, int64_t count, int rank) {
  BackwardLayout L{};
  Carve c;
  L.kp = round_up(rows, kKPad);
  L.ldt = gemm_pitch(L.kp);
  L.wt = c.take(cols * L.ldt, 2);
  L.dyp = c.take(L.kp == rows ? 0 : m * L.ldt, 2);
  L.sums = c.take(split_sums(m, cols, L.kp), 4);
  if (count > 0) {
    const int64_t chunks = grad_chunks(m, count);
    L.v = c.take(m * rank_pitch(rank), 4);
    L.dv = c.take(m * rank_pitch(rank), 4);
    L.bt = c.take(count * rank * round_up(rows, 8), 2);
    L.at = c.take(count * cols * rank_pitch(rank), 2);
    L.list = c.take(m, 4);
    L.chunks = c.take(chunks, sizeof(GradChunk));
    L.ranges = c.take(count, sizeof(int2));
    L.part_a = c.take(chunks * rank * cols, 4);
    L.part_b = c.take(chunks * rank * rows, 4);
  }
  L.total = c.at;
  return L;
}

struct HeadLayout {
  int64_t tokens, width;  // tokens and vocabulary entries per pass
  size_t lse, scale, dz, rest, probs, wt, acc, sums, scales, total;
};

// A pass keeps at most 2^25 probabilities (64 MB, which the 256 MB Infinity
// Cache holds until the product reads them) and 2^26 transposed weights.
HeadLayout head_layout(int64_t m, int64_t rows, int64_t cols, int top) {
  HeadLayout L{};
  Carve c;
  L.tokens = m < kHeadTokens ? m : kHeadTokens;
  int64_t w = ((int64_t)1 << 25) / L.tokens / 256 * 256;
  const int64_t by_weights = most(((int64_t)1 << 26) / cols / 256 * 256, 256);
  if (w > by_weights) w = by_weights;
  if (w > round_up(rows, 256)) w = round_up(rows, 256);
  L.width = w;
  L.lse = c.take(m, 4);
  L.scale = c.take(m, 4);
  L.probs = c.take(L.tokens * gemm_pitch(w), 2);
  L.wt = c.take(cols * gemm_pitch(w), 2);
  L.acc = c.take(L.tokens * cols, 4);
  L.dz = c.take(m * top, 2);
  L.rest = c.take(m * top, 4);
  // the last pass over the tokens may split more than the others
  const int64_t rest = m % L.tokens;
  L.sums = c.take(most(split_sums(L.tokens, cols, w), rest > 0 ? split_sums(rest, cols, w) : 0), 4);
  // (so may the last piece of the vocabulary have another tile shape)
  const int64_t tail = rows % w, few = rest > 0 ? rest : L.tokens;
  int64_t copy = most(scales_copy(L.tokens, w, cols), scales_copy(few, w, cols));
  if (tail > 0)
    copy = most(copy, most(scales_copy(L.tokens, tail, cols), scales_copy(few, tail, cols)));
  L.scales = c.take(copy, 4);
  L.total = c.at;
  return L;
}

size_t partials_bytes(int64_t m, int64_t rows) {
  return align_up((size_t)(most(head_tiles(4, m, rows), head_tiles(8, m, rows)) * m) *
                  sizeof(float2));
}

// The tokens' v, then what the product needs beside it: the splits' sums or
// the scales' copy (many tokens), or x in the decode product's order (whole
// 64-token passes).
size_t forward_v_bytes(int64_t m, int rank) {
  return align_up((size_t)m * rank_pitch(rank) * sizeof(float));
}

size_t forward_bytes(int64_t m, int64_t rows, int64_t cols, int rank) {
  // groups of 128: the most splits a layer of these sizes can have
  const int s4 = linear_splits(4, m, rows, cols, 128), s8 = linear_splits(8, m, rows, cols, 128);
  const int splits = s4 > s8 ? s4 : s8;
  const size_t sums = splits > 1 ? (size_t)splits * m * rows * sizeof(float) : 0;
  const size_t xp = cols % 128 == 0 ? (size_t)round_up(m, 64) * cols * sizeof(_Float16) : 0;
  const size_t copy = (size_t)scales_copy(m, rows, cols) * sizeof(float);  // with one split only
  const size_t more = sums > xp ? sums : xp;
  return forward_v_bytes(m, rank) + align_up(more > copy ? more : copy);
}

bool sizes_ok(int64_t m, int64_t rows, int64_t cols, int bits, int groupsize) {
  return m >= 0 && rows >= 1 && cols >= 1 && rows <= kMaxDim && cols <= kMaxDim && bits >= 2 &&
         bits <= 8 && groupsize >= 1;
}

bool layer_ok(const uint32_t* packed, const float* scales, const float* zeros) {
  return packed != nullptr && scales != nullptr && zeros != nullptr && aligned(packed, 4) &&
         aligned(scales, 4) && aligned(zeros, 4);
}

// a matrix of m rows of n values, ld apart, of `size` bytes each
bool matrix_ok(const void* p, int64_t m, int64_t n, int64_t ld, size_t size) {
  if (m == 0) return true;  // never read
  return p != nullptr && ld >= n && m <= kMaxElems / ld && aligned(p, size);
}

bool adapters_ok(const gptq_adapters* ad, int64_t m) {
  if (ad == nullptr || ad->A == nullptr || ad->B == nullptr || ad->scaling == nullptr) return false;
  if (m > 0 && ad->index == nullptr) return false;
  if (ad->count < 1 || ad->count > kMaxAdapters || ad->rank < 1) return false;
  return aligned(ad->A, 2) && aligned(ad->B, 2) && aligned(ad->scaling, 4) && aligned(ad->index, 4);
}

gptq_status workspace_ok(const void* ws, size_t bytes, size_t need) {
  if (need > 0 && (ws == nullptr || bytes < need)) return GPTQ_ERR_WORKSPACE;
  if (need > 0 && !aligned(ws, kAlign)) return GPTQ_ERR_INVALID_ARG;
  return GPTQ_OK;
}

ShrinkJob forward_job(const gptq_adapters* ad, const void* x, int64_t ldx, int64_t cols, float* v) {
  ShrinkJob j{};
  j.x = reinterpret_cast<const _Float16*>(x);
  j.ldx = ldx;
  j.K = cols;
  j.down = reinterpret_cast<const _Float16*>(ad->A);
  j.ldd = cols;
  j.stride = (int64_t)ad->rank * cols;
  j.scaling = ad->scaling;
  j.index = ad->index;
  j.count = (int)ad->count;
  j.rank = ad->rank;
  j.v = v;
  j.ldv = rank_pitch(ad->rank);
  return j;
}

AdapterTile forward_tile(const gptq_adapters* ad, int64_t rows, const float* v) {
  AdapterTile t{};
  t.v = v;
  t.ldv = rank_pitch(ad->rank);
  t.index = ad->index;
  t.up = reinterpret_cast<const _Float16*>(ad->B);
  t.stride = rows * ad->rank;
  t.ns = ad->rank;
  t.rank = ad->rank;
  t.count = (int)ad->count;
  return t;
}

#define GPTQ_TRY(call)                             \
  do {                                             \
    if ((call) != hipSuccess) return GPTQ_ERR_HIP; \
  } while (0)

}  // namespace

extern "C" {

size_t gptq_adapters_workspace_bytes(int op, int64_t m, int64_t rows, int64_t cols, int64_t count,
                                     int rank) {
  if (m < 0 || m > kMaxTokens || rows < 1 || cols < 1 || rows > kMaxDim || cols > kMaxDim ||
      count < 0 || count > kMaxAdapters || rank < 0 || rank > kMaxRank)
    return 0;
  if ((count == 0) != (rank == 0)) return 0;
  switch (op) {
    case GPTQ_OP_FORWARD_ADAPTERS:
      return m > 0 && rank > 0 ? forward_bytes(m, rows, cols, rank) : 0;
    case GPTQ_OP_BACKWARD:
      if (m == 0 || count > kMaxGradAdapters) return 0;
      return backward_layout(m, rows, cols, count, rank).total;
    default: return 0;
  }
}

gptq_status gptq_dequant_gemm_adapters(const void* x, int64_t m, int64_t cols, int64_t ldx,
                                       const uint32_t* packed, int bits, int64_t rows,
                                       const float* scales, const float* zeros, int groupsize,
                                       const int32_t* g_idx, const gptq_adapters* ad, float* y,
                                       int64_t ldy, void* workspace, size_t workspace_bytes,
                                       void* stream) {
  if (!sizes_ok(m, rows, cols, bits, groupsize) || !layer_ok(packed, scales, zeros) ||
      !matrix_ok(x, m, cols, ldx, 2) || !matrix_ok(y, m, rows, ldy, 4) || !adapters_ok(ad, m) ||
      !aligned(g_idx, 4))
    return GPTQ_ERR_INVALID_ARG;
  if (ad->rank > kMaxRank || m > kMaxTokens) return GPTQ_ERR_UNSUPPORTED;
  if (m == 0) return GPTQ_OK;
  const gptq_status ok = workspace_ok(
      workspace, workspace_bytes,
      gptq_adapters_workspace_bytes(GPTQ_OP_FORWARD_ADAPTERS, m, rows, cols, ad->count, ad->rank));
  if (ok != GPTQ_OK) return ok;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const _Float16* xh = reinterpret_cast<const _Float16*>(x);
  float* v = reinterpret_cast<float*>(workspace);
  ShrinkJob job = forward_job(ad, x, ldx, cols, v);
  if (decode_mfma_ok(xh, ldx, m, packed, bits, cols, groupsize, g_idx))
    job.xp = reinterpret_cast<_Float16*>(reinterpret_cast<char*>(workspace) +
                                         forward_v_bytes(m, ad->rank));
  GPTQ_TRY(launch_shrink(job, nullptr, m, s));
  GPTQ_TRY(launch_decode_adapters(xh, job.xp, ldx, m, packed, bits, rows,
                                  cols, scales, zeros, groupsize, g_idx, forward_tile(ad, rows, v),
                                  y, ldy, s));
  return GPTQ_OK;
}

gptq_status gptq_linear_forward_adapters(const void* x, int64_t m, int64_t cols, int64_t ldx,
                                         const uint32_t* packed, int bits, int64_t rows,
                                         const float* scales, const float* zeros, int groupsize,
                                         int relu, const gptq_adapters* ad, void* y, int64_t ldy,
                                         void* workspace, size_t workspace_bytes, void* stream) {
  if (!sizes_ok(m, rows, cols, bits, groupsize) || !layer_ok(packed, scales, zeros) ||
      !matrix_ok(x, m, cols, ldx, 2) || !matrix_ok(y, m, rows, ldy, 2) || !adapters_ok(ad, m) ||
      (relu != 0 && relu != 1))
    return GPTQ_ERR_INVALID_ARG;
  if (ad->rank > kMaxRank || m > kMaxTokens ||
      !linear_forward_supported(bits, m, rows, cols, groupsize, x, m > 0 ? ldx : 8, packed))
    return GPTQ_ERR_UNSUPPORTED;
  if (m == 0) return GPTQ_OK;
  const gptq_status ok = workspace_ok(
      workspace, workspace_bytes,
      gptq_adapters_workspace_bytes(GPTQ_OP_FORWARD_ADAPTERS, m, rows, cols, ad->count, ad->rank));
  if (ok != GPTQ_OK) return ok;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  float* v = reinterpret_cast<float*>(workspace);
  GPTQ_TRY(launch_shrink(forward_job(ad, x, ldx, cols, v), nullptr, m, s));
  GPTQ_TRY(launch_linear_forward_adapters(bits, reinterpret_cast<const _Float16*>(x), ldx, m,
                                          packed, rows, cols, scales, zeros, groupsize, relu == 1,
                                          forward_tile(ad, rows, v),
                                          reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) +
                                                                   forward_v_bytes(m, ad->rank)),
                                          reinterpret_cast<_Float16*>(y), ldy, s));
  return GPTQ_OK;
}

gptq_status gptq_linear_backward(const void* dy, int64_t m, int64_t rows, int64_t lddy,
                                 const uint32_t* packed, int bits, int64_t cols,
                                 const float* scales, const float* zeros, int groupsize,
                                 const int32_t* g_idx, const gptq_adapters* ad, const void* x,
                                 int64_t ldx, void* dx, int64_t lddx, float* dA, float* dB,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  if (!sizes_ok(m, rows, cols, bits, groupsize) || !layer_ok(packed, scales, zeros) ||
      !matrix_ok(dy, m, rows, lddy, 2) || !matrix_ok(dx, m, cols, lddx, 2) || !aligned(g_idx, 4))
    return GPTQ_ERR_INVALID_ARG;
  if (ad != nullptr && (!adapters_ok(ad, m) || !matrix_ok(x, m, cols, ldx, 2) || dA == nullptr ||
                        dB == nullptr || !aligned(dA, 4) || !aligned(dB, 4)))
    return GPTQ_ERR_INVALID_ARG;
  if (m > kMaxTokens || (ad != nullptr && (ad->rank > kMaxRank || ad->count > kMaxGradAdapters)))
    return GPTQ_ERR_UNSUPPORTED;
  if (prepare_groups(rows, cols, ad != nullptr ? ad->count : 0) >= kMaxGroups)
    return GPTQ_ERR_UNSUPPORTED;
  // dy goes into LDS by 16-byte loads, unless it is copied to padded rows first
  if (m > 0 && rows % kKPad == 0 && (!aligned(dy, 16) || lddy % 8 != 0)) return GPTQ_ERR_UNSUPPORTED;
  const int64_t count = ad != nullptr ? ad->count : 0;
  const int rank = ad != nullptr ? ad->rank : 0;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (m == 0) {
    if (ad != nullptr) {
      GPTQ_TRY(launch_fill_zero(dA, count * rank * cols, s));
      GPTQ_TRY(launch_fill_zero(dB, count * rank * rows, s));
    }
    return GPTQ_OK;
  }
  const BackwardLayout L = backward_layout(m, rows, cols, count, rank);
  const gptq_status ok = workspace_ok(workspace, workspace_bytes, L.total);
  if (ok != GPTQ_OK) return ok;
  char* ws = reinterpret_cast<char*>(workspace);
  _Float16* wt = reinterpret_cast<_Float16*>(ws + L.wt);
  const _Float16* g = reinterpret_cast<const _Float16*>(dy);
  int64_t ldg = lddy;
  const StoredWeights stored{packed, bits, rows, cols, scales, zeros, groupsize};
  const bool words = words_ok(m, bits, cols, groupsize, g_idx);
  if (L.kp != rows) {
    _Float16* p = reinterpret_cast<_Float16*>(ws + L.dyp);
    GPTQ_TRY(launch_pad_rows(g, lddy, m, rows, L.kp, L.ldt, p, s));
    g = p;
    ldg = L.ldt;
  }
  AdapterTile tile{};
  if (ad != nullptr) {
    float* v = reinterpret_cast<float*>(ws + L.v);
    float* dv = reinterpret_cast<float*>(ws + L.dv);
    _Float16* bt = reinterpret_cast<_Float16*>(ws + L.bt);
    _Float16* at = reinterpret_cast<_Float16*>(ws + L.at);
    int* list = reinterpret_cast<int*>(ws + L.list);
    GradChunk* chunks = reinterpret_cast<GradChunk*>(ws + L.chunks);
    int2* ranges = reinterpret_cast<int2*>(ws + L.ranges);
    const int64_t ldt = round_up(rows, 8);
    const PrepareAdapters pa{reinterpret_cast<const _Float16*>(ad->B), count, rank, ldt, bt,
                             reinterpret_cast<const _Float16*>(ad->A), rank_pitch(rank), at,
                             ad->index, m, list, chunks, ranges};
    GPTQ_TRY(launch_prepare(packed, bits, rows, cols, scales, zeros, groupsize, g_idx, L.kp, L.ldt,
                            words ? nullptr : wt, &pa, s));
    const ShrinkJob jx = forward_job(ad, x, ldx, cols, v);
    ShrinkJob jy = jx;  // dv = s dy B, over the rows
    jy.x = g;
    jy.ldx = ldg;
    jy.K = ldt;  // dy's copy holds zeros behind the rows, as Bt does
    jy.down = bt;
    jy.ldd = ldt;
    jy.stride = rank * ldt;
    jy.v = dv;
    GPTQ_TRY(launch_shrink(jx, &jy, m, s));
    GradJob ga{}, gb{};
    ga.left = dv;
    ga.right = reinterpret_cast<const _Float16*>(x);
    ga.ldr = ldx;
    ga.N = cols;
    ga.R = cols;
    ga.part = reinterpret_cast<float*>(ws + L.part_a);
    ga.out = dA;
    ga.js = cols;
    ga.cs = 1;
    gb.left = v;
    gb.right = g;
    gb.ldr = ldg;
    gb.N = rows;
    gb.R = ldt;
    gb.part = reinterpret_cast<float*>(ws + L.part_b);
    gb.out = dB;
    gb.js = 1;
    gb.cs = rank;
    GPTQ_TRY(launch_grads(ga, gb, m, count, rank, rank_pitch(rank), list, chunks, ranges, s));
    tile = forward_tile(ad, rows, dv);
    tile.up = at;
    tile.stride = cols * rank_pitch(rank);
    tile.ns = rank_pitch(rank);
  } else if (!words) {
    GPTQ_TRY(launch_prepare(packed, bits, rows, cols, scales, zeros, groupsize, g_idx, L.kp, L.ldt,
                            wt, nullptr, s));
  }
  GPTQ_TRY(launch_gemm_nt_f16(g, ldg, m, wt, L.ldt, cols, L.kp, words ? &stored : nullptr,
                              ad != nullptr ? &tile : nullptr,
                              reinterpret_cast<float*>(ws + L.sums),
                              reinterpret_cast<_Float16*>(dx), lddx, s));
  return GPTQ_OK;
}

size_t gptq_head_workspace_bytes(int op, int64_t m, int64_t rows, int64_t cols, int top) {
  if (m < 1 || top < 1 || top > kMaxTop || m > kMaxTokens || rows < 1 || cols < 1 ||
      rows > kMaxDim || cols > kMaxDim)
    return 0;
  switch (op) {
    case GPTQ_OP_HEAD_LOSS:
      return partials_bytes(m, rows) + align_up((size_t)scales_copy(m, rows, cols) * sizeof(float));
    case GPTQ_OP_HEAD_BACKWARD: return head_layout(m, rows, cols, top).total;
    default: return 0;
  }
}

}  // extern "C"

namespace {

// The targets' checks, and what the kernels take of them; `teacher` NULL for
// labels (top = 1, temperature 1).
bool targets(const int32_t* index, const float* teacher, bool distill, int top, float temperature,
             int64_t m, HeadTargets* tg) {
  if (top < 1 || !(temperature > 0.f) || !isfinite(temperature) || !isfinite(1.f / temperature))
    return false;
  if (m > 0 && (index == nullptr || (distill && teacher == nullptr))) return false;
  if (!aligned(index, 4) || !aligned(teacher, 4)) return false;
  tg->index = index;
  tg->logits = teacher;
  tg->top = top;
  tg->inv_t = 1.f / temperature;
  return true;
}

gptq_status head_forward(const void* h, int64_t m, int64_t cols, int64_t ldh,
                         const uint32_t* packed, int bits, int64_t rows, const float* scales,
                         const float* zeros, int groupsize, const int32_t* index,
                         const float* teacher, bool distill, int top, float temperature,
                         float* loss, float* lse, float* zk, void* workspace,
                         size_t workspace_bytes, void* stream) {
  HeadTargets tg{};
  if (!sizes_ok(m, rows, cols, bits, groupsize) || !layer_ok(packed, scales, zeros) ||
      !matrix_ok(h, m, cols, ldh, 2) || !targets(index, teacher, distill, top, temperature, m, &tg))
    return GPTQ_ERR_INVALID_ARG;
  if (m > 0 && (loss == nullptr || lse == nullptr || zk == nullptr || !aligned(loss, 4) ||
                !aligned(lse, 4) || !aligned(zk, 4)))
    return GPTQ_ERR_INVALID_ARG;
  if (m > kMaxTokens || top > kMaxTop ||
      !linear_forward_supported(bits, m, rows, cols, groupsize, h, m > 0 ? ldh : 8, packed))
    return GPTQ_ERR_UNSUPPORTED;
  if (m == 0) return GPTQ_OK;
  const gptq_status ok = workspace_ok(workspace, workspace_bytes,
                                      gptq_head_workspace_bytes(GPTQ_OP_HEAD_LOSS, m, rows, cols,
                                                                top));
  if (ok != GPTQ_OK) return ok;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const _Float16* x = reinterpret_cast<const _Float16*>(h);
  float2* part = reinterpret_cast<float2*>(workspace);
  GPTQ_TRY(launch_head_partials(bits, x, ldh, m, packed, rows, cols, scales, zeros, groupsize,
                                tg, part,
                                reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) +
                                                         partials_bytes(m, rows)),
                                zk, s));
  GPTQ_TRY(launch_head_finish(m, rows, tg, part, head_tiles(bits, m, rows), loss, lse, zk, s));
  return GPTQ_OK;
}

gptq_status head_backward(const void* h, int64_t m, int64_t cols, int64_t ldh,
                          const uint32_t* packed, int bits, int64_t rows, const float* scales,
                          const float* zeros, int groupsize, const int32_t* index,
                          const float* teacher, bool distill, int top, float temperature,
                          const float* lse, const float* zk, const float* dloss, void* dh,
                          int64_t lddh, void* workspace, size_t workspace_bytes, void* stream) {
  HeadTargets tg{};
  if (!sizes_ok(m, rows, cols, bits, groupsize) || !layer_ok(packed, scales, zeros) ||
      !matrix_ok(h, m, cols, ldh, 2) || !matrix_ok(dh, m, cols, lddh, 2) ||
      !targets(index, teacher, distill, top, temperature, m, &tg))
    return GPTQ_ERR_INVALID_ARG;
  if (m > 0 && (lse == nullptr || zk == nullptr || dloss == nullptr || !aligned(lse, 4) ||
                !aligned(zk, 4) || !aligned(dloss, 4)))
    return GPTQ_ERR_INVALID_ARG;
  if (m > kMaxTokens || top > kMaxTop ||
      !linear_forward_supported(bits, m, rows, cols, groupsize, h, m > 0 ? ldh : 8, packed))
    return GPTQ_ERR_UNSUPPORTED;
  if (m == 0) return GPTQ_OK;
  const HeadLayout L = head_layout(m, rows, cols, top);
  const gptq_status ok = workspace_ok(workspace, workspace_bytes, L.total);
  if (ok != GPTQ_OK) return ok;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  char* ws = reinterpret_cast<char*>(workspace);
  float* lse_eff = reinterpret_cast<float*>(ws + L.lse);
  float* gscale = reinterpret_cast<float*>(ws + L.scale);
  _Float16* P = reinterpret_cast<_Float16*>(ws + L.probs);
  _Float16* wt = reinterpret_cast<_Float16*>(ws + L.wt);
  float* acc = reinterpret_cast<float*>(ws + L.acc);
  const int64_t nw = packed_words(cols, bits), ng = ceil_div(cols, groupsize);
  _Float16* dz = reinterpret_cast<_Float16*>(ws + L.dz);
  float* rest = reinterpret_cast<float*>(ws + L.rest);
  GPTQ_TRY(launch_head_entries(tg, m, rows, zk, lse, dloss, lse_eff, gscale, dz, rest, s));
  for (int64_t t0 = 0; t0 < m; t0 += L.tokens) {
    const int64_t mt = m - t0 < L.tokens ? m - t0 : L.tokens;
    const _Float16* x = reinterpret_cast<const _Float16*>(h) + t0 * ldh;
    _Float16* out = reinterpret_cast<_Float16*>(dh) + t0 * lddh;
    HeadTargets tt = tg;
    tt.index += t0 * top;
    if (tt.logits != nullptr) tt.logits += t0 * top;
    GPTQ_TRY(launch_head_rest(bits, tt, mt, packed, cols, scales, zeros, groupsize, rest + t0 * top,
                              acc, s));
    for (int64_t v0 = 0; v0 < rows; v0 += L.width) {
      const int64_t w = rows - v0 < L.width ? rows - v0 : L.width;
      const int64_t wp = round_up(w, kKPad), ld = gemm_pitch(wp);
      const bool last = v0 + w == rows;
      GPTQ_TRY(launch_head_probs(bits, x, ldh, mt, packed + v0 * nw, w, cols, scales + v0 * ng,
                                 zeros + v0 * ng, groupsize, tg.inv_t, lse_eff + t0,
                                 reinterpret_cast<float*>(ws + L.scales), P, ld, s));
      GPTQ_TRY(launch_head_scatter(tt, mt, rows, v0, w, dz + t0 * top, P, ld, s));
      const StoredWeights stored{packed + v0 * nw, bits, w, cols, scales + v0 * ng, zeros + v0 * ng,
                                 groupsize};
      const bool words = words_ok(mt, bits, cols, groupsize, nullptr);
      if (!words)
        GPTQ_TRY(launch_prepare(packed + v0 * nw, bits, w, cols, scales + v0 * ng, zeros + v0 * ng,
                                groupsize, nullptr, wp, ld, wt, nullptr, s));
      GPTQ_TRY(launch_gemm_nt_acc(P, ld, mt, wt, ld, cols, wp, words ? &stored : nullptr, acc,
                                  gscale + t0,
                                  reinterpret_cast<float*>(ws + L.sums), last ? out : nullptr, lddh,
                                  s));
    }
  }
  return GPTQ_OK;
}

}  // namespace

extern "C" {

gptq_status gptq_head_loss(const void* h, int64_t m, int64_t cols, int64_t ldh,
                           const uint32_t* packed, int bits, int64_t rows, const float* scales,
                           const float* zeros, int groupsize, const int32_t* target, float* loss,
                           float* lse, float* target_logit, void* workspace,
                           size_t workspace_bytes, void* stream) {
  return head_forward(h, m, cols, ldh, packed, bits, rows, scales, zeros, groupsize, target, nullptr,
                      false, 1, 1.f, loss, lse, target_logit, workspace, workspace_bytes, stream);
}

gptq_status gptq_head_loss_backward(const void* h, int64_t m, int64_t cols, int64_t ldh,
                                    const uint32_t* packed, int bits, int64_t rows,
                                    const float* scales, const float* zeros, int groupsize,
                                    const int32_t* target, const float* lse,
                                    const float* target_logit, const float* dloss, void* dh,
                                    int64_t lddh, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  return head_backward(h, m, cols, ldh, packed, bits, rows, scales, zeros, groupsize, target,
                       nullptr, false, 1, 1.f, lse, target_logit, dloss, dh, lddh, workspace,
                       workspace_bytes, stream);
}

gptq_status gptq_head_distill(const void* h, int64_t m, int64_t cols, int64_t ldh,
                              const uint32_t* packed, int bits, int64_t rows, const float* scales,
                              const float* zeros, int groupsize, const int32_t* top_index,
                              const float* top_logits, int top, float temperature, float* loss,
                              float* lse, float* student_logits, void* workspace,
                              size_t workspace_bytes, void* stream) {
  return head_forward(h, m, cols, ldh, packed, bits, rows, scales, zeros, groupsize, top_index,
                      top_logits, true, top, temperature, loss, lse, student_logits, workspace,
                      workspace_bytes, stream);
}

gptq_status gptq_head_distill_backward(const void* h, int64_t m, int64_t cols, int64_t ldh,
                                       const uint32_t* packed, int bits, int64_t rows,
                                       const float* scales, const float* zeros, int groupsize,
                                       const int32_t* top_index, const float* top_logits, int top,
                                       float temperature, const float* lse,
                                       const float* student_logits, const float* dloss, void* dh,
                                       int64_t lddh, void* workspace, size_t workspace_bytes,
                                       void* stream) {
  return head_backward(h, m, cols, ldh, packed, bits, rows, scales, zeros, groupsize, top_index,
                       top_logits, true, top, temperature, lse, student_logits, dloss, dh, lddh,
                       workspace, workspace_bytes, stream);
}

}  // extern "C"
