// Internal helpers shared by the gfx950 kernels and the host entry points.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/gptq.h"

namespace gptq {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int kWave = 64;

__host__ __device__ inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
__host__ __device__ inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

// Index of a lower-triangle tile (bi >= bj) in row-major order of the lower
// triangle: t = bi*(bi+1)/2 + bj.
__host__ __device__ inline void lower_tile(int64_t t, int& bi, int& bj) {
  int64_t i = (int64_t)((__builtin_sqrt(8.0 * (double)t + 1.0) - 1.0) * 0.5);
  while (i * (i + 1) / 2 > t) --i;
  while ((i + 1) * (i + 2) / 2 <= t) ++i;
  bi = (int)i;
  bj = (int)(t - i * (i + 1) / 2);
}

// ---------------------------------------------------------------- launches
// Each launcher returns hipSuccess or the launch error.
hipError_t launch_syrk_partial(const _Float16* X, int64_t ldx, int d, int64_t n, int splits,
                               int64_t kper, float* partials, hipStream_t s);
hipError_t launch_syrk_reduce(const float* partials, int d, int splits, float alpha, float* H,
                              hipStream_t s);

int syrk_splits(int64_t d, int64_t n);
int64_t syrk_kper(int64_t n, int splits);
constexpr int kSyrkTile = 256;

// fp64 Cholesky route
// perm == nullptr: A = H + lambda I; else A = P H P^T + lambda I (act-order).
// reverse: rows and columns in reversed order, A = J (...) J with J the
// reversal permutation.
hipError_t launch_damp_to_f64(const float* H, int d, double percdamp, const int* perm, bool reverse,
                              double* A, int* flag, hipStream_t s);
// Cholesky of panel k's 64x64 diagonal block, with its inverse stored in Xi
hipError_t launch_potrf_diag(double* A, int lda, int d, int k, int* flag, int info_offset,
                             double* Xi, int ldxi, hipStream_t s);
// L_ik = A_ik L_kk^-T below panel k's diagonal block
hipError_t launch_potrf_trsm(double* A, int lda, int d, int k, const double* Xi, int ldxi,
                             hipStream_t s);
// update after panel k of the first ncol 64-column blocks to its right, fused
// with the diagonal block of panel k+1
hipError_t launch_potrf_update(double* A, int lda, int d, int k, int ncol, int* flag,
                               int info_offset, double* Xi, int ldxi, hipStream_t s);
// one whole panel step (solve, update, next diagonal block) for a small
// trailing matrix
hipError_t launch_potrf_fused(double* A, int lda, int d, int k, int* flag, int info_offset,
                              double* Xi, int ldxi, hipStream_t s);
hipError_t launch_copy_panels(double* A, int lda, int d, int k0, const double* Xi, int ldxi,
                              hipStream_t s);
// rank-(k1-k0) update of A[k1:, k1:] by the finished outer block [k0, k1)
hipError_t launch_potrf_outer_update(double* A, int lda, int d, int k0, int k1, hipStream_t s);
hipError_t launch_trtri_level(const double* L, int ldl, double* X, int ldx, int d, int half,
                              hipStream_t s);
hipError_t launch_lauum(const double* X, int ldx, double* S, int lds, int d, hipStream_t s);
hipError_t launch_store_upper_f32(const double* L2, int ld2, float* Hinv, int d, hipStream_t s);
// Hinv[i][j] = X[d-1-i][d-1-j] on and above the diagonal, 0 below (fp32)
hipError_t launch_store_reversed_f32(const double* X, int ldx, float* Hinv, int d, hipStream_t s);
constexpr int kPanel = 64;
constexpr int kOuterPanel = 1024;  // columns per outer block of the two-level Cholesky

// sweep
// perm != nullptr gathers W's columns into processing order (act-order)
hipError_t launch_convert_w(const void* W, int w_dtype, int64_t rows, int64_t cols, int64_t ldw,
                            const int* perm, float* Wk, int64_t ldk, hipStream_t s);
// sweep of the block at column i1; with p0 < i1 (groups inside blocks), the
// pending errors of blocks [p0, i1) are applied to the block first
hipError_t launch_sweep_block(float* Wk, int64_t ldk, int64_t rows, int64_t cols, int i1, int p0,
                              const float* Hinv, int bits, int groupsize, uint8_t* codes,
                              float* scales, float* zeros, float* Err, float* loss_part,
                              hipStream_t s);
hipError_t launch_lazy_update(float* Wk, int64_t ldk, int64_t rows, int64_t cols, int k0, int k1,
                              int c0, int c1, const float* Err, const float* Hinv, hipStream_t s);
hipError_t launch_loss_reduce(const float* loss_part, int64_t nparts, int64_t cols,
                              float* losses, hipStream_t s);
// act-order
constexpr int64_t kStageBytes = 48 * 1024;  // largest row a gather kernel stages in LDS
hipError_t launch_act_order(const float* H, int64_t d, int* perm, hipStream_t s);
// *bad = 0 if perm is a permutation of [0, n), else 1 (inv: n ints of scratch)
hipError_t launch_perm_check(const int* perm, int64_t n, int* inv, int* bad, hipStream_t s);
hipError_t launch_perm_inverse(const int* perm, int64_t n, int* inv, hipStream_t s);
hipError_t launch_unpermute_outputs(const uint8_t* cp, int64_t rows, int64_t cols, const int* inv,
                                    uint8_t* codes, const float* lp, float* losses, int g,
                                    int* g_idx, hipStream_t s);
hipError_t launch_group_index(int64_t cols, int g, int* g_idx, hipStream_t s);
// inference with the packed codes
int64_t packed_words(int64_t cols, int bits);
hipError_t launch_pack_codes(const uint8_t* codes, int64_t rows, int64_t cols, int bits,
                             uint32_t* packed, hipStream_t s);
hipError_t launch_dequant_gemv(const _Float16* x, int64_t ldx, int64_t m, const uint32_t* packed,
                               int bits, int64_t rows, int64_t cols, const float* scales,
                               const float* zeros, int groupsize, const int* g_idx, float* y,
                               int64_t ldy, hipStream_t s);
// the forward product of a 4- or 8-bit layer for many tokens (MFMA), fp16 out
bool linear_forward_supported(int bits, int64_t m, int64_t rows, int64_t cols, int groupsize,
                              const void* x, int64_t ldx, const void* packed);
hipError_t launch_linear_forward(int bits, const _Float16* x, int64_t ldx, int64_t m,
                                 const uint32_t* packed, int64_t rows, int64_t cols,
                                 const float* scales, const float* zeros, int groupsize, bool relu,
                                 _Float16* y, int64_t ldy, hipStream_t s);
// low-rank adapters
// v[t][j] = scaling[a] * sum_k x[t][k] down[a][j][k], a = index[t] (zeros
// where index is outside [0, count)); down rows are ldd apart
struct ShrinkJob {
  const _Float16* x;
  int64_t ldx, K;
  const _Float16* down;
  int64_t ldd, stride;  // row and adapter strides
  const float* scaling;
  const int* index;
  int count, rank;
  float* v;
  int ldv;
  _Float16* xp;  // if given (the first job): x also laid out as launch_pack_x does
};
// one or two jobs (of the same ldv)
hipError_t launch_shrink(const ShrinkJob& j0, const ShrinkJob* j1, int64_t m, hipStream_t s);
// xp: x (K % 128 == 0, 16-byte aligned rows) in 16-byte pieces of 8 columns:
// [16-token tile][128-column chunk][32-column step][8-column piece][token]
hipError_t launch_pack_x(const _Float16* x, int64_t ldx, int64_t m, int64_t K, _Float16* xp,
                         hipStream_t s);
// out[a] = sum over the tokens t of adapter a of left[t][j] right[t][c]
struct GradJob {
  const float* left;
  const _Float16* right;
  int64_t ldr, N;
  int64_t R;           // N, or more where right goes on in zeros
  float* part;
  float* out;
  int64_t js, cs;
};
struct GradChunk {
  int adapter, begin, count;  // adapter -1: no chunk
};
// Tokens per partial sum: few enough that a short batch fills the CUs (160
// tokens at 4096 x 4096: 11 us in chunks of 64, 18 of 256), many enough that
// the partial sums of a long one are small beside its tokens.
constexpr int kGradChunk = 256;
inline int grad_chunk(int64_t m) { return m <= 1024 ? 64 : kGradChunk; }
constexpr int kMaxGradAdapters = 4096;   // token counts held in LDS
int64_t grad_chunks(int64_t m, int64_t count);
hipError_t launch_grads(const GradJob& g0, const GradJob& g1, int64_t m, int64_t count, int rank,
                        int ldv, const int* list, const GradChunk* chunks, const int2* ranges,
                        hipStream_t s);
hipError_t launch_fill_zero(float* p, int64_t n, hipStream_t s);
constexpr int kMaxRank = 128;
// the adapters' part of a product (adapters_dev.h)
struct AdapterTile;
// xp: x as launch_shrink or launch_pack_x laid it out, where decode_mfma_ok
bool decode_mfma_ok(const _Float16* x, int64_t ldx, int64_t m, const uint32_t* packed, int bits,
                    int64_t cols, int groupsize, const int* g_idx);
hipError_t launch_decode_adapters(const _Float16* x, const _Float16* xp, int64_t ldx, int64_t m,
                                  const uint32_t* packed, int bits, int64_t rows, int64_t cols,
                                  const float* scales, const float* zeros, int groupsize,
                                  const int* g_idx, const AdapterTile& ad, float* y, int64_t ldy,
                                  hipStream_t s);
bool gemv_fast_ok(int bits, int64_t cols, int groupsize, const int* g_idx,
                  const uint32_t* packed);
hipError_t launch_gemv_adapters(const _Float16* x, int64_t ldx, int64_t m, const uint32_t* packed,
                                int bits, int64_t rows, int64_t cols, const float* scales,
                                const float* zeros, int groupsize, const AdapterTile& ad, float* y,
                                int64_t ldy, hipStream_t s);
hipError_t launch_linear_forward_adapters(int bits, const _Float16* x, int64_t ldx, int64_t m,
                                          const uint32_t* packed, int64_t rows, int64_t cols,
                                          const float* scales, const float* zeros, int groupsize,
                                          bool relu, const AdapterTile& ad, float* sums,
                                          _Float16* y, int64_t ldy, hipStream_t s);
// splits of the input columns when the tiles leave CUs idle (1: none); their
// fp32 sums, splits x m x rows, go to the workspace
int linear_splits(int bits, int64_t m, int64_t rows, int64_t cols, int groupsize);
// whether the tiles are the wide ones, and the floats of workspace that those
// need for a copy of the scales and zeros (at most: groups of 128)
bool linear_wide(int bits, int64_t m, int64_t rows);
int64_t linear_scales(int bits, int64_t m, int64_t rows, int64_t cols);
hipError_t launch_scales(const float* scales, const float* zeros, int64_t rows, int64_t ngroups,
                         float* scales_t, float* zeros_t, int64_t pitch, hipStream_t s);
// the transposed weights, cols x kp (kp >= rows a multiple of kKPad, zeros
// behind the rows) with row pitch ldt, and the products with them
constexpr int kKPad = 64;  // K of the fp16 product, padded with zeros
struct PrepareAdapters {  // what the adapters' gradients need beside them
  const _Float16* B;
  int64_t count;
  int rank;
  int64_t ldb;      // Bt: count x rank x ldb, zeros behind the rows
  _Float16* bt;
  const _Float16* A;
  int lda;          // At: count x cols x lda, zeros behind the rank
  _Float16* at;
  const int* index;
  int64_t m;
  int* list;
  GradChunk* chunks;
  int2* ranges;     // chunks of each adapter: first, number
};
// At most the workgroups of launch_prepare; 256 times as many work-items have
// to stay below 2^32.
inline int64_t prepare_groups(int64_t rows, int64_t cols, int64_t count) {
  return ceil_div(rows, 64) * ceil_div(cols, 64) +
         count * (1 + ceil_div(round_up(rows, 8), 256) + ceil_div(cols, 256));
}
// (wt NULL: without the weights)
hipError_t launch_prepare(const uint32_t* packed, int bits, int64_t rows, int64_t cols,
                          const float* scales, const float* zeros, int groupsize, const int* g_idx,
                          int64_t kp, int64_t ldt, _Float16* wt, const PrepareAdapters* ad,
                          hipStream_t s);
// dst[t][0 .. kp) = src[t][0 .. K) and zeros, row pitch ldd
hipError_t launch_pad_rows(const _Float16* src, int64_t lds, int64_t m, int64_t K, int64_t kp,
                           int64_t ldd, _Float16* dst, hipStream_t s);
// The layer itself in B's place, where words_ok: few tokens do without a
// transposed copy.  words_splits >= 1 splits of K, all through the workspace.
struct StoredWeights {
  const uint32_t* packed;
  int bits;
  int64_t rows, cols;
  const float *scales, *zeros;
  int groupsize;
};
bool words_ok(int64_t m, int bits, int64_t cols, int groupsize, const int* g_idx);
int words_splits(int64_t m, int64_t n, int64_t K);
// C = A B^T, A m x K, B n x K (K % kKPad == 0, 16-byte aligned rows; w: not
// read)
hipError_t launch_gemm_nt_f16(const _Float16* A, int64_t lda, int64_t m, const _Float16* B,
                              int64_t ldb, int64_t n, int64_t K, const StoredWeights* w,
                              const AdapterTile* ad,
                              float* sums, _Float16* C, int64_t ldc, hipStream_t s);
// C32 += A B^T, or with C16 the finished rows: C16 = fp16(scale[t] (C32 + A B^T))
hipError_t launch_gemm_nt_acc(const _Float16* A, int64_t lda, int64_t m, const _Float16* B,
                              int64_t ldb, int64_t n, int64_t K, const StoredWeights* w,
                              float* C32,
                              const float* scale, float* sums, _Float16* C16, int64_t ldc,
                              hipStream_t s);
// splits of K when the tiles leave CUs idle (1: none); their fp32 sums,
// splits x m x n, go to the workspace
int gemm_splits(int64_t m, int64_t n, int64_t K);
// the vocabulary losses
// what is learnt: K entries per token, logits (their softmax) or one label
struct HeadTargets {
  const int* index;     // m x top
  const float* logits;  // m x top, or NULL: one label of probability 1
  int top;
  float inv_t;
};
constexpr int kMaxTop = 256;
int64_t head_tiles(int bits, int64_t m, int64_t rows);
// part[tile][t] = (max, sum exp(z - max)) over the tile's outputs, z = (x
// W_hat^T) inv_t, and zk[t][k] = z of the named outputs inside [0, rows)
hipError_t launch_head_partials(int bits, const _Float16* x, int64_t ldx, int64_t m,
                                const uint32_t* packed, int64_t rows, int64_t cols,
                                const float* scales, const float* zeros, int groupsize,
                                const HeadTargets& tg, float2* part, float* scales_t, float* zk,
                                hipStream_t s);
// P[t][r] = exp(z - lse[t]) in fp16, 0 where lse[t] is +inf and for rows <= r < ldp
hipError_t launch_head_probs(int bits, const _Float16* x, int64_t ldx, int64_t m,
                             const uint32_t* packed, int64_t rows, int64_t cols,
                             const float* scales, const float* zeros, int groupsize, float inv_t,
                             const float* lse, float* scales_t, _Float16* P, int64_t ldp,
                             hipStream_t s);
// lse and the loss from the tiles' partials and the named logits (zk: 0 where
// an entry takes no part)
hipError_t launch_head_finish(int64_t m, int64_t rows, const HeadTargets& tg, const float2* part,
                              int64_t tiles, float* loss, float* lse, float* zk, hipStream_t s);
// the gradient's terms at the named entries (see head.hip)
hipError_t launch_head_entries(const HeadTargets& tg, int64_t m, int64_t rows, const float* zk,
                               const float* lse, const float* dloss, float* lse_eff,
                               float* gscale, _Float16* dz16, float* rest, hipStream_t s);
// P[t][index - v0] = dz16 for the entries inside [v0, v0 + width)
hipError_t launch_head_scatter(const HeadTargets& tg, int64_t m, int64_t rows, int64_t v0,
                               int64_t width, const _Float16* dz16, _Float16* P, int64_t ldp,
                               hipStream_t s);
// sums[t] = sum_k rest[t][k] W_hat[index[t][k]]
hipError_t launch_head_rest(int bits, const HeadTargets& tg, int64_t m, const uint32_t* packed,
                            int64_t cols, const float* scales, const float* zeros, int groupsize,
                            const float* rest, float* sums, hipStream_t s);
constexpr int kSweepRows = 16;  // rows per sweep workgroup
constexpr int kBlock = 128;     // columns per block
constexpr int kSuperBlock = 512;  // columns per superblock of the two-level lazy update

}  // namespace gptq
