// A wave's 16 x 16 BT sums written as fp16 rows by 16-byte stores: through LDS
// of its own, 16 rows at a time (2-byte stores, 32 adjacent bytes of four rows
// each, are eight times as many).
#pragma once

#include "common.h"

namespace gptq {

#ifdef __HIPCC__
template <int BT>
struct StoreTile {
  static constexpr int kPitch = 16 * BT + 8;       // halves
  static constexpr int kBytes = 16 * kPitch * 2;   // of LDS per wave
};

// Whether 16-byte pieces of y's rows are aligned (columns start at multiples of 8).
__device__ inline bool wide_rows(const _Float16* y, int64_t ldy) {
  return ldy % 8 == 0 && (reinterpret_cast<uintptr_t>(y) & 15) == 0;
}

// v (lane (li, kg): rows 4 kg + i, column 16 b + li) to tokens t.., columns
// c..; nothing from m or n on.
template <int BT>
__device__ inline void store_rows(const f32x4 (&v)[BT], char* lds, _Float16* y, int64_t ldy,
                                  int64_t t, int64_t m, int64_t c, int64_t n, bool wide) {
  constexpr int P = StoreTile<BT>::kPitch;
  const int lane = threadIdx.x & 63, li = lane & 15, kg = lane >> 4;
  if (wide && c + 16 * BT <= n) {
    _Float16* buf = reinterpret_cast<_Float16*>(lds);
#pragma unroll
    for (int b = 0; b < BT; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) buf[(4 * kg + i) * P + 16 * b + li] = (_Float16)v[b][i];
#pragma unroll
    for (int u = 0; u < (32 * BT + 63) / 64; ++u) {
      const int p = lane + 64 * u, row = p / (2 * BT), q = p % (2 * BT);
      if (row < 16 && t + row < m)
        *reinterpret_cast<half8*>(y + (t + row) * ldy + c + 8 * q) =
            *reinterpret_cast<const half8*>(buf + row * P + 8 * q);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int b = 0; b < BT; ++b)
      if (t + 4 * kg + i < m && c + 16 * b + li < n)
        y[(t + 4 * kg + i) * ldy + c + 16 * b + li] = (_Float16)v[b][i];
}
#endif

}  // namespace gptq
