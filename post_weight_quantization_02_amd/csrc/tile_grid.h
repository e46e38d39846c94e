// Which tiles of a product an XCD works on, and in which order.  Workgroup b
// runs on XCD b % 8.  The XCDs form an xm x (8 / xm) grid over the token and
// output tiles; an XCD walks its token tiles in groups of gm, and within a
// group output tile by output tile, so the ~32 workgroups it runs at once
// share a block of both operands in its L2.
#pragma once

#include "common.h"

namespace gptq {

constexpr int kXcds = 8;

struct TileGrid {
  int64_t ntm, ntn;
  int xm, gm;

  // workgroups, some of them without a tile: every XCD gets the same whole
  // number of gm-token-tile groups
  int64_t blocks() const {
    return kXcds * round_up(ceil_div(ntm, xm), gm) * ceil_div(ntn, kXcds / xm);
  }
};

#ifdef __HIPCC__
__device__ inline bool tile_of(const TileGrid& g, int64_t bid, int64_t& tm, int64_t& tn) {
  const int xcd = (int)(bid % kXcds);
  const int64_t local = bid / kXcds;
  const int xi = xcd % g.xm, xj = xcd / g.xm, xn = kXcds / g.xm;
  const int64_t ntj = (g.ntn + xn - 1) / xn;
  const int64_t grp = local / (g.gm * ntj), idx = local % (g.gm * ntj);
  tm = (grp * g.gm + idx % g.gm) * g.xm + xi;
  tn = (idx / g.gm) * xn + xj;
  return tm < g.ntm && tn < g.ntn;
}
#endif

}  // namespace gptq
