// tc_plan.h -- which tiles of a tensor-core GEMM are shared stream-K style.  Plain
// C++, so that a host test can go through the sizes without a GPU.
#pragma once

#include <stdint.h>

namespace swiglu {

struct TcPlan {
  int grid, sk_tiles, seg_max;
};

// Whole tiles round-robin, unless the last round would leave more than 3% of
// the SMs' time idle: then the (tiles mod SMs) tiles of that round (all of
// them when there are fewer tiles than SMs) are shared stream-K style.  A
// CTA's shared range is at most one tile long, so it meets at most two tiles.
// No tiles (an empty batch): nothing to share, and no share to divide by.
inline TcPlan tc_plan(int64_t tiles, int64_t kb, int nsm) {
  TcPlan p{(int)(tiles < nsm ? tiles : nsm), 0, 1};
  if (tiles < 1 || kb < 8) return p;
  const int64_t waves = (tiles + nsm - 1) / nsm;
  const double fill = (double)tiles / ((double)waves * nsm);
  if (fill >= 0.97) return p;
  p.sk_tiles = (int)(tiles >= nsm ? tiles % nsm : tiles);
  const int64_t total = (int64_t)p.sk_tiles * kb;
  p.grid = nsm;
  if (tiles < nsm && total < nsm) p.grid = (int)total;
  const int64_t range = (total + p.grid - 1) / p.grid;
  p.seg_max = (int)((range + kb - 1) / kb) + 1;
  return p;
}

}  // namespace swiglu
