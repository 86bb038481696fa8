// simt_plan.h -- how the fp32 products of linear layers are cut into tiles and
// parts.  Plain C++, so that a host test can go through the sizes without a GPU.
#pragma once

#include <stdint.h>

namespace swiglu {

constexpr int SL_BN = 128, SL_BK = 16;  // columns of a tile, k of a step

// Which tiles are split over the contraction (parts of 64 k at least), so that two
// blocks an SM are busy to the end.
struct SlPlan {
  int tm, m_tiles, n_tiles, whole, parts, per;
  int split() const { return m_tiles * n_tiles - whole; }
};
inline SlPlan sl_plan(int64_t M, int64_t N, int64_t K, int nsm) {
  SlPlan p;
  p.tm = M <= 32 ? 2 : 8;
  p.m_tiles = (int)((M + 16 * p.tm - 1) / (16 * p.tm));
  p.n_tiles = (int)((N + SL_BN - 1) / SL_BN);
  const int64_t tiles = (int64_t)p.m_tiles * p.n_tiles, room = 2 * (int64_t)nsm, rest = tiles % room;
  // Rounds of the places that the last tiles' parts take, a whole tile's being 1, and
  // the parts' way through memory (128 KB at 6 TB/s against 0.16 us a k of a tile).
  // 2816 x 1024 over 4096: 176 tiles for 304 places, 731 us whole, 436 in 5 parts.
  int64_t parts = 1;
  double best = 1.0;
  const int64_t most = rest > 0 ? 4 * room / rest : 0;
  for (int64_t n = 2; n <= most && n <= (K + 63) / 64; ++n) {
    const double cost = (double)((rest * n + room - 1) / room) / n + (double)rest * n / (7.6 * K);
    if (cost < best) {
      best = cost;
      parts = n;
    }
  }
  p.whole = (int)(parts > 1 ? tiles - rest : tiles);
  // (one step at least: with no k at all, the parts would be counted in steps of 0)
  p.per = (int)(((K + parts - 1) / parts + SL_BK - 1) / SL_BK * SL_BK);
  if (p.per < SL_BK) p.per = SL_BK;
  p.parts = (int)((K + p.per - 1) / p.per);
  if (p.parts <= 1) {
    p.parts = 1;
    p.whole = (int)tiles;
  }
  return p;
}

}  // namespace swiglu
