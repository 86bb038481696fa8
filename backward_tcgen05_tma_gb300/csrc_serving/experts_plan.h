// experts_plan.h -- shared memory of the experts kernels: token lists, sums on
// their way, the warps' rings.  Plain C++, so that a host test can go through
// the sizes without a GPU.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define SWIGLU_HD __host__ __device__
#else
#define SWIGLU_HD
#endif

namespace swiglu {

constexpr int WX_MAX_STAGES = 8;
// What a block takes as a rule (the rest of an SM's 256 KB caches the token
// rows), and the most where that leaves a ring of one stage, in which nothing
// would be fetched ahead (64 tokens over 8 of 64 16-bit experts of 2048/1024: 160.0
// us, with two stages 158.4): both with 1024 bytes for the ring's alignment, beside
// static shared memory of 1 KB.
constexpr int WX_SMEM = 200 * 1024, WX_SMEM_MOST = 224 * 1024;

// Entries (an expert's runs of at most `per` of its assignments) and bytes of
// the lists of M topk assignments.
SWIGLU_HD inline int ft_max_entries(int M, int topk, int E, int per) {
  const int a = M * topk, b = (E < a ? E : a) + a / per;
  return a < b ? a : b;
}
SWIGLU_HD inline int ft_lists_bytes(int M, int topk, int E, int per) {
  const int b = 16 + E * 12 + ft_max_entries(M, topk, E, per) * 8 + M * topk * 14;
  return (b + 127) & ~127;
}

struct WxPlan {
  int run;                        // items of a run (gate/up)
  int list_off, red_off, ring_off;
  int stages;                     // of a warp's ring
  int bytes;                      // of dynamic shared memory
};

// nt: 8-token columns of a pass; stage: bytes of a warp's stage; most: items of
// a block (gate/up).
inline WxPlan wx_plan(int warps, int nt, int stage, bool combine, int M, int topk, int E, int64_t most) {
  WxPlan p;
  p.run = (int)(most < 64 / nt ? most : 64 / nt);
  p.list_off = 0;
  p.red_off = ft_lists_bytes(M, topk, E, 8 * nt);
  p.ring_off = p.red_off + (combine ? warps * M * 64 : (p.run + warps - 1) * nt * 512);
  const int ring = warps * stage;
  p.stages = (WX_SMEM - p.ring_off) / ring;
  if (p.stages < 2) p.stages = (WX_SMEM_MOST - 1024 - p.ring_off) / ring < 2 ? p.stages : 2;
  if (p.stages > WX_MAX_STAGES) p.stages = WX_MAX_STAGES;
  p.bytes = p.ring_off + p.stages * ring + 1024;
  return p;
}

}  // namespace swiglu
