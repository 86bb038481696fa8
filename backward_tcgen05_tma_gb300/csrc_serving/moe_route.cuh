// moe_route.cuh -- the router of a mixture-of-experts layer for a few tokens:
//   l[t, e] = sum_d X[t, d] Wr[e, d] (fp32),   p = softmax over e,
//   the topk largest l of each token (a tie goes to the lower index),
//   weight = scale * p, or with `norm` scale * p / (sum of the chosen p).
//
// The cost is reading Wr and the latency of doing so, not arithmetic: a
// cluster of up to 8 blocks shares 8 tokens, each block taking E / 8 experts
// (16 per mma.sync tile, its 8 warps splitting d), so that no SM reads more
// than an eighth of Wr.  The logits meet in the first block's shared memory,
// where one warp per token picks the experts.  Products of two 32-element
// runs of d go through the tensor core; the runs are added in fp32.
// Measured: 2048 x 64 experts, 1 to 64 tokens, 3.4 us in front of the experts'
// kernels (11.3 us as a call of its own from Python), all of it latency: two
// rounds of loads, the cluster's exchange, a warp's topk passes.
#pragma once

#include "fewtok.cuh"

namespace swiglu {

constexpr int RT_TOKENS = 8;    // tokens of a cluster
constexpr int RT_CLUSTER = 8;   // blocks of a cluster, at most
constexpr int RT_THREADS = 256;

struct RtArgs {
  const uint8_t* X;   // [M, D]
  const uint8_t* Wr;  // [E, D]
  int* idx;           // [M, topk]
  float* wts;         // [M, topk]
  int M, D, E, topk, norm;
  int per_block;      // experts of a block
  float scale;
  int* err;           // cleared here (first kernel of a call), or null
#ifdef SWIGLU_DEBUG
  DbgWin dbg;         // idx, wts, X, Wr
#endif
};

// Order of the logits as unsigned numbers: NaN above everything (as a softmax
// over them is NaN whatever is chosen), the two zeros alike; 0 is below all.
__device__ __forceinline__ uint32_t rt_key(float v) {
  if (v != v) return 0xffffffffu;
  const uint32_t b = __float_as_uint(v + 0.0f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// V: 32 V >= E
template <bool BF16, int V>
__global__ void __launch_bounds__(RT_THREADS) route_kernel(const RtArgs a) {
  __shared__ float4 part[RT_THREADS];                          // [warp][lane]
  __shared__ float logits[RT_TOKENS][32 * V];          // the first block's are used
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t rank = cluster_rank();
  uint32_t nblocks;
  asm volatile("mov.u32 %0, %cluster_nctarank;" : "=r"(nblocks));
  const int t0 = (int)(blockIdx.x / nblocks) * RT_TOKENS;
  pdl_wait();  // launched early: nothing is touched before the kernel before has ended
  cluster_arrive();  // waited for before the first store to another block
  pdl_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.err != nullptr) *a.err = 0;

  const int e_begin = (int)rank * a.per_block, e_end = min(a.E, e_begin + a.per_block);
  bool met = false;
  for (int e0 = e_begin; e0 < e_begin + a.per_block; e0 += 16) {
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const bool hx = t0 + g < a.M, hl = e0 + g < e_end, hh = e0 + g + 8 < e_end;
    const uint8_t* px = a.X + ((int64_t)(t0 + g) * a.D + t * 8) * 2;
    const uint8_t* pl = a.Wr + ((int64_t)(e0 + g) * a.D + t * 8) * 2;
    const uint8_t* ph = pl + (int64_t)a.D * 16;
    const int steps = (a.D + 31) >> 5;
    constexpr int U = 8;  // all the loads of d = 2048 at once: they are all latency
    for (int s0 = warp; s0 < steps; s0 += 8 * U) {
      uint4 x[U], wl[U], wh[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int64_t k = (int64_t)(s0 + 8 * i) * 32;
        const bool in = k + t * 8 < a.D;
        x[i] = wl[i] = wh[i] = make_uint4(0, 0, 0, 0);
        if (in && hx && SWIGLU_CHECK_PTR(a.dbg, px + k * 2, 16, a.err))
          x[i] = ft_load16(px + k * 2);
        if (in && hl && SWIGLU_CHECK_PTR(a.dbg, pl + k * 2, 16, a.err))
          wl[i] = ft_load16(pl + k * 2);
        if (in && hh && SWIGLU_CHECK_PTR(a.dbg, ph + k * 2, 16, a.err))
          wh[i] = ft_load16(ph + k * 2);
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        float p[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        mma_16816<BF16>(p, wl[i].x, wh[i].x, wl[i].y, wh[i].y, x[i].x, x[i].y);
        mma_16816<BF16>(p, wl[i].z, wh[i].z, wl[i].w, wh[i].w, x[i].z, x[i].w);
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[c] += p[c];
      }
    }
    part[threadIdx.x] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    __syncthreads();
    if (!met) cluster_wait();
    met = true;
    if (threadIdx.x < 128) {
      const float* f = reinterpret_cast<const float*>(part) + threadIdx.x;
      float v = f[0];
#pragma unroll
      for (int w = 1; w < 8; ++w) v += f[w * 128];
      const int ln = threadIdx.x >> 2, c = threadIdx.x & 3;
      const int e = e0 + (ln >> 2) + 8 * (c >> 1), m = 2 * (ln & 3) + (c & 1);
      if (e < e_end) cluster_store(cluster_map(smem_u32(&logits[m][e]), 0), v);
    }
    __syncthreads();
  }
  cluster_arrive();
  cluster_wait();
  const int token = t0 + warp;
  if (rank != 0 || token >= a.M) return;

  const float* l = logits[warp];
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * 32 + lane;
    key[i] = e < a.E ? rt_key(l[e]) : 0;
  }
  int mine = 0;  // lane j: the j-th choice
  for (int j = 0; j < a.topk; ++j) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) m = max(m, key[i]);
    m = __reduce_max_sync(0xffffffffu, m);
    uint32_t at = 0xffffffffu;
#pragma unroll
    for (int i = V - 1; i >= 0; --i)
      if (key[i] == m) at = i * 32 + lane;
    at = __reduce_min_sync(0xffffffffu, at);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (at == (uint32_t)(i * 32 + lane)) key[i] = 0;
    if (lane == j) mine = (int)at;
  }
  const float top = l[__shfl_sync(0xffffffffu, mine, 0)];
  const float e_mine = lane < a.topk ? expf(l[mine] - top) : 0.0f;
  float den = e_mine;
  if (!a.norm) {
    den = 0.0f;
    for (int e = lane; e < a.E; e += 32) den += expf(l[e] - top);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) den += __shfl_xor_sync(0xffffffffu, den, d);
  if (lane < a.topk) {
    int* oi = a.idx + (int64_t)token * a.topk + lane;
    float* ow = a.wts + (int64_t)token * a.topk + lane;
    if (SWIGLU_CHECK_PTR(a.dbg, oi, 4, a.err)) *oi = mine;
    if (SWIGLU_CHECK_PTR(a.dbg, ow, 4, a.err)) *ow = a.scale * (e_mine / den);
  }
}

}  // namespace swiglu
