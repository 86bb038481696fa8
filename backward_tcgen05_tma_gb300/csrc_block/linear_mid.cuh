// linear_mid.cuh -- linear layers of some tens to some hundreds of tokens:
//
//   Z = X W^T + b,  Y = act(Z) + R
//
// The weights' bytes are the bound, so every SM has to stream an equal share of
// them from the first moment, and nothing may follow the last byte but a short
// epilogue.  Tiles are small (MT tokens x BN weight rows, one a block, two blocks
// an SM, so one block's start and epilogue lie under the other's stream), and where
// they are too few for the SMs a cluster's blocks take a tile together, each a part
// of the contraction; their sums meet in the blocks' shared memory, in the
// parts' order, each block finishing its share of the tile's columns.  No partial
// sum goes through memory.
//
// The tokens take the MMA's M = 128.  Where the box of tokens is smaller (MT = 64, or
// fewer tokens), the MMA reads on past it into whatever the ring holds: those rows of
// the accumulator are no token's and are never read.
//
// Measured, back to back, weights from HBM: 11008 x 4096 64 tokens 20 us, 128 tokens 22,
// 512 tokens 38 (the forms before: 34, 35, 48); 4096 x 11008 64 tokens 19.6 (34); 1024 x
// 2816 128 tokens 7.9 (24); 2816 x 1024 64 tokens 6.4 (8.0).  About 5 us of each are the
// start, the first bytes' way and the end.  One block takes 0.28 us a step of 64 k, of
// whatever depth its ring is and whether one or two warps send its loads, so two a
// SM are better than one with twice the ring unless the tiles are large.
#pragma once

#include "linear_epi.cuh"

namespace swiglu {

constexpr int LM_THREADS = 192;  // producer warp, MMA warp, 4 epilogue warps

// Shared memory: the ring of `stages` times MT token rows and bn weight rows of 128
// bytes, with a tail that the last stage's MMA may read (128 rows), then barriers.
constexpr int LM_MAX_STAGES = 16;
constexpr int LM_BARS = (2 * LM_MAX_STAGES + 2) * 8 + 16;
__host__ __device__ constexpr int lm_ring(int mt, int bn, int stages) {
  return stages * (mt + bn) * 128 + (mt + bn < 128 ? (128 - mt - bn) * 128 : 0);
}

struct LmArgs {
  int M, N;
  int kb;       // blocks of 64 of the contraction
  int m_tiles;
  int split;    // blocks of a cluster
  int bn;       // weight rows of a tile, a multiple of 16 up to 256
  int stages;
  int ring;     // bytes
  int x_rows;   // token rows of a box
  const uint8_t* bias;
  const uint8_t* res;
  uint8_t* z;
  uint8_t* y;
  int act;
  int inject;
  uint64_t wait_limit_ns;
  int* err;
#ifdef SWIGLU_DEBUG
  DbgWin dbg;
#endif
};

// What W columns of token m from column nc need beside their sums, asked for ahead.
template <int W>
struct LmSide {
  uint4 b[W / 8], r[W / 8];
  __device__ __forceinline__ void load(const LmArgs& a, bool on, int m, int nc) {
    const int64_t at = ((int64_t)m * a.N + nc) * 2;
#pragma unroll
    for (int h = 0; h < W / 8; ++h) {
      const bool in = on && nc + h * 8 < a.N;
      const uint8_t *pb = a.bias + (int64_t)nc * 2 + h * 16, *pr = a.res + at + h * 16;
      b[h] = in && a.bias != nullptr && SWIGLU_CHECK_PTR(a.dbg, pb, 16, a.err) ? *reinterpret_cast<const uint4*>(pb)
                                                                              : make_uint4(0u, 0u, 0u, 0u);
      r[h] = in && a.res != nullptr && SWIGLU_CHECK_PTR(a.dbg, pr, 16, a.err) ? *reinterpret_cast<const uint4*>(pr)
                                                                             : make_uint4(0u, 0u, 0u, 0u);
    }
  }
};

template <bool BF16, int W>
__device__ __forceinline__ void lm_finish(const LmArgs& a, int m, int nc, float (&v)[W], const LmSide<W>& side) {
  using P = Pack<BF16>;
  const int64_t at = ((int64_t)m * a.N + nc) * 2;
  auto put = [&](uint8_t* p) {
#pragma unroll
    for (int h = 0; h < W / 8; ++h) {
      if (nc + h * 8 < a.N && SWIGLU_CHECK_PTR(a.dbg, p + h * 16, 16, a.err))
        *reinterpret_cast<uint4*>(p + h * 16) =
            make_uint4(P::two(v[h * 8], v[h * 8 + 1]), P::two(v[h * 8 + 2], v[h * 8 + 3]),
                       P::two(v[h * 8 + 4], v[h * 8 + 5]), P::two(v[h * 8 + 6], v[h * 8 + 7]));
    }
  };
#pragma unroll
  for (int i = 0; i < W / 2; ++i) {
    const float2 q = P::unpack((&side.b[i >> 2].x)[i & 3]);
    v[2 * i] += q.x;
    v[2 * i + 1] += q.y;
  }
  if (a.z != nullptr) put(a.z + at);
  act_switch(a.act, [&](auto t) {
#pragma unroll
    for (int i = 0; i < W; i += 2) act_value2<decltype(t)::value>(v[i], v[i + 1]);
  });
  if (a.res != nullptr) {
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
      const float2 q = P::unpack((&side.r[i >> 2].x)[i & 3]);
      v[2 * i] += q.x;
      v[2 * i + 1] += q.y;
    }
  }
  put(a.y + at);
}

template <bool BF16, int MT>
__global__ void __launch_bounds__(LM_THREADS, 2)
    linear_mid_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                      const LmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem), bar0 = sbase + a.ring;
  auto full = [&](int i) { return bar0 + 8u * i; };
  auto empty = [&](int i) { return bar0 + 8u * (LM_MAX_STAGES + i); };
  const uint32_t acc_bar = bar0 + 8u * (2 * LM_MAX_STAGES), drained = acc_bar + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + a.ring + LM_BARS - 16);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + a.ring + LM_BARS - 12);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, bn = a.bn;
  const uint32_t stage_bytes = (uint32_t)(MT + bn) * 128u;
  uint32_t columns = 32;  // of TMEM, a power of two
  while ((int)columns < bn) columns *= 2;

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tmX);
      tma_prefetch_desc(&tmW);
      *abort_flag = 0;
    }
    for (int i = lane; i < 2 * LM_MAX_STAGES + 2; i += 32) mbar_init(bar0 + 8u * i, 1);
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();  // launched early: nothing is touched before the kernel before has ended
  // TMEM is asked for only now: that kernel, beside this one on the SM, may not have
  // asked for its own yet, and would wait for a block that waits for it.  The next
  // kernel is let in behind it for the same reason.
  uint32_t tmem = 0;
  if (warp != 0) {
    if (warp == 1) {
      tmem_alloc(smem_u32(tmem_slot), columns);
      tmem_relinquish();
    }
    tc_fence_before();
    asm volatile("bar.sync 1, 160;" ::: "memory");
    tc_fence_after();
    tmem = *tmem_slot;
    pdl_launch_dependents();
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;

  const int rank = a.split > 1 ? (int)cluster_ctarank() : 0, tile = (int)blockIdx.x / a.split;
  const int m0 = tile % a.m_tiles * MT, n0 = tile / a.m_tiles * bn;
  const int kb0 = a.kb * rank / a.split, nkb = a.kb * (rank + 1) / a.split - kb0;
  const int row = (threadIdx.x & 96) + lane;  // of the accumulator
  const bool mine = warp >= 2 && row < MT && m0 + (row & ~31) < a.M;  // a warp of tokens
  // a cluster's blocks: the columns that a thread finishes, 8 or 16 of each chunk
  constexpr int W = MT == 64 ? 8 : 16;
  const int frow = MT == 64 ? (row & 63) : row, fcol = MT == 64 ? (row >> 6) * 8 : 0;
  const bool alone = a.split == 1, live = warp >= 2 && m0 + (alone ? row : frow) < a.M && (!alone || row < MT);
  LmSide<16> side;
  LmSide<W> part;
  int ok = 1;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0, i = 0;
      uint32_t phase = 0;
      const uint32_t bytes = (uint32_t)(a.x_rows + bn) * 128u;
      for (; i < nkb; ++i) {
        if (!mbar_wait_bounded(empty(stage), phase ^ 1u, a.wait_limit_ns, abort_flag, a.err)) break;
        const uint32_t s = sbase + stage * stage_bytes;
        if (a.inject && blockIdx.x == 0) break;  // test hook
        mbar_arrive_expect_tx(full(stage), bytes);
        tma_load_2d(s + MT * 128, &tmW, full(stage), (kb0 + i) * TC_BK, n0);
        tma_load_2d(s, &tmX, full(stage), (kb0 + i) * TC_BK, m0);
        if (++stage == a.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      // what was sent for lands before the block ends, whether the MMA warp gave up or not
      for (int q = max(0, i - a.stages); q < i; ++q)
        mbar_wait_bounded(full(q % a.stages), (uint32_t)(q / a.stages) & 1u, a.wait_limit_ns, nullptr, a.err);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = make_idesc_f16(BF16, false, false, 128, bn);
      int stage = 0;
      uint32_t phase = 0;
      for (int i = 0; i < nkb && ok; ++i) {
        ok = mbar_wait_bounded(full(stage), phase, a.wait_limit_ns, abort_flag, a.err);
        if (!ok) break;
        tc_fence_after();
        const uint32_t s = sbase + stage * stage_bytes;
#pragma unroll
        for (int kk = 0; kk < TC_BK / TC_UMMA_K; ++kk)
          umma_f16_ss(tmem, make_sw128_desc(s + kk * 32, 16, 1024), make_sw128_desc(s + MT * 128 + kk * 32, 16, 1024),
                      idesc, (i | kk) != 0 ? 1u : 0u);
        umma_commit(empty(stage));
        if (++stage == a.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (ok) umma_commit(acc_bar);
      umma_commit(drained);
      mbar_wait_bounded(drained, 0, a.wait_limit_ns, nullptr, a.err);
    }
  } else {
    if (alone)
      side.load(a, live, m0 + row, n0);
    else
      part.load(a, live && rank * 16 + fcol < bn, m0 + frow, n0 + rank * 16 + fcol);
    if (lane == 0) ok = mbar_wait_bounded(acc_bar, 0, a.wait_limit_ns, abort_flag, a.err);
    ok = __shfl_sync(0xffffffffu, ok, 0);
    tc_fence_after();
  }
  const uint32_t tacc = tmem + ((uint32_t)(row & 96) << 16);
  if (alone) {
    if (mine && ok) {
#pragma unroll 1
      for (int c = 0; c < bn; c += 16) {
        if (n0 + c >= a.N) break;
        uint32_t r[16];
        tmem_ld_32x32b_x16(tacc + c, r);
        const LmSide<16> now = side;
        side.load(a, live && c + 16 < bn, m0 + row, n0 + c + 16);
        tmem_ld_wait();
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
        if (live) lm_finish<BF16, 16>(a, m0 + row, n0 + c, v, now);
      }
    }
  } else {
    // Chunk q of 16 columns is block q % split's; its part from block p is at
    // [p][q / split][column / 4][row][4] of that block's ring, which nothing uses any
    // more once every block's accumulator is complete.
    const int each = (bn / 16 + a.split - 1) / a.split;
    __syncwarp();
    cluster_sync();
    if (mine) {
#pragma unroll 1
      for (int c = 0; c < bn; c += 16) {
        uint32_t r[16];
        tmem_ld_32x32b_x16(tacc + c, r);
        tmem_ld_wait();
        const int q = c / 16, slot = q / a.split;
        const uint32_t to = mapa_shared(sbase + (uint32_t)(rank * each + slot) * 8192u + row * 16u, q - slot * a.split);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + i * 2048u), "r"(r[4 * i]),
                       "r"(r[4 * i + 1]), "r"(r[4 * i + 2]), "r"(r[4 * i + 3])
                       : "memory");
      }
    }
    cluster_sync();
    if (live && ok) {
#pragma unroll 1
      for (int slot = 0; slot < each; ++slot) {
        const int c = (slot * a.split + rank) * 16 + fcol, next = c + a.split * 16;
        if (c >= bn || n0 + c >= a.N) break;
        const LmSide<W> now = part;
        part.load(a, next < bn && slot + 1 < each, m0 + frow, n0 + next);
        float v[W];
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = 0.0f;
        for (int p = 0; p < a.split; ++p) {
#pragma unroll
          for (int q = 0; q < W / 4; ++q) {
            const float4 f =
                *reinterpret_cast<const float4*>(smem + (p * each + slot) * 8192 + (fcol / 4 + q) * 2048 + frow * 16);
            v[4 * q] += f.x;
            v[4 * q + 1] += f.y;
            v[4 * q + 2] += f.z;
            v[4 * q + 3] += f.w;
          }
        }
        lm_finish<BF16, W>(a, m0 + frow, n0 + c, v, now);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, columns);
  }
}

}  // namespace swiglu
