// w4_tensor.cuh -- products of 17 to 64 tokens with 4-bit weights on the
// tcgen05 tensor core (the packed weights and the results of w4_stream.cuh):
//   Y[m, r] = sum_G s[r, G] sum_{k in G} (q[r, k] - z[r, G]) X[m, k].
//
// Beyond 16 tokens the rate of mma.sync (1024 products a cycle and SM,
// measured) and the shared-memory reads of the token rows bound w4_stream.cuh;
// on tcgen05 the products are far from a bound again (tensor pipe 18% busy).
// wt_serves in serving.cu says which of the two takes a product.
//
// Swap-AB: 128 weight rows (8 of the packed 16-row tiles) take the MMA's M
// dimension, the tokens its N dimension (NT = 32, 48 or 64).  Roles of a block:
//   producer  (1 thread) stages of 256 k, two tensor-map boxes each: the 8
//                        tiles' records, and the token rows;
//   unpackers (8 warps)  32 weight rows each, a thread per row: codes -> whole
//                        numbers q - z in 16 bits (exact) -> the A operand, which
//                        the MMA reads from TMEM;
//   MMA       (1 warp)   4 MMAs per 64 k into one of 4 TMEM accumulators, a
//                        new one for each group of k that shares its scales;
//   epilogue  (8 warps)  a thread per weight row and half of the tokens: adds
//                        scale * accumulator to its fp32 sums, group by group,
//                        so no weight is rounded here either.
// The roles meet once per stage and once per pair of accumulators: a barrier
// that is ready still costs a warp some 200 cycles of dependent instructions,
// and with one per 64 or 128 k those bounded the loop (64 tokens, 22016 x 4096:
// 42 us, then 37).  Before that the same product took 58 us with A in shared
// memory (written and read there once more) and an epilogue unrolled over its
// registers (its code, run once and cold, took 10 us to fetch), and 44 without
// the two.  16 unpacking warps (72 registers a thread) take 42 us, 8 took 38.
// With neighbouring lanes on one chunk and mask-and-or in one instruction (a
// third fewer instructions in all to unpack 64 k) it is 35.4.
//
// The stages of the tiles beyond a multiple of the blocks are laid end to end
// and shared evenly by the blocks; the other tiles are whole.  Partial tiles
// meet in the workspace, and the last block of a tile to finish (a counter per
// tile) adds them in block order and writes.  No block waits for another.
//
// Measured (bf16, groups of 128): MLP 4096/11008, 72 MB, 10.7 us at the HBM
// rate, 58 us at 64 tokens (w4_stream.cuh, reading the weights twice, 122), 50 at
// 32 (57); groups of 32: 79 at 64 tokens, where an accumulator per 32 k makes the
// epilogue the bound.  At 64 tokens gate/up takes 38.9 us alone, issue slots 44%
// and the ALU 35% used (over the whole kernel; the unpackers never wait in the
// loop).  Next after that: each tile reads all token rows, 88
// MB through L2, 24 us with the weights at the 5.8 TB/s that reach the SMs; some
// 5 us are start and shared tiles' sums.
#pragma once

#include "fewtok.cuh"

namespace swiglu {

constexpr int WT_THREADS = 576;   // producer, MMA, 8 unpackers, 8 epilogue warps
constexpr int WT_KB = 4;          // 64-k blocks of a stage
constexpr int WT_SETS = 2;        // pairs of TMEM accumulators, columns 0 to 255
constexpr int WT_ABUFS = 2;       // unpacked A operands of a stage, 128 columns each from 256 on
constexpr int WT_OUT = 8 * 2048;  // epilogue warps' [16][32] sums on their way out
constexpr int WT_MAX_STAGES = 4;
constexpr int WT_MAX_SHARED = 512; // counters of a kernel: its shared tiles, fewer than SMs

struct WtArgs {
  int gate_up;       // out = rnd(SiLU(scale g) u), else rnd(scale v)
  int M, K;          // tokens; contraction, a multiple of 8
  int rows;          // rows of out: output features, or hidden units (gate/up)
  int tiles16, tiles;           // 16- and 128-row tiles
  int sk_tiles, sharers, seg_max;  // tiles shared between blocks, by how many, in segments a block
  int pair;          // 64-k blocks of one accumulator (2: groups of 128)
  const uint8_t* W;  // packed
  void* out;         // [M, rows]
  float scale;
  int first;         // first kernel of a call
  int inject;        // test hook: the first stage is never filled
  int stages;
  float* part;       // partial tiles [block][segment][NT][128]
  int* counters;     // [tiles], zero
  uint64_t wait_limit_ns;
  int* err;
#ifdef SWIGLU_DEBUG
  DbgWin dbg;        // out, X, packed weights, workspace
#endif
};

template <int NT, bool G32, bool ZP>
struct WtShape {
  static constexpr int GROUPS = G32 ? 2 : 1;
  static constexpr int RECORD = 512 + GROUPS * (ZP ? 48 : 32);
  static constexpr int PIECE = WT_KB * RECORD;         // one 16-row tile's part of a stage
  static constexpr int X_BYTES = WT_KB * NT * 128;     // first: boxes are 1024-byte aligned
  static constexpr int FILL = X_BYTES + 8 * PIECE;     // bytes that fill a stage
  static constexpr int STAGE = (FILL + 1023) / 1024 * 1024;
  static_assert(WT_SETS * 2 * NT <= 256, "accumulators exceed their columns");
};

// D += A B with A in TMEM: a lane per row, two neighbouring k in a column.
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr)
      : "memory");
}

// A block's segments: its range of the shared tiles' stages, then whole tiles.
struct WtSegs {
  int x, x_end, dp, dp_end, spt, sk_tiles;
  __device__ __forceinline__ bool next(int& tile, int& s0, int& n, bool& whole) {
    if (x < x_end) {
      tile = x / spt;
      s0 = x - tile * spt;
      n = min(spt - s0, x_end - x);
      x += n;
      whole = n == spt;
      return true;
    }
    if (dp < dp_end) {
      tile = sk_tiles + (int)blockIdx.x + dp * (int)gridDim.x;
      s0 = 0;
      n = spt;
      whole = true;
      ++dp;
      return true;
    }
    return false;
  }
};
// The shared tiles' stages lie over the first `sharers` blocks, none of which
// gets nothing (there are at least as many stages).
__device__ __forceinline__ int wt_start(int c, int total, int sharers) {
  return c >= sharers ? total : (int)((int64_t)c * total / sharers);
}
__device__ __forceinline__ int wt_owner(int x, int total, int sharers) {  // the block that holds stage x
  int c = (int)((int64_t)x * sharers / total);
  while (c + 1 < sharers && wt_start(c + 1, total, sharers) <= x) ++c;
  while (c > 0 && wt_start(c, total, sharers) > x) --c;
  return c;
}

template <bool BF16, int NT, bool G32, bool ZP>
__global__ void __launch_bounds__(WT_THREADS, 1)
    w4_tensor_kernel(const __grid_constant__ CUtensorMap tmW,
                     const __grid_constant__ CUtensorMap tmX, const WtArgs a) {
  using S = WtShape<NT, G32, ZP>;
  using P = Ft16<BF16>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ uint64_t bars[2 * WT_MAX_STAGES + 2 * WT_ABUFS + 2 * WT_SETS + 1];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word, last_word;
  uint8_t* const smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem), bar0 = smem_u32(bars);
  auto full_bar = [&](int i) { return bar0 + 8u * i; };
  auto empty_bar = [&](int i) { return bar0 + 8u * (WT_MAX_STAGES + i); };
  auto aready_bar = [&](int i) { return bar0 + 8u * (2 * WT_MAX_STAGES + i); };
  auto afree_bar = [&](int i) { return bar0 + 8u * (2 * WT_MAX_STAGES + WT_ABUFS + i); };
  auto accf_bar = [&](int i) { return bar0 + 8u * (2 * WT_MAX_STAGES + 2 * WT_ABUFS + i); };
  auto acce_bar = [&](int i) { return bar0 + 8u * (2 * WT_MAX_STAGES + 2 * WT_ABUFS + WT_SETS + i); };
  const uint32_t drain_bar = bar0 + 8u * (2 * WT_MAX_STAGES + 2 * WT_ABUFS + 2 * WT_SETS);
  volatile int* const abort_flag = &abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (a.first) {
    pdl_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;
  }
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(full_bar(i), 1);
      mbar_init(empty_bar(i), 9);  // 8 unpackers, the MMAs that read the token rows
    }
    for (int i = 0; i < WT_ABUFS; ++i) {
      mbar_init(aready_bar(i), 8);
      mbar_init(afree_bar(i), 1);
    }
    for (int i = 0; i < WT_SETS; ++i) {
      mbar_init(accf_bar(i), 1);
      mbar_init(acce_bar(i), 256);
    }
    mbar_init(drain_bar, 1);
    abort_word = last_word = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  const int nk = (a.K + 63) >> 6, spt = (nk + WT_KB - 1) / WT_KB;  // 64-k blocks, stages of a tile
  const int total = a.sk_tiles * spt;
  auto segs = [&]() {
    return WtSegs{wt_start(blockIdx.x, total, a.sharers),
                  wt_start(blockIdx.x + 1, total, a.sharers), 0,
                  (a.tiles - a.sk_tiles) / (int)gridDim.x, spt, a.sk_tiles};
  };
  auto wait = [&](uint32_t bar, uint32_t parity) {
    return mbar_wait_bounded(bar, parity, a.wait_limit_ns, abort_flag, a.err);
  };
  const uint32_t ring = sbase + WT_OUT;

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      // boxes past the end of the contraction or of the tiles fill with zeros
      auto load_w = [&](int slot, int tile, int st) {
        mbar_arrive_expect_tx(full_bar(slot), S::FILL);
        tma_load_3d(ring + slot * S::STAGE + S::X_BYTES, &tmW, full_bar(slot), 0, st * WT_KB, tile * 8);
      };
      auto load_x = [&](int slot, int st) {
        const uint32_t dst = ring + slot * S::STAGE;
        if (a.K % 64 == 0) {  // [K / 64][M][64]: one box
          tma_load_3d(dst, &tmX, full_bar(slot), 0, 0, st * WT_KB);
        } else {
          for (int q = 0; q < WT_KB; ++q)
            tma_load_3d(dst + q * NT * 128, &tmX, full_bar(slot), (st * WT_KB + q) * 64, 0, 0);
        }
      };
      // the weights of the first stages, then (the kernel before this one
      // writes them) the token rows
      int pre = 0;
      WtSegs it = segs();
      int tile, s0, n;
      bool whole;
      if (!a.first) {
        while (pre < a.stages && it.next(tile, s0, n, whole))
          for (int i = 0; i < n && pre < a.stages; ++i, ++pre)
            if (!(a.inject && pre == 0)) load_w(pre, tile, s0 + i);
        pdl_wait();
      }
      int slot = 0, done = 0;
      uint32_t phase = 0, issued = 0, parity = 0;
      bool ok = true;
      it = segs();
      while (ok && it.next(tile, s0, n, whole))
        for (int i = 0; i < n; ++i, ++done) {
          const bool skip = a.inject && done == 0;
          if (done >= pre) {
            if (!(ok = wait(empty_bar(slot), phase ^ 1u))) break;
            if (!skip) load_w(slot, tile, s0 + i);
          }
          if (!skip) {
            load_x(slot, s0 + i);
            issued |= 1u << slot;
            parity = (parity & ~(1u << slot)) | (phase << slot);
          }
          if (++slot == a.stages) {
            slot = 0;
            phase ^= 1u;
          }
        }
      if (!ok)  // no copy may land after the block has gone
        for (int i = 0; i < a.stages; ++i)
          if (issued & (1u << i))
            mbar_wait_bounded(full_bar(i), (parity >> i) & 1u, a.wait_limit_ns, nullptr, a.err);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA
    // All lanes keep the loop's state, so that descriptors stay in uniform
    // registers, and an elected one issues.
    constexpr uint32_t idesc = make_idesc_f16(BF16, false, false, 128, NT);
    const uint64_t desc0 = make_sw128_desc(0, 16, 1024);  // descriptors differ in their address alone
    const uint32_t d0 = __shfl_sync(0xffffffffu, tmem, 0);
    const bool leader = elect_one();
    int slot = 0, ab = 0, set = 0;
    uint32_t phase = 0, aphase = 0, setphase = 0;
    auto all_wait = [&](uint32_t bar, uint32_t parity) {
      return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
    };
    bool ok = true;
    WtSegs it = segs();
    int tile, s0, n;
    bool whole;
    while (ok && it.next(tile, s0, n, whole))
      for (int i = 0; ok && i < n; ++i) {
        const int nb = min(WT_KB, nk - (s0 + i) * WT_KB);
        if (!(ok = all_wait(full_bar(slot), phase) && all_wait(aready_bar(ab), aphase))) break;
        const uint64_t dx = desc0 + ((ring + slot * S::STAGE) >> 4);
        const uint32_t ta = d0 + 256 + ab * 128;
        // a pair of accumulators: 64 k (groups of 32), 128 k or 256 k
        const int per = G32 ? 1 : 2 * a.pair;
#pragma unroll 1
        for (int q = 0; q < nb; q += per) {
          if (!(ok = all_wait(acce_bar(set), setphase ^ 1u))) break;
          tc_fence_after();
          if (leader) {
            const uint32_t d = d0 + set * 2 * NT;
            if (G32) {
              const uint32_t tp = ta + q * 32;
              const uint64_t dp = dx + q * (NT * 8);
              umma_f16_ts(d, tp, dp, idesc, 0u);
              umma_f16_ts(d, tp + 8, dp + 2, idesc, 1u);
              umma_f16_ts(d + NT, tp + 16, dp + 4, idesc, 0u);
              umma_f16_ts(d + NT, tp + 24, dp + 6, idesc, 1u);
            } else {
              const int last = min(per, nb - q);
#pragma unroll 1
              for (int p = 0; p < last; ++p) {
                const uint32_t tp = ta + (q + p) * 32;
                const uint64_t dp = dx + (q + p) * (NT * 8);
                const uint32_t dd = d + (p >= a.pair ? NT : 0);
                umma_f16_ts(dd, tp, dp, idesc, p == 0 || p == a.pair ? 0u : 1u);
                umma_f16_ts(dd, tp + 8, dp + 2, idesc, 1u);
                umma_f16_ts(dd, tp + 16, dp + 4, idesc, 1u);
                umma_f16_ts(dd, tp + 24, dp + 6, idesc, 1u);
              }
            }
            umma_commit(accf_bar(set));
            if (q + per >= nb) {
              umma_commit(afree_bar(ab));
              umma_commit(empty_bar(slot));
            }
          }
          __syncwarp();
          if (++set == WT_SETS) {
            set = 0;
            setphase ^= 1u;
          }
        }
        if (++ab == WT_ABUFS) {
          ab = 0;
          aphase ^= 1u;
        }
        if (++slot == a.stages) {
          slot = 0;
          phase ^= 1u;
        }
      }
    if (leader) {
      umma_commit(drain_bar);
      mbar_wait_bounded(drain_bar, 0, a.wait_limit_ns, nullptr, a.err);
    }
    __syncwarp();
  } else if (warp < 10) {
    // ---------------------------------------------------------------- unpackers
    // a warp reaches the TMEM lanes of its quarter: rows 32 (warp % 4).. of
    // the tile, and takes the even or the odd 64-k blocks
    const int p = (warp - 2) >> 2, t16 = (warp & 3) * 2 + (lane >> 4), g = (lane >> 1) & 7, hi = lane & 1;
    const uint32_t ta = tmem + ((uint32_t)(warp & 3) << 21) + 256;
    // TMEM lane 2 g + hi of a 16-row tile holds row g + 8 hi: neighbouring lanes
    // read the same 16 bytes, at (4 g + t) 16 of a record, and 8 lanes meet a
    // bank twice.
    int slot = 0, ab = 0;
    uint32_t phase = 0, aphase = 0;
    bool ok = true;
    WtSegs it = segs();
    int tile, s0, n;
    bool whole;
    while (ok && it.next(tile, s0, n, whole))
      for (int i = 0; ok && i < n; ++i) {
        const int nb = min(WT_KB, nk - (s0 + i) * WT_KB);
        ok = __all_sync(0xffffffffu, wait(full_bar(slot), phase));
        if (!ok) break;
        const uint32_t rec0 = ring + slot * S::STAGE + S::X_BYTES + t16 * S::PIECE;
#pragma unroll 1
        for (int q = p; q < nb; q += 2) {
          const uint32_t rec = rec0 + q * S::RECORD;
          uint32_t v[2][4], z[2] = {8u, 8u};
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const uint4 x = lds128(rec + g * 64 + t * 16);
            v[0][t] = hi ? x.y : x.x;
            v[1][t] = hi ? x.w : x.z;
          }
          if (ZP) {
            z[0] = lds8(rec + 512 + S::GROUPS * 32 + g * 2 + hi);
            z[1] = G32 ? lds8(rec + 512 + S::GROUPS * 32 + 16 + g * 2 + hi) : z[0];
          }
          uint32_t out[32];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const uint32_t m = P::MAGIC | (z[h] * 0x10001u);
              auto number = [&](uint32_t x) {
                return ft_sub2<BF16>(and_or<0x000f000fu>(x, P::MAGIC), m);
              };
              uint32_t* o = out + h * 16 + t * 4;
              o[0] = number(v[h][t]);
              o[1] = number(v[h][t] >> 8);
              o[2] = number(v[h][t] >> 4);
              o[3] = number(v[h][t] >> 12);
            }
          if (q < 2) {
            ok = __all_sync(0xffffffffu, wait(afree_bar(ab), aphase ^ 1u));
            if (!ok) break;
            tc_fence_after();
          }
          tmem_st_32x32b_x32(ta + ab * 128 + q * 32, out);
        }
        if (ok && p >= nb) ok = __all_sync(0xffffffffu, wait(afree_bar(ab), aphase ^ 1u));
        if (!ok) break;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(aready_bar(ab));
          mbar_arrive(empty_bar(slot));
        }
        if (++ab == WT_ABUFS) {
          ab = 0;
          aphase ^= 1u;
        }
        if (++slot == a.stages) {
          slot = 0;
          phase ^= 1u;
        }
      }
  } else {
    // ---------------------------------------------------------------- epilogue
    constexpr int NC = NT / 2;  // tokens of a warp
    const int e = (warp & 3) * 32 + lane;  // TMEM lane, weight row of the tile
    const int col0 = warp < 14 ? 0 : NC;
    const uint32_t tacc = tmem + ((uint32_t)(e & 96) << 16) + col0;
    const uint32_t stage = sbase + (warp - 10) * 2048;
    const int slot16 = e & 15;  // this row's place among 16 scales
    const int row32 = (lane & 16) + (lane & 1) * 8 + ((lane >> 1) & 7);  // its place among 32 rows
    int set = 0, seg = 0;
    uint32_t setphase = 0;
    bool live = true;  // false after a wait ran out: go through the motions, add nothing
    uint16_t* const out = static_cast<uint16_t*>(a.out);
    WtSegs it = segs();
    int tile, s0, n;
    bool whole;
    for (; it.next(tile, s0, n, whole); ++seg) {
      const int kb0 = s0 * WT_KB, kb1 = min(nk, (s0 + n) * WT_KB);
      const int t16 = tile * 8 + (e >> 4);
      // the scales of this row's groups, one per accumulator of the segment
      const uint8_t* scales = a.W + ((int64_t)min(t16, a.tiles16 - 1) * nk + kb0) * S::RECORD + 512 +
                              slot16 * 2;
      const int step = a.pair * S::RECORD, most = (kb1 - kb0) * S::RECORD;
      auto scale_at = [&](int u) -> uint32_t {
        const int o = G32 ? (u >> 1) * S::RECORD + (u & 1) * 32 : u * step;
        return o < most && SWIGLU_CHECK_PTR(a.dbg, scales + o, 2, a.err)
                   ? *reinterpret_cast<const uint16_t*>(scales + o)
                   : 0u;
      };
      const int units = G32 ? 2 * (kb1 - kb0) : (kb1 - kb0 + a.pair - 1) / a.pair;
      float sum[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) sum[c] = 0.0f;
      uint32_t sc[4];  // four accumulators ahead: they come from L2
#pragma unroll
      for (int q = 0; q < 4; ++q) sc[q] = scale_at(q);
      for (int u0 = 0; u0 < units; u0 += 4) {
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
          if (u0 + q >= units) break;
          if (live) live = __all_sync(0xffffffffu, wait(accf_bar(set), setphase));
          if (live) tc_fence_after();
#pragma unroll
          for (int p = q; p < q + 2; ++p) {
            const float s = P::lo(sc[p]);
            sc[p] = scale_at(u0 + p + 4);
            if (live && u0 + p < units) {
              uint32_t r[NC / 8][8];
#pragma unroll
              for (int c = 0; c < NC / 8; ++c)
                tmem_ld_32x32b_x8(tacc + (set * 2 + (p & 1)) * NT + c * 8, r[c]);
              tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < NC; ++c) sum[c] = fmaf(s, __uint_as_float(r[c / 8][c % 8]), sum[c]);
            }
          }
          if (live) {
            tc_fence_before();
            mbar_arrive(acce_bar(set));
          }
          if (++set == WT_SETS) {
            set = 0;
            setphase ^= 1u;
          }
        }
      }
      // Writes a finished tile's rows, through shared memory so that the code
      // is a short loop: unrolled over the registers it ran once and cold, and
      // its fetches took 10 us.  Gate/up: a unit's up row is 8 rows on.
      auto finish = [&]() {
        const int u = lane & 15, row0 = lane >> 4;
#pragma unroll
        for (int c0 = 0; c0 < NC; c0 += 16) {
#pragma unroll
          for (int c = c0; c < c0 + 16 && c < NC; ++c) sts32(stage + ((c - c0) * 32 + row32) * 4, sum[c]);
          __syncwarp();
          const int n = min(min(16, NC - c0), a.M - col0 - c0);
          if (a.gate_up) {  // 16 units of two tokens
            const int r = (t16 & ~1) * 8 + u, at = (u >> 3) * 16 + (u & 7);
#pragma unroll 1
            for (int c = row0; c < n; c += 2) {
              const float gate = a.scale * lds32f(stage + (c * 32 + at) * 4);
              const float v = ft_silu(gate) * lds32f(stage + (c * 32 + at + 8) * 4);
              uint16_t* o = out + (int64_t)(col0 + c0 + c) * a.rows + r;
              if (r < a.rows && SWIGLU_CHECK_PTR(a.dbg, o, 2, a.err)) *o = P::rnd(v);
            }
          } else {
            const int r = tile * 128 + e;
#pragma unroll 1
            for (int c = 0; c < n; ++c) {
              uint16_t* o = out + (int64_t)(col0 + c0 + c) * a.rows + r;
              if (r < a.rows && SWIGLU_CHECK_PTR(a.dbg, o, 2, a.err))
                *o = P::rnd(a.scale * lds32f(stage + (c * 32 + lane) * 4));
            }
          }
          __syncwarp();
        }
      };
      if (whole) {
        finish();
        continue;
      }
      float* mine = a.part + ((int64_t)blockIdx.x * a.seg_max + seg) * NT * 128 + col0 * 128 + e;
      if (SWIGLU_CHECK(seg < a.seg_max, a.err) && SWIGLU_CHECK_PTR(a.dbg, mine, 4, a.err)) {
#pragma unroll
        for (int c = 0; c < NC; ++c) mine[c * 128] = sum[c];
      }
      const int c_first = wt_owner(tile * spt, total, a.sharers);
      const int c_last = wt_owner((tile + 1) * spt - 1, total, a.sharers);
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (warp == 10 && lane == 0) {
        __threadfence();  // the 256 threads' stores before the count
        last_word = live && !*abort_flag && SWIGLU_CHECK(tile < WT_MAX_SHARED, a.err) &&
                    atomicAdd(a.counters + tile, 1) == c_last - c_first;
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      const bool last = *const_cast<volatile int*>(&last_word) != 0;
      asm volatile("bar.sync 1, 256;" ::: "memory");  // read before it is written again
      if (last) {
        __threadfence();
#pragma unroll
        for (int c = 0; c < NC; ++c) sum[c] = 0.0f;
        for (int b = c_first; b <= c_last; ++b) {  // in block order
          const int j = tile - wt_start(b, total, a.sharers) / spt;
          const float* p = a.part + ((int64_t)b * a.seg_max + j) * NT * 128 + col0 * 128 + e;
          if (!SWIGLU_CHECK(j >= 0 && j < a.seg_max, a.err)) continue;
#pragma unroll
          for (int c = 0; c < NC; ++c) sum[c] += __ldcg(p + c * 128);
        }
        finish();
        if (warp == 10 && lane == 0) a.counters[tile] = 0;  // for the next call
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace swiglu
