// w4_stream.cuh -- products of a few tokens (1..32) with 4-bit weights:
//   Y[m, r] = sum_k X[m, k] W[r, k],   W[r, k] = s[r, k/G] (q[r, k] - z[r, k/G])
// and the SwiGLU of such products (gate/up).
//
// What bounds it: half a byte per weight, so at the HBM rate an SM meets 46
// weights per cycle, and unpacking them takes most of its issue slots.  The
// design spends as few instructions per weight as it can:
//   * Each pair of codes becomes a pair of 16-bit whole numbers q - z in two
//     instructions (W4Off in fewtok.cuh): OR-ed into a mantissa, and the
//     constant taken off; in fp16 one shift serves two nibbles.  The tensor core
//     then adds up terms of the formula itself, so a sum is as good as a plain
//     fp32 one whatever the elements.  (Leaving 128 + q or 1024 + q in the
//     products and taking the rest off each sum, from sums of the token's
//     elements, was slower, 34 us at 16 tokens, and put fp16 outputs 3% off, bf16
//     ones 0.5%, where elements of 30000 met weights of 0.)
//   * A warp's weights are runs of unit records (codes, then scales, then zero
//     points) that bulk copies bring into a ring of its own, 8 records a copy.
// Each group's sum is scaled in fp32; no weight is rounded.
//
// Work: a block takes a contiguous run of tiles of 16 RT weight rows (gate/up:
// each 16 are 8 rows of Wg and the 8 rows of Wu of the same hidden units), cuts
// each into chunks of units, lays the chunks end to end and gives each of its
// warps an equal share.  A share that ends inside a tile leaves a partial
// tile in shared memory; at the end of the run the block adds each tile's
// partials in order, applies the epilogue and writes, so results are
// deterministic.  Where the tokens' rows do not fit a block's shared memory the
// contraction is split over a cluster of 2, 4 or 8 blocks: each holds its part
// of the rows and works on all the cluster's tiles, and at the end of a run the
// blocks add up each other's sums through distributed shared memory, in rank
// order.  (What still does not fit is taken in phases.)  From 9 tokens on a
// tile has 32 rows (RT = 2): shared memory, which delivers 128 bytes a cycle,
// would otherwise give most of them to the token rows.
//
// Measured (bf16, groups of 128, MLP 4096/11008, 70 MB, 10.3 us at the HBM rate):
// 23.7 to 24.5 us at 1 to 8 tokens (2.9 TB/s), 31.3 at 16 (46 at 17, 57 at 32,
// where w4_tensor.cuh takes over); one token times 11008 x 4096 8.6 us, times
// 2816 x 1024 3.8 us back to back.  At one token gate/up takes 18.6 us alone:
// issue slots 42% used, DRAM 33%; some 6 us of each kernel are its start (tensor
// cores idle until the token rows and the first records are in) and its end
// (partials meet, 16-bit stores).  Before the present layout (codes apart from
// scales, one code form, sums on the scalar cores) the same MLP took 47 us; before
// clusters split the contraction 44 us at 16 tokens.
#pragma once

#include "fewtok.cuh"

namespace swiglu {

constexpr int WS_MAX_STAGES = 8;

struct WsArgs {
  int gate_up;       // out = rnd(SiLU(scale g) u), else rnd(scale v)
  int M, K;          // tokens; contraction, a multiple of 8
  int rows;          // rows of out: output features, or hidden units (gate/up)
  int tiles16;       // 16-row tiles
  int split;         // blocks of a cluster, which share the contraction
  int tile_quot, tile_rem;  // tiles of 16 RT rows: quot a cluster, one more in the first rem
  const uint8_t* W;  // packed
  const void* X;     // [M, K]
  void* out;         // [M, rows]
  float scale;
  int first;         // first kernel of a call: waits for the work before it at once, and
                     //   block 0 clears the error word; else the weights are read before
                     //   the kernel before it, which writes X, is waited for
  int inject;        // test hook: no warp's first stage is ever filled
  // plan: k-units of a phase, tiles of a run, ring stages, shared-memory offsets
  int phase_units, run, stages;
  int phased;        // the contraction (or a block's part of it) takes several phases
  int part_off, tile_off, ring_off;
  uint64_t wait_limit_ns;
  int* err;
#ifdef SWIGLU_DEBUG
  DbgWin dbg;        // out, X, packed weights, workspace
#endif
};

template <int RT, int NT, bool G32, bool ZP>
struct WsShape {
  // more columns need more registers a warp (and give it more to do at once)
  static constexpr int WARPS = NT == 1 ? 12 : 8;
  static constexpr int TOKENS = 8 * NT;
  static constexpr int UNITS = 8 / RT;                             // units of a chunk
  static constexpr int GROUPS = G32 ? 2 : 1;                       // scales of a unit and row
  static constexpr int RECORD = 512 + GROUPS * (ZP ? 48 : 32);     // bytes of a unit
  static constexpr int PIECE = UNITS * RECORD;                     // one 16-row tile's chunk
  static constexpr int STAGE = RT * PIECE;
  static constexpr int PART = RT * NT * 512;                       // a partial tile
  static constexpr int RUN = NT == 1 ? 24 : NT == 2 ? 12 : 10;     // tiles of a run, at most
  static __host__ __device__ constexpr int xrow(int units) { return units * 128 + 64; }
};

// Shared-memory loads at a compile-time distance from a lane's base address.
template <int OFF>
__device__ __forceinline__ uint4 lds128_at(uint32_t base) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4+%5];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(base), "n"(OFF));
  return v;
}
template <int OFF>
__device__ __forceinline__ uint32_t lds32_at(uint32_t base) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1+%2];" : "=r"(v) : "r"(base), "n"(OFF));
  return v;
}
template <int OFF>
__device__ __forceinline__ uint32_t lds16_at(uint32_t base) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1+%2];" : "=h"(v) : "r"(base), "n"(OFF));
  return v;
}
template <int N>
struct WsInt {
  static constexpr int value = N;
};

template <bool BF16>
__device__ __forceinline__ float4 mma_ws(float4 c, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  float4 d;
  if (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d.x), "=f"(d.y), "=f"(d.z), "=f"(d.w)
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c.x), "f"(c.y), "f"(c.z),
          "f"(c.w));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d.x), "=f"(d.y), "=f"(d.z), "=f"(d.w)
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c.x), "f"(c.y), "f"(c.z),
          "f"(c.w));
  return d;
}

// One warp's place in the block's work: run of tiles, phase of the
// contraction, and the chunks [v, v_end) of the run and phase laid end to end;
// chunk v is chunk c of the run's tile j.
struct WsWalk {
  int run, phase, v, v_end, j, c;
};

template <bool BF16, int RT, int NT, bool G32, bool ZP>
__global__ void __launch_bounds__(WsShape<RT, NT, G32, ZP>::WARPS * 32, 1)
    w4_stream_kernel(const WsArgs a) {
  using S = WsShape<RT, NT, G32, ZP>;
  using P = Ft16<BF16>;
  constexpr int WS_WARPS = S::WARPS;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[WS_WARPS * WS_MAX_STAGES + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = smem_u32(bars) + warp * WS_MAX_STAGES * 8;
  const uint32_t xbar = smem_u32(bars + WS_WARPS * WS_MAX_STAGES);

  // Every launch is a programmatic dependent of the one before it, so that its
  // blocks are in place when that one ends; the first kernel of a call touches
  // nothing before then.
  if (a.first) {
    pdl_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;
  }
  pdl_launch_dependents();
  if (lane == 0) {
    for (int i = 0; i < a.stages; ++i) mbar_init(bar0 + 8 * i, 1);
    if (warp == 0) mbar_init(xbar, 1);
    fence_mbar_init();
  }
  __syncthreads();  // every warp waits on xbar

  const int nk = (a.K + 63) >> 6;
  // this block's part of the contraction, units [kbase, kbase + kunits)
  const int rank = a.split > 1 ? (int)cluster_rank() : 0;
  const int kbase = nk * rank / a.split, kunits = nk * (rank + 1) / a.split - kbase;
  const int b = a.split > 1 ? blockIdx.x / a.split : blockIdx.x;
  const int tile0 = b * a.tile_quot + min(b, a.tile_rem);
  const int tiles = a.tile_quot + (b < a.tile_rem ? 1 : 0);
  const int runs = tiles <= a.run ? 1 : (tiles + a.run - 1) / a.run;
  const int phases = (kunits + a.phase_units - 1) / a.phase_units;
  auto run_tiles = [&](int r) { return min(a.run, tiles - r * a.run); };
  auto phase_len = [&](int p) { return min(a.phase_units, kunits - p * a.phase_units); };  // units
  auto chunks_of = [&](int len) { return (len + S::UNITS - 1) / S::UNITS; };
  auto enter = [&](WsWalk& w) {  // this warp's share from here on, skipping empty ones
    for (; w.run < runs; ++w.run, w.phase = 0) {
      for (; w.phase < phases; ++w.phase) {
        const int per = chunks_of(phase_len(w.phase)), total = run_tiles(w.run) * per;
        w.v = total * warp / WS_WARPS;
        w.v_end = total * (warp + 1) / WS_WARPS;
        w.j = w.v / per;
        w.c = w.v - w.j * per;
        if (w.v < w.v_end) return;
      }
    }
  };

  // ---------------------------------------------------------------- weights in
  WsWalk in = {0, 0, 0, 0, 0, 0};
  const uint8_t* src = nullptr;       // the next chunk
  int in_per = 0, in_last = 0;        // chunks of a tile; bytes of its last chunk (16 rows)
  auto locate = [&]() {
    if (in.run >= runs) return;
    const int len = phase_len(in.phase);
    in_per = chunks_of(len);
    in_last = (len - (in_per - 1) * S::UNITS) * S::RECORD;
    src = a.W + ((int64_t)(tile0 + in.run * a.run + in.j) * RT * nk + kbase +
                 in.phase * a.phase_units + in.c * S::UNITS) * S::RECORD;
  };
  enter(in);
  locate();
  uint32_t slot_in = 0;               // byte offset of the next stage to fill, in its ring
  uint32_t bar_in = bar0;             // and its barrier
  int filled = 0;                     // stages filled and not yet consumed
  const uint32_t ring = sbase + a.ring_off + warp * a.stages * S::STAGE;
  const uint32_t ring_bytes = a.stages * S::STAGE, bar_end = bar0 + 8 * a.stages;
  bool skip = a.inject != 0;  // test hook
  auto fill = [&]() {  // the next stage: the units of one chunk
    if (in.run >= runs) return;
    const uint32_t bytes = in.c == in_per - 1 ? in_last : S::PIECE;
    if (lane == 0 && !skip) {
      // the second half of the last tile may lie past the matrix
      const int parts = RT == 1 ? 1 : min(RT, a.tiles16 - (tile0 + in.run * a.run + in.j) * RT);
      mbar_arrive_expect_tx(bar_in, parts * bytes);
#pragma unroll
      for (int i = 0; i < RT; ++i)
        if (i < parts) {
          const uint8_t* p = src + (int64_t)i * nk * S::RECORD;
          if (SWIGLU_CHECK_PTR(a.dbg, p, bytes, a.err))
            bulk_load(ring + slot_in + i * S::PIECE, p, bytes, bar_in);
        }
    }
    skip = false;
    src += bytes;
    slot_in += S::STAGE;
    bar_in += 8;
    if (slot_in == ring_bytes) {
      slot_in = 0;
      bar_in = bar0;
    }
    ++filled;
    if (++in.c == in_per) {
      in.c = 0;
      ++in.j;
      src += (int64_t)(RT * nk - phase_len(in.phase)) * S::RECORD;  // the next tile
    }
    if (++in.v == in.v_end) {
      ++in.phase;
      enter(in);
      locate();
    }
  };
  for (int i = 0; i < a.stages; ++i) fill();
  if (!a.first) pdl_wait();  // before the first read of a token row

  // ---------------------------------------------------------------- token rows
  // Units [u0, u0 + len) of the rows: bulk copies bring them.
  uint32_t xparity = 0;
  bool xlive = true;  // false, for the whole block, after a wait for the rows ran out: no more copies
  auto stage_rows = [&](int u0, int len) {
    const int xrow = S::xrow(a.phase_units);
    const int inside = min(len * 64, a.K - u0 * 64);  // elements of a row
    if (warp == 0 && xlive) {
      // what was read or written here before is ordered with the copies
      fence_proxy_async_shared();
      if (lane == 0) mbar_arrive_expect_tx(xbar, a.M * inside * 2);
      __syncwarp();
      if (lane < a.M) {
        const uint8_t* p = static_cast<const uint8_t*>(a.X) + ((int64_t)lane * a.K + u0 * 64) * 2;
        if (SWIGLU_CHECK_PTR(a.dbg, p, inside * 2, a.err))
          bulk_load(sbase + lane * xrow, p, inside * 2, xbar);
      }
    }
    // zeros from the end of a row to the end of its last unit
    const int gap = (len * 64 - inside) / 8;  // 16-byte pieces, 0..7
    if ((int)threadIdx.x < a.M * gap) {
      const int m = threadIdx.x / gap, c = threadIdx.x - m * gap;
      *reinterpret_cast<uint4*>(smem + m * xrow + inside * 2 + c * 16) = make_uint4(0, 0, 0, 0);
    }
    if (xlive) xlive = mbar_wait_bounded(xbar, xparity, a.wait_limit_ns, nullptr, a.err);
    xlive = __syncthreads_and(xlive) != 0;
    if (xlive) xparity ^= 1u;
  };

  // ---------------------------------------------------------------- products
  float4 acc[RT][NT];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[i][nt] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  };
  clear();
  float* const part = reinterpret_cast<float*>(smem + a.part_off);
  float* const tsum = reinterpret_cast<float*>(smem + a.tile_off);
  auto flush = [&](int j) {  // the partial of the run's tile j
    float4* p = reinterpret_cast<float4*>(part + (j + warp) * (S::PART / 4)) + lane;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) p[(i * NT + nt) * 32] = acc[i][nt];
    clear();
  };
  // Unit Q of a chunk: base addresses of the chunk's records (rc, the lane's
  // codes; rs, its scales) and of its token rows.
  auto multiply = [&](auto q, uint32_t rc, uint32_t rs, const uint32_t (&xu)[NT]) {
    constexpr int Q = decltype(q)::value, R = Q * S::RECORD;
    uint4 x0[NT], x1[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      x0[nt] = lds128_at<Q * 128>(xu[nt]);
      x1[nt] = lds128_at<Q * 128 + 64>(xu[nt]);
    }
    auto tile = [&](auto which) {
      constexpr int I = decltype(which)::value, RI = R + I * S::PIECE, Z = RI + S::GROUPS * 32;
      const uint4 cw = lds128_at<RI>(rc);
      const uint32_t w[4] = {cw.x, cw.y, cw.z, cw.w};  // rows g, g + 8 of k 0..31, then of 32..63
      const uint32_t sc0 = lds32_at<RI>(rs), sc1 = G32 ? lds32_at<RI + 32>(rs) : sc0;
      const uint32_t z0 = ZP ? lds16_at<Z>(rs - g * 2) : 0x808u;
      const uint32_t z1 = ZP && G32 ? lds16_at<Z + 16>(rs - g * 2) : z0;
      // A[h][f]: half h, elements k + {0..3} (f = 0) and k + {4..7}
      uint32_t A[2][2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t v = w[2 * h + r], z = h ? z1 : z0;
          const W4Off<BF16> off(r ? z >> 8 : z & 0xffu);
          A[h][0][r] = w4_first<BF16>(v, off);
          A[h][0][2 + r] = w4_first<BF16>(v >> 8, off);
          A[h][1][r] = w4_second<BF16>(v, off);
          A[h][1][2 + r] = w4_second<BF16>(v >> 8, off);
        }
      auto scale_in = [&](float4& o, float4 p, uint32_t sc) {
        const float sg = P::lo(sc), sh = P::hi(sc);
        o.x = fmaf(sg, p.x, o.x);
        o.y = fmaf(sg, p.y, o.y);
        o.z = fmaf(sh, p.z, o.z);
        o.w = fmaf(sh, p.w, o.w);
      };
      const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        auto half = [&](float4 c, int h, uint4 x) {
          c = mma_ws<BF16>(c, A[h][0][0], A[h][0][1], A[h][0][2], A[h][0][3], x.x, x.y);
          return mma_ws<BF16>(c, A[h][1][0], A[h][1][1], A[h][1][2], A[h][1][3], x.z, x.w);
        };
        float4 p = half(zero, 0, x0[nt]);
        if (G32) {
          scale_in(acc[I][nt], p, sc0);
          p = zero;
        }
        scale_in(acc[I][nt], half(p, 1, x1[nt]), sc1);
      }
    };
    tile(WsInt<0>{});
    if constexpr (RT > 1) tile(WsInt<1>{});
  };

  uint32_t slot_at = 0, bar_at = bar0, parity = 0;  // the next stage to consume
  bool live = true;  // false after a wait ran out: go through the motions, read nothing
  uint16_t* const out = static_cast<uint16_t*>(a.out);
  // The warps whose shares, of n tiles of `per` chunks laid end to end, meet
  // tile jt: their partials are at (jt + warp) * PART.
  auto meeting = [&](int n, int per, int jt) {
    const int total = n * per;
    const int s0 = total * lane / WS_WARPS, s1 = total * (lane + 1) / WS_WARPS;  // lane's share
    return __ballot_sync(0xffffffffu, lane < WS_WARPS && s0 < s1 && s0 < (jt + 1) * per &&
                                          s1 > jt * per);
  };
  auto plus = [](float4 a, float4 b) {
    return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
  };
  // The epilogue of 16 rows and 8 tokens, part `rest` of the run's tile jt: lane
  // (g, t) has rows g and g + 8 of tokens 2 t and 2 t + 1.
  auto finish = [&](int jt, int rest, float4 v, int run) {
    const int t16 = (tile0 + run * a.run + jt) * RT + rest / NT, m = rest % NT * 8 + 2 * t;
    auto put = [&](int row, int token, float x) {
      if (row >= a.rows || token >= a.M) return;
      uint16_t* o = out + (int64_t)token * a.rows + row;
      if (SWIGLU_CHECK_PTR(a.dbg, o, 2, a.err)) *o = P::rnd(x);
    };
    if (a.gate_up) {
      put(t16 * 8 + g, m, ft_silu(a.scale * v.x) * v.z);
      put(t16 * 8 + g, m + 1, ft_silu(a.scale * v.y) * v.w);
    } else {
      put(t16 * 16 + g, m, a.scale * v.x);
      put(t16 * 16 + g, m + 1, a.scale * v.y);
      put(t16 * 16 + g + 8, m, a.scale * v.z);
      put(t16 * 16 + g + 8, m + 1, a.scale * v.w);
    }
  };
  uint32_t xa[NT];  // this lane's token rows; columns past the last repeat it, unread
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
    xa[nt] = sbase + min(nt * 8 + g, a.M - 1) * S::xrow(a.phase_units) + t * 16;
  for (int run = 0; run < runs; ++run) {
    const int n = run_tiles(run);
    for (int phase = 0; phase < phases; ++phase) {
      const int len = phase_len(phase);
      if (phases > 1 || run == 0) {
        stage_rows(kbase + phase * a.phase_units, len);
      }
      const int per = chunks_of(len), total = n * per;  // chunks of a tile, of the run
      const int v0 = total * warp / WS_WARPS, v1 = total * (warp + 1) / WS_WARPS;
      int j = v0 / per, c = v0 - j * per;
      const int tail = len - (per - 1) * S::UNITS;  // units of a tile's last chunk
      uint32_t xu[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) xu[nt] = xa[nt] + c * (S::UNITS * 128);
      for (int v = v0; v < v1; ++v) {
        if (live && !mbar_try_wait(bar_at, parity))
          live = mbar_wait_bounded(bar_at, parity, a.wait_limit_ns, nullptr, a.err);
        live = __all_sync(0xffffffffu, live);
        const bool last = ++c == per;
        if (live) {
          uint32_t rc = ring + slot_at + lane * 16, rs = ring + slot_at + 512 + g * 4;
          int left = last ? tail : S::UNITS;
          constexpr int STEP = 4 / RT;  // independent chains in flight
          for (; left >= STEP; left -= STEP) {
            multiply(WsInt<0>{}, rc, rs, xu);
            multiply(WsInt<1>{}, rc, rs, xu);
            if constexpr (STEP == 4) {
              multiply(WsInt<2>{}, rc, rs, xu);
              multiply(WsInt<3>{}, rc, rs, xu);
            }
            rc += STEP * S::RECORD;
            rs += STEP * S::RECORD;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) xu[nt] += STEP * 128;
          }
          for (; left > 0; --left) {
            multiply(WsInt<0>{}, rc, rs, xu);
            rc += S::RECORD;
            rs += S::RECORD;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) xu[nt] += 128;
          }
          __syncwarp();
          --filled;
          slot_at += S::STAGE;
          bar_at += 8;
          if (slot_at == ring_bytes) {
            slot_at = 0;
            bar_at = bar0;
            parity ^= 1u;
          }
          fill();
        }
        if (last) {
          c = 0;
          flush(j++);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) xu[nt] = xa[nt];
        }
      }
      if (c != 0) flush(j);
      __syncthreads();
      // a tile's partials, in warp order; a warp takes 16 rows and 8 tokens at
      // a time.  Sums that are not final yet wait in tsum (for the next phase)
      // or in the place of the first partial (for the cluster).
      for (int i = warp; i < n * RT * NT; i += WS_WARPS) {
        const int jt = i / (RT * NT), rest = i % (RT * NT);
        const uint32_t meet = meeting(n, per, jt);
        float4* const p = reinterpret_cast<float4*>(part) + rest * 32 + lane;
        float4* const p0 = p + (jt + __ffs(meet) - 1) * (S::PART / 16);
        float4 v = *p0;
        for (uint32_t m = meet & (meet - 1); m != 0; m &= m - 1)
          v = plus(v, p[(jt + __ffs(m) - 1) * (S::PART / 16)]);
        if (a.phased) {
          float4* ts = reinterpret_cast<float4*>(tsum) + jt * (S::PART / 16) + rest * 32 + lane;
          if (phase > 0) v = plus(*ts, v);
          *ts = v;
        } else if (a.split > 1) {
          *p0 = v;
        }
        if (a.split == 1 && phase + 1 == phases) finish(jt, rest, v, run);
      }
      __syncthreads();
    }
    if (a.split > 1) {
      // the blocks' sums, in rank order
      cluster_arrive();
      cluster_wait();
      for (int i = warp * a.split + rank; i < n * RT * NT; i += WS_WARPS * a.split) {
        const int jt = i / (RT * NT), rest = i % (RT * NT);
        float4 q[8];  // all loads at once: they are all latency
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r < a.split) {
            uint32_t at = a.tile_off + jt * S::PART;
            if (!a.phased) {
              const int per = chunks_of(nk * (r + 1) / a.split - nk * r / a.split);
              at = a.part_off + (jt + __ffs(meeting(n, per, jt)) - 1) * S::PART;
            }
            q[r] = cluster_load4(cluster_map(sbase + at + rest * 512 + lane * 16, r));
          }
        float4 v = q[0];
#pragma unroll
        for (int r = 1; r < 8; ++r)
          if (r < a.split) v = plus(v, q[r]);
        finish(jt, rest, v, run);
      }
      __syncwarp();
      cluster_arrive();  // before the partials are written again, or the block goes
      cluster_wait();
    }
  }
  // after a wait ran out: no copy may land after the block has gone
  if (!xlive) mbar_wait_bounded(xbar, xparity, a.wait_limit_ns, nullptr, a.err);
  if (!live)
    for (; filled > 0; --filled) {
      mbar_wait_bounded(bar_at, parity, a.wait_limit_ns, nullptr, a.err);
      bar_at += 8;
      if (bar_at == bar_end) {
        bar_at = bar0;
        parity ^= 1u;
      }
    }
}

}  // namespace swiglu
