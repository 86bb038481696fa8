// experts.cuh -- the experts of a mixture-of-experts layer for a few tokens,
// with 16-bit or 4-bit weights: gate/up over the chosen experts' rows, and the
// down products with the weighted sum over a token's experts.
//
// Bound by streaming the chosen experts' weights (4-bit: and by unpacking them,
// as in w4_stream.cuh, whose unit records and code forms are used here).
//   * 16-bit weights come as tensor-map boxes of 16 rows x 64 k (one copy per
//     unit, issued by one lane, whole 128-byte lines, swizzled so that the
//     lanes' 16-byte reads meet no bank conflicts); 4-bit ones as runs of
//     records.  Each warp has a ring of its own, so that warps never wait for
//     one another while they stream.
//   * An expert meets its own few tokens, 8 NT at most per pass over its
//     weights.  Token rows are read by the lanes that need them, a chunk ahead
//     in registers, through L1 (gate/up: all experts read rows of the same few
//     tokens) or L2 (down: the hidden values of the expert's own assignments).
//
// Work: gate/up gives a block a contiguous run of (expert, tile) items; down
// gives it the tiles of its output rows and goes through all experts.  Either
// way a run's chunks are laid end to end and shared evenly by the block's
// warps; partial tiles (down: weighted sums per token and warp) meet in shared
// memory in warp order, so results are deterministic.
//
// Measured (whole layer with the router, bf16): 16-bit weights, 16 tokens over 8
// of 64 experts, 2048/1024: 124 us for 711 MB (5.7 TB/s of 6.8; gate/up 85 us
// alone, DRAM 71%), 64 tokens 158 us; one token, 2 of 8 experts of 1024/2816 18.5
// us, of which the router and the two kernels' starts are some 12.  One token over
// all 8 experts of 4096/11008: 342 us for 2.16 GB = 6.3 TB/s, 8 tokens 369 us.
// 4-bit: one token 20 us, 32 tokens over 8 of 128 experts of 2048/512 in groups of
// 32 73 us (199 MB; gate/up: issue slots 51%, ALU 44%, 96 instructions to unpack
// and multiply a unit, and each expert's two to three tokens cannot share more).
// (With constant rows' products in place of subtractions: 82 us.)
// An expert with more than 8 NT tokens is streamed once per 8 NT of them.
#pragma once

#include "w4_stream.cuh"

namespace swiglu {

template <bool W4, int NT, bool G32, bool ZP>
struct WxShape {
  // 4-bit: 12 warps of 168 registers (16 of 128 spill); 16-bit weights need more
  // warps to hide their latencies than registers (16 tokens, 64 experts: 125
  // against 130 us)
  static constexpr int WARPS = W4 ? 12 : 16;
  static constexpr int TOKENS = 8 * NT;                       // tokens of a pass
  static constexpr int UNITS = W4 && NT == 1 ? 8 : 4;         // units of a chunk
  static constexpr int HALF = UNITS / 2;                      // units whose token rows are loaded at once
  static constexpr int STAGE_UNITS = W4 ? UNITS : HALF;       // units of a ring stage
  static constexpr int GROUPS = G32 ? 2 : 1;
  static constexpr int RECORD = W4 ? 512 + GROUPS * (ZP ? 48 : 32) : 2048;
  static constexpr int STAGE = STAGE_UNITS * RECORD;
};

// One warp's place: run, chunk v of its share [v, v_end), which is chunk c of
// the run's piece j (gate/up: an item; down: an entry).
struct WxWalk {
  int run, v, v_end, j, c;
};

template <bool BF16, bool W4, int NT, bool G32, bool ZP>
__global__ void __launch_bounds__(WxShape<W4, NT, G32, ZP>::WARPS * 32, 1)
    experts_kernel(const __grid_constant__ CUtensorMap tm, const FtArgs a) {
  using S = WxShape<W4, NT, G32, ZP>;
  using P = Ft16<BF16>;
  constexpr int GROUPS = S::GROUPS, RECORD = S::RECORD, STAGE = S::STAGE, UNITS = S::UNITS,
                HALF = S::HALF, WX_WARPS = S::WARPS, WX_THREADS = WX_WARPS * 32;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[WX_WARPS * WX_MAX_STAGES];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t bar0 = smem_u32(bars) + warp * WX_MAX_STAGES * 8;
  const bool combine = a.mode == FT_COMBINE;

  ft_begin(a);
  if (lane == 0) {
    for (int i = 0; i < a.stages; ++i) mbar_init(bar0 + 8 * i, 1);
    fence_mbar_init();
  }
  const FtLists l = ft_lists(smem + a.list_off, a, S::TOKENS);
  float* const red = reinterpret_cast<float*>(smem + a.red_off);
  if (combine)
    for (int i = threadIdx.x; i < WX_WARPS * a.M * 16; i += WX_THREADS) red[i] = 0.0f;
  ft_build_lists<WX_THREADS>(a, l, S::TOKENS);

  const int nk = (a.K + 63) >> 6, per = (nk + UNITS - 1) / UNITS;  // units, chunks of a tile
  const int entries = *l.n;
  const int items = combine ? a.tiles : entries * a.tiles;
  const int item0 = (int)((int64_t)items * blockIdx.x / gridDim.x);
  const int item1 = (int)((int64_t)items * (blockIdx.x + 1) / gridDim.x);
  const int run_len = combine ? 1 : a.run;
  const int runs = (item1 - item0 + run_len - 1) / run_len;
  auto pieces_of = [&](int r) { return combine ? entries : min(run_len, item1 - item0 - r * run_len); };
  auto enter = [&](WxWalk& w) {  // this warp's share of run w.run, skipping runs without one
    for (; w.run < runs; ++w.run) {
      const int total = pieces_of(w.run) * per;
      w.v = total * warp / WX_WARPS;
      w.v_end = total * (warp + 1) / WX_WARPS;
      if (w.v < w.v_end) {
        w.j = w.v / per;
        w.c = w.v - w.j * per;
        return;
      }
    }
  };
  auto step = [&](WxWalk& w) {  // to the next chunk; true where it belongs to another piece
    const bool turn = ++w.c == per;
    if (turn) {
      w.c = 0;
      ++w.j;
    }
    if (++w.v < w.v_end) return turn;
    ++w.run;
    enter(w);
    return true;
  };
  auto piece_at = [&](int run, int j, int& tile) -> int2 {  // its tile and entry
    const int item = item0 + (combine ? run : run * run_len + j);
    const int en = combine ? j : (int)((unsigned)item / (unsigned)a.tiles);
    tile = combine ? item : item - en * a.tiles;
    return l.entry[en];
  };

  // ---------------------------------------------------------------- weights in
  // (a tensor-map box is a swizzle atom: 1024-byte aligned)
  const uint32_t ring = ((smem_u32(smem) + a.ring_off + 1023) & ~1023u) + warp * a.stages * STAGE;
  const uint32_t ring_bytes = a.stages * STAGE;
  WxWalk in = {0, 0, 0, 0, 0};
  const uint8_t* src = nullptr;   // 4-bit: the next records
  int in_row = 0, in_z = 0;       // 16-bit: first row of the tile, its slice of the tensor map
  auto locate = [&]() {
    if (in.run >= runs) return;
    int tile;
    const int2 e = piece_at(in.run, in.j, tile);
    if (W4) {
      src = a.W + (int64_t)(e.x & 0xffff) * a.expert_bytes +
            ((int64_t)tile * nk + in.c * UNITS) * RECORD;
    } else {  // gate/up: 8 rows of two slices, else 16 of one
      in_row = tile * (combine ? 16 : 8);
      in_z = (e.x & 0xffff) * (combine ? 1 : 2);
    }
  };
  uint32_t slot_in = 0, bar_in = bar0;
  int filled = 0;
  bool skip = a.inject != 0;  // test hook
  int in_half = 0;  // 16-bit: a chunk's halves are stages of their own
  auto fill = [&]() {
    if (in.run >= runs) return;
    const int u = in.c * UNITS + in_half * HALF, n = min(S::STAGE_UNITS, nk - u);
    if (lane == 0 && !skip) {
      mbar_arrive_expect_tx(bar_in, n * RECORD);
      if (W4) {
        bulk_load(ring + slot_in, src, n * RECORD, bar_in);
      } else {
        for (int q = 0; q < n; ++q)
          tma_load_3d(ring + slot_in + q * RECORD, &tm, bar_in, (u + q) * 64, in_row, in_z);
      }
    }
    skip = false;
    if (W4) src += n * RECORD;
    slot_in += STAGE;
    bar_in += 8;
    if (slot_in == ring_bytes) {
      slot_in = 0;
      bar_in = bar0;
    }
    ++filled;
    if (!W4 && in_half == 0 && u + HALF < nk) {
      in_half = 1;
      return;
    }
    in_half = 0;
    if (step(in)) locate();
  };
  enter(in);
  WxWalk at = in;
  locate();
  for (int i = 0; i < a.stages; ++i) fill();
  if (!ft_waits_first(a)) pdl_wait();  // before the first read of a token row

  // ---------------------------------------------------------------- products
  // token rows of the first and the second half of a chunk: [8 tokens][unit][half unit]
  using Rows = uint4[NT][HALF][2];
  Rows xa, xb;
  const uint8_t* px[NT];  // this lane's token rows, at its elements of unit 0
  auto tokens_of = [&](const WxWalk& w) {
    int tile;
    const int2 e = piece_at(w.run, w.j, tile);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      // columns past the entry's last token repeat its first; no one reads them
      int r = e.y + (nt * 8 + g < e.x >> 16 ? nt * 8 + g : 0);
      if (!combine) r = (int)((unsigned)l.at[r] / (unsigned)a.topk);
      px[nt] = static_cast<const uint8_t*>(a.X) + ((int64_t)r * a.K + t * 8) * 2;
    }
  };
  auto load_x = [&](Rows& v, int u) {  // units u .. u + HALF - 1
    const int left = a.K - u * 64;     // elements of the rows from there on
    const bool whole = left >= HALF * 64;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint8_t* p = px[nt] + (int64_t)u * 128;
      if (whole && SWIGLU_CHECK_PTR(a.dbg, p, HALF * 128 - 48, a.err)) {
#pragma unroll
        for (int q = 0; q < HALF; ++q) {
          v[nt][q][0] = ft_load16(p + q * 128);
          v[nt][q][1] = ft_load16(p + q * 128 + 64);
        }
      } else {
#pragma unroll
        for (int q = 0; q < HALF; ++q)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint8_t* s = p + q * 128 + h * 64;
            v[nt][q][h] = q * 64 + h * 32 + t * 8 < left && SWIGLU_CHECK_PTR(a.dbg, s, 16, a.err)
                              ? ft_load16(s)
                              : make_uint4(0, 0, 0, 0);
          }
      }
    }
  };
  const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float4 acc[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) acc[nt] = zero;
  // the partial tile of a piece: its place in shared memory, or added to the
  // warp's weighted sums per token
  auto flush = [&](int run, int j) {
    if (combine) {
      int tile;
      const int2 e = piece_at(run, j, tile);
      float* y = red + warp * a.M * 16 + g;
      __syncwarp();
      auto put = [&](int m, float lo, float hi) {
        if (m >= e.x >> 16) return;
        const float w = l.w[e.y + m];
        float* yt = y + (unsigned)l.at[e.y + m] / (unsigned)a.topk * 16;
        yt[0] += w * lo;
        yt[8] += w * hi;
      };
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        put(nt * 8 + 2 * t, acc[nt].x, acc[nt].z);
        put(nt * 8 + 2 * t + 1, acc[nt].y, acc[nt].w);
      }
    } else {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        reinterpret_cast<float4*>(red)[((j + warp) * NT + nt) * 32 + lane] = acc[nt];
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) acc[nt] = zero;
  };
  // 16-bit: this lane's 16 bytes of row g, k 0..31 and 32..63, in a swizzled box
  const uint32_t sw0 = g * 128 + (t ^ g) * 16, sw1 = g * 128 + ((4 + t) ^ g) * 16;
  auto unit16 = [&](auto q, const Rows& x, uint32_t box) {
    constexpr int Q = decltype(q)::value % HALF, R = Q * RECORD;  // in a half's own stage
    const uint4 g0 = lds128_at<R>(box + sw0), g1 = lds128_at<R>(box + sw1);
    const uint4 h0 = lds128_at<R + 1024>(box + sw0), h1 = lds128_at<R + 1024>(box + sw1);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint4 x0 = x[nt][Q][0], x1 = x[nt][Q][1];
      float4 p = mma_ws<BF16>(acc[nt], g0.x, h0.x, g0.y, h0.y, x0.x, x0.y);
      p = mma_ws<BF16>(p, g0.z, h0.z, g0.w, h0.w, x0.z, x0.w);
      p = mma_ws<BF16>(p, g1.x, h1.x, g1.y, h1.y, x1.x, x1.y);
      acc[nt] = mma_ws<BF16>(p, g1.z, h1.z, g1.w, h1.w, x1.z, x1.w);
    }
  };
  auto unit4 = [&](auto q, const Rows& x, uint32_t rc, uint32_t rs) {
    constexpr int Q = decltype(q)::value % HALF, R = decltype(q)::value * RECORD;
    constexpr int Z = R + GROUPS * 32;
    const uint4 cw = lds128_at<R>(rc);
    const uint32_t w[4] = {cw.x, cw.y, cw.z, cw.w};  // rows g, g + 8 of k 0..31, then of 32..63
    const uint32_t sc0 = lds32_at<R>(rs), sc1 = G32 ? lds32_at<R + 32>(rs) : sc0;
    const uint32_t zp0 = ZP ? lds16_at<Z>(rs - g * 2) : 0x808u;
    const uint32_t zp1 = ZP && G32 ? lds16_at<Z + 16>(rs - g * 2) : zp0;
    float4 p[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) p[nt] = zero;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t lo = w[2 * h], hi = w[2 * h + 1], zp = h ? zp1 : zp0;
      const W4Off<BF16> zl(zp & 0xffu), zh(zp >> 8);
      const uint32_t f0 = w4_first<BF16>(lo, zl), f1 = w4_first<BF16>(hi, zh);
      const uint32_t f2 = w4_first<BF16>(lo >> 8, zl), f3 = w4_first<BF16>(hi >> 8, zh);
      const uint32_t s0 = w4_second<BF16>(lo, zl), s1 = w4_second<BF16>(hi, zh);
      const uint32_t s2 = w4_second<BF16>(lo >> 8, zl), s3 = w4_second<BF16>(hi >> 8, zh);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4 v = x[nt][Q][h];
        p[nt] = mma_ws<BF16>(p[nt], f0, f1, f2, f3, v.x, v.y);
        p[nt] = mma_ws<BF16>(p[nt], s0, s1, s2, s3, v.z, v.w);
        if (G32 || h) {
          const uint32_t sc = h ? sc1 : sc0;
          const float sg = P::lo(sc), sh = P::hi(sc);
          acc[nt].x = fmaf(sg, p[nt].x, acc[nt].x);
          acc[nt].y = fmaf(sg, p[nt].y, acc[nt].y);
          acc[nt].z = fmaf(sh, p[nt].z, acc[nt].z);
          acc[nt].w = fmaf(sh, p[nt].w, acc[nt].w);
          p[nt] = zero;
        }
      }
    }
  };

  uint32_t slot_at = 0, bar_at = bar0, parity = 0;
  bool live = true;  // false after a wait ran out: go through the motions, read nothing
  if (at.run < runs) {
    tokens_of(at);
    load_x(xa, at.c * UNITS);
  }
  uint16_t* const out = static_cast<uint16_t*>(a.out);
  for (int run = 0; run < runs; ++run) {
    while (at.run == run) {
      const int j = at.j, left = nk - at.c * UNITS;
      uint32_t rec;
      auto acquire = [&]() {  // the next stage
        if (live && !mbar_try_wait(bar_at, parity))
          live = mbar_wait_bounded(bar_at, parity, a.wait_limit_ns, nullptr, a.err);
        live = __all_sync(0xffffffffu, live);
        rec = ring + slot_at;
      };
      auto release = [&]() {
        if (!live) return;
        __syncwarp();
        --filled;
        slot_at += STAGE;
        bar_at += 8;
        if (slot_at == ring_bytes) {
          slot_at = 0;
          bar_at = bar0;
          parity ^= 1u;
        }
        fill();
      };
      auto unit = [&](auto q, const Rows& x) {
        if (W4)
          unit4(q, x, rec + lane * 16, rec + 512 + g * 4);
        else
          unit16(q, x, rec);
      };
      auto units = [&](auto first, const Rows& x) {  // past the end of a row the stage is stale
        constexpr int Q = decltype(first)::value;
        if (left >= Q + HALF) {
          unit(WsInt<Q>{}, x);
          if constexpr (HALF > 1) unit(WsInt<Q + 1>{}, x);
          if constexpr (HALF > 2) {
            unit(WsInt<Q + 2>{}, x);
            unit(WsInt<Q + 3>{}, x);
          }
        } else {
          if (left > Q) unit(WsInt<Q>{}, x);
          if constexpr (HALF > 2) {
            if (left > Q + 1) unit(WsInt<Q + 1>{}, x);
            if (left > Q + 2) unit(WsInt<Q + 2>{}, x);
          }
        }
      };
      if (left > HALF) load_x(xb, at.c * UNITS + HALF);
      acquire();
      if (live) units(WsInt<0>{}, xa);
      if (!W4) {
        release();
        if (left > HALF) acquire();
      }
      const bool last = step(at);  // of this piece
      if (at.run < runs) {
        if (last) tokens_of(at);
        load_x(xa, at.c * UNITS);
      }
      if (live) units(WsInt<HALF>{}, xb);
      if (W4 || left > HALF) release();
      if (last) flush(run, j);
    }
    __syncthreads();
    if (combine) {
      const int tile = item0 + run;
      for (int i = threadIdx.x; i < a.M * 16; i += WX_THREADS) {
        float part[WX_WARPS], v = 0.0f;
#pragma unroll
        for (int w = 0; w < WX_WARPS; ++w) part[w] = red[w * a.M * 16 + i];
#pragma unroll
        for (int w = 0; w < WX_WARPS; ++w) {
          v += part[w];
          red[w * a.M * 16 + i] = 0.0f;  // for the next run
        }
        const int r = tile * 16 + (i & 15);
        if (r < a.rows) {
          uint16_t* o = out + (int64_t)(i >> 4) * a.rows + r;
          if (SWIGLU_CHECK_PTR(a.dbg, o, 2, a.err)) *o = P::rnd(a.scale * v);
        }
      }
    } else {
      // a tile's partials, in warp order: those of the warps whose shares meet it
      const int n = pieces_of(run), total = n * per;
      const int s0 = total * lane / WX_WARPS, s1 = total * (lane + 1) / WX_WARPS;  // lane's share
      for (int i = warp; i < n * NT; i += WX_WARPS) {
        const int j = i / NT, nt = i % NT;
        uint32_t meet = __ballot_sync(0xffffffffu, lane < WX_WARPS && s0 < s1 &&
                                                       s0 < (j + 1) * per && s1 > j * per);
        float4 v = zero;
        for (; meet != 0; meet &= meet - 1) {
          const float4 q = reinterpret_cast<const float4*>(red)[((j + __ffs(meet) - 1) * NT + nt) * 32 + lane];
          v = make_float4(v.x + q.x, v.y + q.y, v.z + q.z, v.w + q.w);
        }
        int tile;
        const int2 e = piece_at(run, j, tile);
        const int u = tile * 8 + g;
        auto put = [&](int m, float gate, float up) {
          if (m >= e.x >> 16 || u >= a.rows) return;
          uint16_t* o = out + (int64_t)(e.y + m) * a.rows + u;
          if (SWIGLU_CHECK_PTR(a.dbg, o, 2, a.err)) *o = P::rnd(ft_silu(a.scale * gate) * up);
        };
        put(nt * 8 + 2 * t, v.x, v.z);
        put(nt * 8 + 2 * t + 1, v.y, v.w);
      }
    }
    __syncthreads();
  }
  // after a wait ran out: no copy may land after the block has gone
  if (!live)
    for (; filled > 0; --filled) {
      mbar_wait_bounded(bar_at, parity, a.wait_limit_ns, nullptr, a.err);
      bar_at += 8;
      if (bar_at == bar0 + 8 * a.stages) {
        bar_at = bar0;
        parity ^= 1u;
      }
    }
}

}  // namespace swiglu
