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
//   * 4-bit: the sums that cancel the magic numbers are not prepared as in
//     w4_stream.cuh, where all rows share them; an accumulator starts with the
//     product of the same token elements and a constant row, -(m + z) in 16
//     bits, which doubles the tensor core's work, idle otherwise.
//
// Work: gate/up gives a block a contiguous run of (expert, tile) items; down
// gives it the tiles of its output rows and goes through all experts.  Either
// way a run's chunks are laid end to end and shared evenly by the block's
// warps; partial tiles (down: weighted sums per token and warp) meet in shared
// memory in warp order, so results are deterministic.
#pragma once

#include "w4_stream.cuh"

namespace swiglu {

constexpr int WX_WARPS = 12;
constexpr int WX_THREADS = WX_WARPS * 32;
constexpr int WX_MAX_STAGES = 8;

template <bool W4, int NT, bool G32, bool ZP>
struct WxShape {
  static constexpr int TOKENS = 8 * NT;                       // tokens of a pass
  static constexpr int UNITS = W4 && NT == 1 ? 4 : 2;         // units of a chunk, a ring stage
  static constexpr int GROUPS = G32 ? 2 : 1;
  static constexpr int RECORD = W4 ? 512 + GROUPS * (ZP ? 48 : 32) : 2048;
  static constexpr int STAGE = UNITS * RECORD;
};

// One warp's place: run, chunk v of its share [v, v_end), which is chunk c of
// the run's piece j.
struct WxWalk {
  int run, v, v_end, j, c;
};

template <bool BF16, bool W4, int NT, bool G32, bool ZP>
__global__ void __launch_bounds__(WX_THREADS, 1)
    experts_kernel(const __grid_constant__ CUtensorMap tm, const FtArgs a) {
  using S = WxShape<W4, NT, G32, ZP>;
  using P = Ft16<BF16>;
  constexpr int GROUPS = S::GROUPS, RECORD = S::RECORD, STAGE = S::STAGE, UNITS = S::UNITS;
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
    const int en = combine ? j : item / a.tiles;
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
  bool skip = a.inject && warp == 0;  // test hook
  auto fill = [&]() {
    if (in.run >= runs) return;
    const uint32_t bytes = min(UNITS, nk - in.c * UNITS) * RECORD;
    if (lane == 0 && !skip) {
      mbar_arrive_expect_tx(bar_in, bytes);
      if (W4) {
        bulk_load(ring + slot_in, src, bytes, bar_in);
      } else {
        for (int q = 0; q < UNITS && in.c * UNITS + q < nk; ++q)
          tma_load_3d(ring + slot_in + q * RECORD, &tm, bar_in, (in.c * UNITS + q) * 64, in_row, in_z);
      }
    }
    skip = false;
    if (W4) src += bytes;
    slot_in += STAGE;
    bar_in += 8;
    if (slot_in == ring_bytes) {
      slot_in = 0;
      bar_in = bar0;
    }
    ++filled;
    if (step(in)) locate();
  };
  enter(in);
  WxWalk at = in;
  locate();
  for (int i = 0; i < a.stages; ++i) fill();
  if (!ft_waits_first(a)) pdl_wait();  // before the first read of a token row

  // ---------------------------------------------------------------- products
  // token rows of a chunk: [8 tokens][unit][half]
  uint4 x[NT][UNITS][2];
  const uint8_t* px[NT];  // this lane's token rows, at its elements of unit 0
  bool has[NT];
  auto tokens_of = [&](const WxWalk& w) {
    int tile;
    const int2 e = piece_at(w.run, w.j, tile);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      has[nt] = nt * 8 + g < e.x >> 16;
      int r = e.y + (has[nt] ? nt * 8 + g : 0);
      if (!combine) r = l.at[r] / a.topk;
      px[nt] = static_cast<const uint8_t*>(a.X) + ((int64_t)r * a.K + t * 8) * 2;
    }
  };
  auto load_x = [&](uint4 (&v)[NT][UNITS][2], int c) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint8_t* p = px[nt] + (int64_t)c * (UNITS * 128);
      const int left = has[nt] ? a.K - c * (UNITS * 64) - t * 8 : 0;  // elements from p on
#pragma unroll
      for (int q = 0; q < UNITS; ++q)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t* s = p + q * 128 + h * 64;
          v[nt][q][h] = q * 64 + h * 32 < left && SWIGLU_CHECK_PTR(a.dbg, s, 16, a.err)
                            ? ft_load16(s)
                            : make_uint4(0, 0, 0, 0);
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
        float* yt = y + (l.at[e.y + m] / a.topk) * 16;
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
  auto unit16 = [&](auto q, uint32_t box) {
    constexpr int Q = decltype(q)::value, R = Q * RECORD;
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
  auto unit4 = [&](auto q, uint32_t rc, uint32_t rs) {
    constexpr int Q = decltype(q)::value, R = Q * RECORD, Z = R + GROUPS * 32;
    const uint4 cw = lds128_at<R>(rc);
    const uint32_t w[4] = {cw.x, cw.y, cw.z, cw.w};  // rows g, g + 8 of k 0..31, then of 32..63
    const uint32_t sc0 = lds32_at<R>(rs), sc1 = G32 ? lds32_at<R + 32>(rs) : sc0;
    constexpr uint32_t M = P::MAGIC, LO = 0x000f000fu, HI = 0x00f000f0u, NEG = M | 0x80008000u;
    // -(m + z) of rows g and g + 8, twice each; fp16: for the first and second form
    uint32_t n0[4], n1[4];
    auto negatives = [&](uint32_t (&n)[4], uint32_t z) {
      const uint32_t zl = ZP ? (z & 0xffu) * 0x10001u : 0x00080008u;
      const uint32_t zh = ZP ? (z >> 8) * 0x10001u : 0x00080008u;
      n[0] = NEG | zl;
      n[1] = NEG | zh;
      n[2] = BF16 ? n[0] : NEG | zl << 4;
      n[3] = BF16 ? n[1] : NEG | zh << 4;
    };
    negatives(n0, ZP ? lds16_at<Z>(rs - g * 2) : 0);
    negatives(n1, ZP && G32 ? lds16_at<Z + 16>(rs - g * 2) : 0);
    float4 p[NT], r[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) p[nt] = r[nt] = zero;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t lo = w[2 * h], hi = w[2 * h + 1];
      const uint32_t(&n)[4] = G32 && h ? n1 : n0;
      const uint32_t f0 = and_or<LO>(lo, M), f1 = and_or<LO>(hi, M);
      const uint32_t f2 = and_or<LO>(lo >> 8, M), f3 = and_or<LO>(hi >> 8, M);
      const uint32_t s0 = BF16 ? and_or<LO>(lo >> 4, M) : and_or<HI>(lo, M);
      const uint32_t s1 = BF16 ? and_or<LO>(hi >> 4, M) : and_or<HI>(hi, M);
      const uint32_t s2 = BF16 ? and_or<LO>(lo >> 12, M) : and_or<HI>(lo >> 8, M);
      const uint32_t s3 = BF16 ? and_or<LO>(hi >> 12, M) : and_or<HI>(hi >> 8, M);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4 v = x[nt][Q][h];
        p[nt] = mma_ws<BF16>(p[nt], n[0], n[1], n[0], n[1], v.x, v.z);
        r[nt] = mma_ws<BF16>(r[nt], n[2], n[3], n[2], n[3], v.y, v.w);
        p[nt] = mma_ws<BF16>(p[nt], f0, f1, f2, f3, v.x, v.z);
        r[nt] = mma_ws<BF16>(r[nt], s0, s1, s2, s3, v.y, v.w);
        if (G32 || h) {  // fp16: the second form's sums are 16 times too large
          const uint32_t sc = h ? sc1 : sc0;
          const float sg = P::lo(sc), sh = P::hi(sc), by = BF16 ? 1.0f : 0.0625f;
          acc[nt].x = fmaf(sg, fmaf(by, r[nt].x, p[nt].x), acc[nt].x);
          acc[nt].y = fmaf(sg, fmaf(by, r[nt].y, p[nt].y), acc[nt].y);
          acc[nt].z = fmaf(sh, fmaf(by, r[nt].z, p[nt].z), acc[nt].z);
          acc[nt].w = fmaf(sh, fmaf(by, r[nt].w, p[nt].w), acc[nt].w);
          p[nt] = r[nt] = zero;
        }
      }
    }
  };

  uint32_t slot_at = 0, bar_at = bar0, parity = 0;
  bool live = true;  // false after a wait ran out: go through the motions, read nothing
  if (at.run < runs) {
    tokens_of(at);
    load_x(x, at.c);
  }
  uint16_t* const out = static_cast<uint16_t*>(a.out);
  for (int run = 0; run < runs; ++run) {
    while (at.run == run) {
      if (live && !mbar_try_wait(bar_at, parity))
        live = mbar_wait_bounded(bar_at, parity, a.wait_limit_ns, nullptr, a.err);
      live = __all_sync(0xffffffffu, live);
      const int j = at.j, left = nk - at.c * UNITS;
      const bool last = step(at);  // of this piece
      uint4 xn[NT][UNITS][2];
      if (at.run < runs) {
        if (last) tokens_of(at);
        load_x(xn, at.c);
      }
      if (live) {
        const uint32_t rec = ring + slot_at;
        auto unit = [&](auto q) {
          if (W4)
            unit4(q, rec + lane * 16, rec + 512 + g * 4);
          else
            unit16(q, rec);
        };
        unit(WsInt<0>{});
        // past the end of a row the stage is stale: its products are not added
        if (left > 1) unit(WsInt<1>{});
        if constexpr (UNITS == 4) {
          if (left > 2) unit(WsInt<2>{});
          if (left > 3) unit(WsInt<3>{});
        }
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
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int q = 0; q < UNITS; ++q) {
          x[nt][q][0] = xn[nt][q][0];
          x[nt][q][1] = xn[nt][q][1];
        }
      if (last) flush(run, j);
    }
    __syncthreads();
    if (combine) {
      const int tile = item0 + run;
      for (int i = threadIdx.x; i < a.M * 16; i += WX_THREADS) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < WX_WARPS; ++w) {
          v += red[w * a.M * 16 + i];
          red[w * a.M * 16 + i] = 0.0f;
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
