// fewtok.cuh -- products of a few tokens (1..64) with weight matrices, bound
// by streaming the weights from HBM: 4-bit weights with group scales, and the
// experts of a mixture-of-experts layer (16-bit or 4-bit).
//
//   Y[m, r] = sum_k X[m, k] W[r, k],   W[r, k] = s[r, k/G] (q[r, k] - z[r, k/G])
//
// Work: a tile of 16 weight rows (for gate/up 8 rows of Wg and the 8 rows of
// Wu of the same hidden units) over the whole contraction is one block's; its
// 8 warps split each chunk of KC elements of k, and their partial tiles meet
// in shared memory at the tile's end, in warp order, so results are
// deterministic and no block waits for another.  A ninth warp keeps a ring of
// chunks filled by bulk copies (cp.async.bulk): the tile's weights, its group
// scales, and the same chunk of the token rows.
//
// Products: mma.sync m16n8k16 with the weights as the 16-row operand and 8
// tokens as the columns.  The contraction's order is free, so lane t of a
// quad takes 8 consecutive k of every 32: token rows and 16-bit weights are
// read from shared memory by 16-byte loads, and a 4-bit tile is stored so that
// one 16-byte load brings a lane all its codes of 64 k.  A code becomes a
// 16-bit number by OR-ing it into the mantissa of 128 (bf16) or 1024 (fp16)
// and subtracting 128 + z (1024 + z): both steps are exact, so the tensor core
// multiplies whole numbers by the tokens and each 32-k partial sum is scaled
// by its group's scale in fp32.  No weight is ever rounded.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../csrc/sm103_ptx.cuh"

namespace swiglu {

constexpr int FT_WARPS = 8;  // consumer warps; one more warp issues the copies
constexpr int FT_CONSUMERS = FT_WARPS * 32;
constexpr int FT_THREADS = FT_CONSUMERS + 32;
constexpr int FT_MAX_STAGES = 16;
constexpr int FT_MAX_TOKENS = 64;
constexpr int FT_MAX_EXPERTS = 512;
constexpr int FT_MAX_TOPK = 16;

enum FtMode : int { FT_LINEAR = 0, FT_GATE_UP = 1, FT_COMBINE = 2 };

struct FtArgs {
  int mode;          // FT_LINEAR: out = rnd(scale v); FT_GATE_UP: out = rnd(SiLU(scale g) u);
                     //   FT_COMBINE: out[t] = rnd(scale sum_j w[t, j] v_j) over a token's experts
  int M;             // tokens
  int K;             // contraction, a multiple of 8
  int rows;          // rows of out: output features, or hidden units (gate/up)
  int tiles;         // 16-row tiles of one expert's matrix
  const uint8_t* W;  // weights: row-major 16-bit [E][R][K], or packed 4-bit matrices
  int64_t expert_bytes;
  const void* X;     // [*, K]: token rows, or (FT_COMBINE) one row per assignment
  void* out;
  float scale;
  // 4-bit weights: group = 1 << group_log2, groups per row, offsets of the
  // scales and the zero points in a packed matrix
  int group_log2, groups, zeros;
  int64_t scales_off, zeros_off;
  // mixture of experts
  int E, topk;
  const int* idx;    // [M, topk] experts (values outside 0..E-1: none)
  const float* wts;  // [M, topk]
  int dependent;     // launched as a programmatic dependent of the kernel before it
  int idx_ready;     // idx was complete before that kernel began
  int clear_err;     // block 0 clears the error word (first kernel of a call)
  int inject;        // test hook: the first stage is never filled
  // shared-memory plan
  int xrows;         // token rows of a stage
  int stages, stage_bytes, sc_off, z_off, x_off, list_off, red_off, ring_off;
  uint64_t wait_limit_ns;
  int* err;
#ifdef SWIGLU_DEBUG
  DbgWin dbg;        // out, X, idx / wts, workspace
#endif
};

// 16-bit storage types: packed arithmetic and conversions
template <bool BF16>
struct Ft16;
template <>
struct Ft16<true> {
  static constexpr uint32_t MAGIC = 0x43004300u;  // 128, 128
  static __device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ float lo(uint32_t v) { return __uint_as_float(v << 16); }
  static __device__ __forceinline__ float hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
  static __device__ __forceinline__ uint16_t rnd(float v) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }
};
template <>
struct Ft16<false> {
  static constexpr uint32_t MAGIC = 0x64006400u;  // 1024, 1024
  static __device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ float lo(uint32_t v) {
    return __half2float(__ushort_as_half((unsigned short)(v & 0xffffu)));
  }
  static __device__ __forceinline__ float hi(uint32_t v) {
    return __half2float(__ushort_as_half((unsigned short)(v >> 16)));
  }
  static __device__ __forceinline__ uint16_t rnd(float v) {
    return __half_as_ushort(__float2half_rn(v));
  }
};

template <bool BF16>
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  if (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}

// Four 16-bit pairs of whole numbers q - z from the 8 codes of a word: nibble
// i (i < 4) and nibble i + 4 are the halves of pair i; pairs 0 and 2 belong to
// row g (zlo = 128 + z or 1024 + z, twice), 1 and 3 to row g + 8 (zhi).
template <bool BF16>
__device__ __forceinline__ void ft_codes(uint32_t w, uint32_t zlo, uint32_t zhi, uint32_t (&a)[4]) {
  constexpr uint32_t M = Ft16<BF16>::MAGIC;
  a[0] = Ft16<BF16>::sub2((w & 0x000f000fu) | M, zlo);
  a[1] = Ft16<BF16>::sub2(((w >> 4) & 0x000f000fu) | M, zhi);
  a[2] = Ft16<BF16>::sub2(((w >> 8) & 0x000f000fu) | M, zlo);
  a[3] = Ft16<BF16>::sub2(((w >> 12) & 0x000f000fu) | M, zhi);
}

__device__ __forceinline__ float ft_silu(float g) { return g / (1.0f + __expf(-g)); }

// k per ring stage: 1024 for 4-bit weights (8 KB of codes), 512 for 16-bit
// weights (16 KB) and where the token rows would make a stage too large.
template <bool W4, int NT>
struct FtShape {
  static constexpr int KC = W4 && NT <= 2 ? 1024 : 512;
  static constexpr int UNITS = KC / 64 / FT_WARPS;  // 64-k units of a warp per stage
  // row stride in shared memory: 64 bytes past a multiple of 128, so that the
  // 16-byte loads of two neighbouring rows fall into different banks
  static constexpr int ROW = KC * 2 + 64;
  static constexpr int TOKENS = 8 * NT;             // tokens of one pass over a tile
  static constexpr int RED_BYTES = 2 * FT_WARPS * NT * 512;
};

__device__ __forceinline__ void ft_bar_consumers() {
  asm volatile("bar.sync 1, %0;" ::"n"(FT_CONSUMERS) : "memory");
}

// The experts' token lists of a call, built by every block for itself in
// shared memory: the valid assignments sorted by (expert, token), and one
// entry per run of at most `per` assignments of one expert.  An expert named
// twice by one token counts once, with the sum of its weights.
struct FtLists {
  unsigned long long* mask;  // [E] tokens of an expert
  int* start;                // [E] first position of an expert
  int2* entry;               // {expert | count << 16, first position}
  float* w;                  // [M * topk] weight, by position
  uint16_t* at;              // [M * topk] assignment, by position
  int* n;                    // entries
};
__host__ __device__ inline int ft_max_entries(int M, int topk, int E, int per) {
  const int a = M * topk, b = (E < a ? E : a) + a / per;
  return a < b ? a : b;
}
__host__ __device__ inline int ft_lists_bytes(int M, int topk, int E, int per) {
  const int b = 16 + E * 12 + ft_max_entries(M, topk, E, per) * 8 + M * topk * 6;
  return (b + 127) & ~127;
}
__device__ __forceinline__ FtLists ft_lists(uint8_t* p, const FtArgs& a, int per) {
  FtLists l;
  l.n = reinterpret_cast<int*>(p);
  l.mask = reinterpret_cast<unsigned long long*>(p + 16);
  l.entry = reinterpret_cast<int2*>(l.mask + a.E);
  l.start = reinterpret_cast<int*>(l.entry + ft_max_entries(a.M, a.topk, a.E, per));
  l.w = reinterpret_cast<float*>(l.start + a.E);
  l.at = reinterpret_cast<uint16_t*>(l.w + a.M * a.topk);
  return l;
}

// Assignment i's expert, or -1 where it is none or an earlier one of the same
// token names the same expert; with `w` the sum of the expert's weights.
__device__ __forceinline__ int ft_assignment(const FtArgs& a, int i, float* w) {
  const int t = i / a.topk, j = i - t * a.topk;
  const int* row = a.idx + t * a.topk;
  if (!SWIGLU_CHECK_PTR(a.dbg, row, 4 * (int64_t)a.topk, a.err)) return -1;
  const int e = __ldcg(row + j);
  if (e < 0 || e >= a.E) return -1;
  for (int q = 0; q < j; ++q)
    if (__ldcg(row + q) == e) return -1;
  if (w != nullptr) {
    float s = __ldcg(a.wts + i);
    for (int q = j + 1; q < a.topk; ++q)
      if (__ldcg(row + q) == e) s += __ldcg(a.wts + t * a.topk + q);
    *w = s;
  }
  return e;
}

__device__ __forceinline__ void ft_build_lists(const FtArgs& a, const FtLists& l, int per) {
  const int total = a.M * a.topk;
  for (int e = threadIdx.x; e < a.E; e += FT_THREADS) l.mask[e] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < total; i += FT_THREADS) {
    const int e = ft_assignment(a, i, nullptr);
    if (e >= 0) atomicOr(l.mask + e, 1ull << (i / a.topk));
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    int pos = 0, ent = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + threadIdx.x;
      const int n = e < a.E ? __popcll(l.mask[e]) : 0, c = (n + per - 1) / per;
      int ns = n, cs = c;  // inclusive sums over the 32 experts
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int nu = __shfl_up_sync(0xffffffffu, ns, d), cu = __shfl_up_sync(0xffffffffu, cs, d);
        if ((int)threadIdx.x >= d) {
          ns += nu;
          cs += cu;
        }
      }
      const int p0 = pos + ns - n, c0 = ent + cs - c;
      if (e < a.E) l.start[e] = p0;
      for (int q = 0; q < c; ++q)
        l.entry[c0 + q] = make_int2(e | min(per, n - q * per) << 16, p0 + q * per);
      pos += __shfl_sync(0xffffffffu, ns, 31);
      ent += __shfl_sync(0xffffffffu, cs, 31);
    }
    if (threadIdx.x == 0) *l.n = ent;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < total; i += FT_THREADS) {
    float w = 0.0f;
    const int e = ft_assignment(a, i, a.mode == FT_COMBINE ? &w : nullptr);
    if (e < 0) continue;
    const int p = l.start[e] + __popcll(l.mask[e] & ((1ull << (i / a.topk)) - 1));
    l.at[p] = (uint16_t)i;
    l.w[p] = w;
  }
  __syncthreads();
}

template <bool BF16, bool W4, int NT, bool MOE>
__global__ void __launch_bounds__(FT_THREADS, 2) ft_kernel(const FtArgs a) {
  using S = FtShape<W4, NT>;
  using P = Ft16<BF16>;
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  auto full_bar = [&](int i) { return sbase + 8u * i; };
  auto empty_bar = [&](int i) { return sbase + 8u * (FT_MAX_STAGES + i); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + 16 * FT_MAX_STAGES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (blockIdx.x == 0 && a.clear_err && threadIdx.x == 0) *a.err = 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(full_bar(i), 1);
      mbar_init(empty_bar(i), FT_WARPS);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  // A mixture of experts reads idx before anything else.  Where idx comes from
  // the kernel just before (gate/up after the router) that kernel is waited
  // for here, and only then may the next one start: so the combining kernel,
  // whose idx the router wrote, needs no wait before its weights.
  const bool wait_first = MOE && a.dependent && !a.idx_ready;
  if (wait_first) pdl_wait();
  if (a.mode != FT_COMBINE) pdl_launch_dependents();

  FtLists l = {};
  float* yacc = reinterpret_cast<float*>(smem + a.list_off - FT_MAX_TOKENS * 16 * 4);
  if (MOE) {
    l = ft_lists(smem + a.list_off, a, S::TOKENS);
    if (a.mode == FT_COMBINE)
      for (int i = threadIdx.x; i < a.M * 16; i += FT_THREADS) yacc[i] = 0.0f;
    ft_build_lists(a, l, S::TOKENS);
  } else {
    __syncthreads();
  }

  // the block's work: items of one tile; a combining item goes through every
  // entry, the others belong to one
  const int entries = MOE ? *l.n : (a.M + S::TOKENS - 1) / S::TOKENS;
  const bool combine = MOE && a.mode == FT_COMBINE;
  const int items = combine ? a.tiles : entries * a.tiles;
  const int segs = combine ? entries : 1;
  auto segment = [&](int item, int s, int& tile, int& expert, int& first, int& count) {
    const int en = combine ? s : item / a.tiles;
    tile = combine ? item : item - en * a.tiles;
    if (MOE) {
      const int2 v = l.entry[en];
      expert = v.x & 0xffff;
      count = v.x >> 16;
      first = v.y;
    } else {
      expert = 0;
      first = en * S::TOKENS;
      count = min(S::TOKENS, a.M - first);
    }
  };

  if (warp == FT_WARPS) {
    // ---------------------------------------------------------------- producer
    uint32_t issued = 0, parity = 0;
    auto bytes_w = [&](int tile, int kn) -> uint32_t {
      if (W4) {
        const uint32_t ng = (uint32_t)((kn + (1 << a.group_log2) - 1) >> a.group_log2);
        return (uint32_t)((kn + 63) >> 6) * 512u + ng * (a.zeros ? 48u : 32u);
      }
      const int rows = a.mode == FT_GATE_UP ? 16 : min(16, a.rows - tile * 16);
      return (uint32_t)(rows * kn * 2);
    };
    auto load_w = [&](int slot, int tile, int expert, int k0, int kn) {
      const uint32_t dst = sbase + a.ring_off + slot * a.stage_bytes, bar = full_bar(slot);
      const uint8_t* w = a.W + (int64_t)expert * a.expert_bytes;
      if (W4) {
        const int ng = (kn + (1 << a.group_log2) - 1) >> a.group_log2;
        const int64_t g0 = (int64_t)tile * a.groups + (k0 >> a.group_log2);
        if (lane == 0)
          bulk_load(dst, w + ((int64_t)tile * ((a.K + 63) >> 6) + (k0 >> 6)) * 512,
                    (uint32_t)((kn + 63) >> 6) * 512u, bar);
        if (lane == 1) bulk_load(dst + a.sc_off, w + a.scales_off + g0 * 32, (uint32_t)ng * 32u, bar);
        if (lane == 2 && a.zeros)
          bulk_load(dst + a.z_off, w + a.zeros_off + g0 * 16, (uint32_t)ng * 16u, bar);
      } else if (lane < 16) {
        const bool gu = a.mode == FT_GATE_UP;
        const int r = gu ? tile * 8 + (lane & 7) : tile * 16 + lane;
        if (r < a.rows)
          bulk_load(dst + lane * S::ROW,
                    w + ((int64_t)(r + (gu && lane >= 8 ? a.rows : 0)) * a.K + k0) * 2,
                    (uint32_t)kn * 2u, bar);
      }
    };
    auto load_x = [&](int slot, int first, int count, int k0, int kn) {
      const uint32_t dst = sbase + a.ring_off + slot * a.stage_bytes + a.x_off;
      for (int i = lane; i < count; i += 32) {
        int64_t r = first + i;
        if (MOE && a.mode != FT_COMBINE) r = l.at[first + i] / a.topk;
        bulk_load(dst + i * S::ROW, static_cast<const uint8_t*>(a.X) + (r * a.K + k0) * 2,
                  (uint32_t)kn * 2u, full_bar(slot));
      }
    };
    // A dependent launch first fills the ring with weights, which the kernel
    // before it does not write, then waits for it and adds the token rows.
    int pre = 0;
    if (a.dependent && !wait_first) {
      for (int item = blockIdx.x; item < items && pre < a.stages; item += gridDim.x)
        for (int s = 0; s < segs && pre < a.stages; ++s) {
          int tile, expert, first, count;
          segment(item, s, tile, expert, first, count);
          for (int k0 = 0; k0 < a.K && pre < a.stages; k0 += S::KC, ++pre) {
            if (a.inject && pre == 0) continue;
            const int kn = min(S::KC, a.K - k0);
            if (lane == 0)
              mbar_arrive_expect_tx(full_bar(pre), bytes_w(tile, kn) + (uint32_t)(count * kn * 2));
            __syncwarp();
            load_w(pre, tile, expert, k0, kn);
            issued |= 1u << pre;
          }
        }
      pdl_wait();
    }
    int stage = 0, n = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int item = blockIdx.x; ok && item < items; item += gridDim.x)
      for (int s = 0; ok && s < segs; ++s) {
        int tile, expert, first, count;
        segment(item, s, tile, expert, first, count);
        for (int k0 = 0; k0 < a.K; k0 += S::KC, ++n) {
          const int kn = min(S::KC, a.K - k0);
          const bool skip = a.inject && n == 0;
          if (n >= pre && !skip) {
            int w = 1;
            if (lane == 0)
              w = mbar_wait_bounded(empty_bar(stage), phase ^ 1u, a.wait_limit_ns, abort_flag, a.err);
            ok = __shfl_sync(0xffffffffu, w, 0) != 0;
            if (!ok) break;
            if (lane == 0)
              mbar_arrive_expect_tx(full_bar(stage), bytes_w(tile, kn) + (uint32_t)(count * kn * 2));
            __syncwarp();
            load_w(stage, tile, expert, k0, kn);
            issued |= 1u << stage;
            parity = (parity & ~(1u << stage)) | (phase << stage);
          }
          if (!skip) load_x(stage, first, count, k0, kn);
          if (++stage == a.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    if (!ok)  // no copy may land after the block has gone
      for (int i = 0; i < a.stages; ++i)
        if (issued & (1u << i))
          mbar_wait_bounded(full_bar(i), (parity >> i) & 1u, a.wait_limit_ns, nullptr, a.err);
    return;
  }

  // ------------------------------------------------------------------ consumers
  const int g = lane >> 2, t = lane & 3;
  float* red = reinterpret_cast<float*>(smem + a.red_off);
  int stage = 0, buf = 0;
  uint32_t phase = 0;
  bool live = true;  // false after a wait ran out: go through the motions, read nothing
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    int tile = 0;
    for (int s = 0; s < segs; ++s) {
      int expert, first, count;
      segment(item, s, tile, expert, first, count);
      const int nts = (count + 7) >> 3;
      float acc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[nt][c] = 0.0f;

      for (int k0 = 0; k0 < a.K; k0 += S::KC) {
        if (live)
          live = __all_sync(0xffffffffu, mbar_wait_bounded(full_bar(stage), phase, a.wait_limit_ns,
                                                           abort_flag, a.err));
        if (live) {
          const uint32_t sw = sbase + a.ring_off + stage * a.stage_bytes;
          const int left = a.K - k0;
          const bool tail = left < S::KC;
#pragma unroll
          for (int i = 0; i < S::UNITS; ++i) {
            const int u = warp + FT_WARPS * i;
            if (tail && u * 64 >= left) continue;
            // k of this lane past the end of the row: what lies there is stale
            const bool z0 = tail && u * 64 + t * 8 >= left;
            const bool z1 = tail && u * 64 + 32 + t * 8 >= left;
            const uint4 zero = make_uint4(0, 0, 0, 0);
            uint32_t A[4][4];
            float s0g = 0.0f, s0h = 0.0f, s1g = 0.0f, s1h = 0.0f;
            if (W4) {
              const uint4 c = lds128(sw + u * 512 + lane * 16);
              const int g0 = (u * 64) >> a.group_log2;
              int g1 = (u * 64 + 32) >> a.group_log2;
              if (tail && u * 64 + 32 >= left) g1 = g0;
              const uint32_t sc0 = lds32(sw + a.sc_off + g0 * 32 + g * 4);
              const uint32_t sc1 = lds32(sw + a.sc_off + g1 * 32 + g * 4);
              uint32_t q0 = 0x0808u, q1 = 0x0808u;
              if (a.zeros) {
                q0 = lds16(sw + a.z_off + g0 * 16 + g * 2);
                q1 = lds16(sw + a.z_off + g1 * 16 + g * 2);
              }
              s0g = P::lo(sc0);
              s0h = P::hi(sc0);
              s1g = P::lo(sc1);
              s1h = P::hi(sc1);
              const uint32_t z0l = P::MAGIC + (q0 & 0xffu) * 0x10001u;
              const uint32_t z0h = P::MAGIC + (q0 >> 8) * 0x10001u;
              const uint32_t z1l = P::MAGIC + (q1 & 0xffu) * 0x10001u;
              const uint32_t z1h = P::MAGIC + (q1 >> 8) * 0x10001u;
              ft_codes<BF16>(c.x, z0l, z0h, A[0]);
              ft_codes<BF16>(c.y, z0l, z0h, A[1]);
              ft_codes<BF16>(c.z, z1l, z1h, A[2]);
              ft_codes<BF16>(c.w, z1l, z1h, A[3]);
            } else {
              const uint32_t p = sw + g * S::ROW + u * 128 + t * 16;
              uint4 g0 = lds128(p), g1 = lds128(p + 64);
              uint4 h0 = lds128(p + 8 * S::ROW), h1 = lds128(p + 8 * S::ROW + 64);
              if (z0) g0 = h0 = zero;
              if (z1) g1 = h1 = zero;
              A[0][0] = g0.x, A[0][1] = h0.x, A[0][2] = g0.y, A[0][3] = h0.y;
              A[1][0] = g0.z, A[1][1] = h0.z, A[1][2] = g0.w, A[1][3] = h0.w;
              A[2][0] = g1.x, A[2][1] = h1.x, A[2][2] = g1.y, A[2][3] = h1.y;
              A[3][0] = g1.z, A[3][1] = h1.z, A[3][2] = g1.w, A[3][3] = h1.w;
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (nt >= nts) continue;
              const int r = min(nt * 8 + g, a.xrows - 1);
              const uint32_t p = sw + a.x_off + r * S::ROW + u * 128 + t * 16;
              uint4 x0 = lds128(p), x1 = lds128(p + 64);
              if (z0) x0 = zero;
              if (z1) x1 = zero;
              if (W4) {
                float p0[4] = {0.0f, 0.0f, 0.0f, 0.0f}, p1[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma_16816<BF16>(p0, A[0][0], A[0][1], A[0][2], A[0][3], x0.x, x0.y);
                mma_16816<BF16>(p1, A[2][0], A[2][1], A[2][2], A[2][3], x1.x, x1.y);
                mma_16816<BF16>(p0, A[1][0], A[1][1], A[1][2], A[1][3], x0.z, x0.w);
                mma_16816<BF16>(p1, A[3][0], A[3][1], A[3][2], A[3][3], x1.z, x1.w);
                acc[nt][0] = fmaf(s0g, p0[0], fmaf(s1g, p1[0], acc[nt][0]));
                acc[nt][1] = fmaf(s0g, p0[1], fmaf(s1g, p1[1], acc[nt][1]));
                acc[nt][2] = fmaf(s0h, p0[2], fmaf(s1h, p1[2], acc[nt][2]));
                acc[nt][3] = fmaf(s0h, p0[3], fmaf(s1h, p1[3], acc[nt][3]));
              } else {
                mma_16816<BF16>(acc[nt], A[0][0], A[0][1], A[0][2], A[0][3], x0.x, x0.y);
                mma_16816<BF16>(acc[nt], A[1][0], A[1][1], A[1][2], A[1][3], x0.z, x0.w);
                mma_16816<BF16>(acc[nt], A[2][0], A[2][1], A[2][2], A[2][3], x1.x, x1.y);
                mma_16816<BF16>(acc[nt], A[3][0], A[3][1], A[3][2], A[3][3], x1.z, x1.w);
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty_bar(stage));
        if (++stage == a.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }

      // the warps' partial tiles meet, in warp order
      float* mine = red + ((buf * FT_WARPS + warp) * NT * 32 + lane) * 4;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        *reinterpret_cast<float4*>(mine + nt * 128) =
            make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
      ft_bar_consumers();
      const float* part = red + buf * FT_WARPS * NT * 128;
      buf ^= 1;
      // element (row of the tile, token of the entry) of the summed tile
      auto sum = [&](int row, int m) {
        const float* p = part + (m >> 3) * 128 + ((row & 7) * 4 + ((m & 7) >> 1)) * 4 + (m & 1) +
                         2 * (row >> 3);
        float v = p[0];
#pragma unroll
        for (int w = 1; w < FT_WARPS; ++w) v += p[w * NT * 128];
        return v;
      };
      uint16_t* out = static_cast<uint16_t*>(a.out);
      if (a.mode == FT_GATE_UP) {
        for (int i = threadIdx.x; i < count * 8; i += FT_CONSUMERS) {
          const int m = i >> 3, u = tile * 8 + (i & 7);
          if (u >= a.rows) continue;
          const float v = ft_silu(a.scale * sum(i & 7, m)) * sum((i & 7) + 8, m);
          uint16_t* o = out + (int64_t)(first + m) * a.rows + u;
          if (SWIGLU_CHECK_PTR(a.dbg, o, 2, a.err)) *o = P::rnd(v);
        }
      } else {
        for (int i = threadIdx.x; i < count * 16; i += FT_CONSUMERS) {
          const int m = i >> 4, r = tile * 16 + (i & 15);
          if (r >= a.rows) continue;
          const float v = sum(i & 15, m);
          if (combine) {
            // one thread per (token, row): an expert's entries name a token once
            yacc[(l.at[first + m] / a.topk) * 16 + (i & 15)] += l.w[first + m] * v;
          } else {
            uint16_t* o = out + (int64_t)(first + m) * a.rows + r;
            if (SWIGLU_CHECK_PTR(a.dbg, o, 2, a.err)) *o = P::rnd(a.scale * v);
          }
        }
      }
    }
    if (combine) {
      if (segs == 0) tile = item;
      ft_bar_consumers();
      for (int i = threadIdx.x; i < a.M * 16; i += FT_CONSUMERS) {
        const int r = tile * 16 + (i & 15);
        if (r < a.rows) {
          uint16_t* o = static_cast<uint16_t*>(a.out) + (int64_t)(i >> 4) * a.rows + r;
          if (SWIGLU_CHECK_PTR(a.dbg, o, 2, a.err)) *o = P::rnd(a.scale * yacc[i]);
        }
        yacc[i] = 0.0f;
      }
    }
  }
  // a dependent block without work still may not finish before the kernel it
  // depends on has (the next call's first kernel waits for this one alone)
  if (a.dependent && !wait_first) pdl_wait();
}

}  // namespace swiglu
