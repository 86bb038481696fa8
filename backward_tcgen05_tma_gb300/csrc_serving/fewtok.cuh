// fewtok.cuh -- products of a few tokens (1..64) with weight matrices, bound
// by streaming the weights from HBM: 4-bit weights with group scales, and the
// experts of a mixture-of-experts layer (16-bit or 4-bit).
//
//   Y[m, r] = sum_k X[m, k] W[r, k],   W[r, k] = s[r, k/G] (q[r, k] - z[r, k/G])
//
// Work: a tile of 16 RT weight rows (for gate/up, each 16 are 8 rows of Wg and
// the 8 rows of Wu of the same hidden units) over the whole contraction, cut
// into units of 64 k.  A block takes a run of tiles, lays their units end to
// end and gives each of its 16 warps an equal share; a share that ends inside
// a tile leaves a partial tile in shared memory, and at the end of the run the
// block adds each tile's partials in order, applies the epilogue and writes.
// So warps never wait for one another while they stream, shares are even for
// any size, and results are deterministic.  The combining (down) kernel of a
// mixture of experts lays the units of ALL experts' tiles of the same output
// rows end to end, and each warp adds its weighted partials per token.
//
// Loads: every lane copies exactly the 16-byte pieces of the weights that it
// will multiply (cp.async, zero-filled past the end of a row) into a ring of
// its own in shared memory, several units ahead: a queue per lane, with no
// barriers, no swizzle (neighbouring lanes are neighbours there) and no
// registers held.  The token rows, which every tile reads again, come through
// the L1 cache, one unit ahead in registers.
//
// Products: mma.sync m16n8k16 with the weights as the 16-row operand and 8
// tokens as the columns.  The contraction's order is free, so lane t of a
// quad takes 8 consecutive k of every 32: token rows and 16-bit weights come
// in 16-byte pieces, and a 4-bit tile is stored so that one 16-byte piece
// holds all of a lane's codes of 64 k.  A code becomes a 16-bit number by
// OR-ing it into the mantissa of 128 (bf16) or 1024 (fp16) and subtracting
// 128 + z (1024 + z): both steps are exact, so the tensor core multiplies
// whole numbers by the tokens and each group's partial sum is scaled in fp32.
// No weight is ever rounded.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../csrc/sm103_ptx.cuh"

namespace swiglu {

constexpr int FT_WARPS = 16;
constexpr int FT_THREADS = FT_WARPS * 32;
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
  int tiles;         // 16 RT-row tiles of one expert's matrix
  int tiles16;       // ... and its 16-row tiles
  const uint8_t* W;  // weights: row-major 16-bit [E][R][K], or packed 4-bit matrices
  int64_t expert_bytes;
  const void* X;     // [*, K]: token rows, or (FT_COMBINE) one row per assignment
  void* out;
  float scale;
  int group_log2, zeros;  // 4-bit weights: group = 1 << group_log2, zero points
  // mixture of experts
  int E, topk;
  const int* idx;    // [M, topk] experts (values outside 0..E-1: none)
  const float* wts;  // [M, topk]
  int dependent;     // launched as a programmatic dependent of the kernel before it
  int idx_ready;     // idx was complete before that kernel began
  int clear_err;     // block 0 clears the error word (first kernel of a call)
  // shared-memory plan
  int depth;         // units a warp's ring holds
  int run;           // tiles of one run
  int list_off, red_off, ring_off;
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

// The four operand registers of one 16-k product from the codes of rows g (lo)
// and g + 8 (hi), as whole numbers q - z: bits 0..7 and 16..23 of each word
// are used (zlo, zhi = 128 + z or 1024 + z of the two rows, twice).
template <bool BF16>
__device__ __forceinline__ void ft_codes(uint32_t lo, uint32_t hi, uint32_t zlo, uint32_t zhi,
                                         uint32_t (&a)[4]) {
  constexpr uint32_t M = Ft16<BF16>::MAGIC;
  a[0] = Ft16<BF16>::sub2((lo & 0x000f000fu) | M, zlo);
  a[1] = Ft16<BF16>::sub2((hi & 0x000f000fu) | M, zhi);
  a[2] = Ft16<BF16>::sub2(((lo >> 4) & 0x000f000fu) | M, zlo);
  a[3] = Ft16<BF16>::sub2(((hi >> 4) & 0x000f000fu) | M, zhi);
}

__device__ __forceinline__ float ft_silu(float g) { return g / (1.0f + __expf(-g)); }

// One unit's place in a warp's ring.
template <bool W4, int RT, int NT, bool G32, bool ZP>
struct FtUnit {
  static constexpr int TOKENS = 8 * NT;                 // tokens of one pass over a tile
  static constexpr int GROUPS = G32 ? 2 : 1;            // groups of 64 k
  static constexpr int W = 0;                           // RT x (4-bit: 512, 16-bit: 2048) bytes
  static constexpr int RECORD = 512 + GROUPS * (ZP ? 48 : 32);  // a packed unit in memory
  static constexpr int S = RT * (W4 ? 512 : 2048);      // RT x GROUPS x 128: two scales per lane
  static constexpr int Z = S + (W4 ? RT * GROUPS * 128 : 0);  // and two zero points (in 4 bytes)
  static constexpr int BYTES = Z + (ZP ? RT * GROUPS * 128 : 0);
  static constexpr int PART = RT * NT * 512;            // a partial tile
};

__device__ __forceinline__ void cp_async_cg16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
// 16 bytes through the L1 cache.  Not the read-only path: the rows may be
// written while this kernel's prologue runs (before griddepcontrol.wait).
__device__ __forceinline__ uint4 ft_load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ void cp_async_ca4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Wait until at most n of this thread's committed groups are incomplete.
__device__ __forceinline__ void cp_async_wait(int n) {
  switch (n) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
    case 6: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;
  }
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

// A warp's way through its block's work: runs of tiles, in each run the warp's
// share [v, v_end) of the units laid end to end, unit v = piece v / nk, k-unit
// v % nk.  A piece is a tile of the run (linear, gate/up) or one entry's tile
// (combining).
struct FtWalk {
  int run, v, v_end, piece, u;
};

template <bool BF16, bool W4, int RT, int NT, bool G32, bool ZP, bool MOE>
__global__ void __launch_bounds__(FT_THREADS, 1) ft_kernel(const FtArgs a) {
  using U = FtUnit<W4, RT, NT, G32, ZP>;
  using P = Ft16<BF16>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

  if (blockIdx.x == 0 && a.clear_err && threadIdx.x == 0) *a.err = 0;
  // A mixture of experts reads idx before anything else.  Where idx comes from
  // the kernel just before (gate/up after the router) that kernel is waited
  // for here, and only then may the next one start: so the combining kernel,
  // whose idx the router wrote, needs no wait before its weights.
  const bool wait_first = MOE && a.dependent && !a.idx_ready;
  if (wait_first) pdl_wait();
  if (a.mode != FT_COMBINE) pdl_launch_dependents();

  const bool combine = MOE && a.mode == FT_COMBINE;
  FtLists l = {};
  float* red = reinterpret_cast<float*>(smem + a.red_off);
  if (MOE) {
    l = ft_lists(smem + a.list_off, a, U::TOKENS);
    if (combine)
      for (int i = threadIdx.x; i < FT_WARPS * a.M * 16 * RT; i += FT_THREADS) red[i] = 0.0f;
    ft_build_lists(a, l, U::TOKENS);
  }

  // the block's share of the items (tile, or entry and tile): a contiguous run
  const int nk = (a.K + 63) >> 6;
  const int entries = MOE ? *l.n : (a.M + U::TOKENS - 1) / U::TOKENS;
  const int64_t items = combine ? a.tiles : (int64_t)entries * a.tiles;
  const int item0 = (int)(items * blockIdx.x / gridDim.x);
  const int item1 = (int)(items * (blockIdx.x + 1) / gridDim.x);
  const int run_len = combine ? 1 : a.run;
  const int runs = (item1 - item0 + run_len - 1) / run_len;
  auto pieces_of = [&](int r) { return combine ? entries : min(run_len, item1 - item0 - r * run_len); };
  auto enter = [&](FtWalk& w) {  // this warp's share of run w.run, skipping runs without one
    for (; w.run < runs; ++w.run) {
      const int64_t total = (int64_t)pieces_of(w.run) * nk;
      w.v = (int)(total * warp / FT_WARPS);
      w.v_end = (int)(total * (warp + 1) / FT_WARPS);
      if (w.v < w.v_end) {
        w.piece = w.v / nk;
        w.u = w.v - w.piece * nk;
        return;
      }
    }
  };
  auto piece_at = [&](int run, int piece, int& tile, int& expert, int& first, int& count) {
    const int item = item0 + (combine ? run : run * run_len + piece);
    const int en = combine ? piece : item / a.tiles;
    tile = combine ? item : item - en * a.tiles;
    if (MOE) {
      const int2 v = l.entry[en];
      expert = v.x & 0xffff;
      count = v.x >> 16;
      first = v.y;
    } else {
      expert = 0;
      first = en * U::TOKENS;
      count = min(U::TOKENS, a.M - first);
    }
  };

  // ---------------------------------------------------------------- copies in
  const uint32_t ring = smem_u32(smem) + a.ring_off + warp * a.depth * U::BYTES;
  FtWalk in = {0, 0, 0, 0, 0};
  const uint8_t *pw[RT], *pw8[RT];  // this lane's sources at u = 0
  auto weights_of = [&](const FtWalk& w) {
    int tile, expert, first, count;
    piece_at(w.run, w.piece, tile, expert, first, count);
    const uint8_t* m = a.W + (int64_t)expert * a.expert_bytes;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int t16 = min(tile * RT + i, a.tiles16 - 1);  // a tile past the end repeats the last
      if (W4) {
        pw[i] = m + (int64_t)t16 * nk * U::RECORD;
      } else {
        // a row past the end repeats the last one (its results are not stored)
        const bool gu = a.mode == FT_GATE_UP;
        const int64_t r0 = gu ? t16 * 8 + g : min(t16 * 16 + g, a.rows - 1);
        const int64_t r1 = gu ? a.rows + t16 * 8 + g : min(t16 * 16 + 8 + g, a.rows - 1);
        pw[i] = m + (r0 * a.K + t * 8) * 2;
        pw8[i] = m + (r1 * a.K + t * 8) * 2;
      }
    }
  };
  const uint8_t* px[NT];  // the token rows of this lane's columns
  bool has_x[NT];
  auto tokens_of = [&](const FtWalk& w) {
    int tile, expert, first, count;
    piece_at(w.run, w.piece, tile, expert, first, count);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int c = nt * 8 + g;
      has_x[nt] = c < count;
      int64_t r = first + (has_x[nt] ? c : 0);
      if (MOE && !combine) r = l.at[r] / a.topk;
      px[nt] = static_cast<const uint8_t*>(a.X) + (r * a.K + t * 8) * 2;
    }
  };
  // bytes of the 16 at element k of a row that lie inside it (K % 8 == 0): 16 or 0
  auto inside = [&](int k) { return k < a.K ? 16u : 0u; };
  auto copy_w = [&](uint32_t slot, int u) {
    const uint32_t d = slot + lane * 16;
    if (W4) {
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const uint8_t* rec = pw[i] + (int64_t)u * U::RECORD;
        cp_async_cg16(d + U::W + i * 512, rec + lane * 16, 16u);
#pragma unroll
        for (int h = 0; h < U::GROUPS; ++h) {
          const uint32_t at = (i * U::GROUPS + h) * 128 + lane * 4;
          cp_async_ca4(slot + U::S + at, rec + 512 + h * 32 + g * 4);
          if (ZP) cp_async_ca4(slot + U::Z + at, rec + 512 + U::GROUPS * 32 + h * 16 + (g >> 1) * 4);
        }
      }
    } else {
      const uint32_t b0 = inside(u * 64 + t * 8), b1 = inside(u * 64 + 32 + t * 8);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int64_t o0 = b0 ? (int64_t)u * 128 : 0, o1 = b1 ? (int64_t)u * 128 + 64 : 0;
        cp_async_cg16(d + U::W + i * 2048, pw[i] + o0, b0);
        cp_async_cg16(d + U::W + i * 2048 + 512, pw[i] + o1, b1);
        cp_async_cg16(d + U::W + i * 2048 + 1024, pw8[i] + o0, b0);
        cp_async_cg16(d + U::W + i * 2048 + 1536, pw8[i] + o1, b1);
      }
    }
  };
  const uint4 none = make_uint4(0, 0, 0, 0);
  auto load_x = [&](uint4 (&x)[2], int nt, int u) {
    const bool in0 = has_x[nt] && u * 64 + t * 8 < a.K, in1 = has_x[nt] && u * 64 + 32 + t * 8 < a.K;
    const uint8_t* p = px[nt] + (int64_t)u * 128;
    x[0] = in0 && SWIGLU_CHECK_PTR(a.dbg, p, 16, a.err) ? ft_load16(p) : none;
    x[1] = in1 && SWIGLU_CHECK_PTR(a.dbg, p + 64, 16, a.err) ? ft_load16(p + 64) : none;
  };
  auto step = [&](FtWalk& w) {  // to the next unit; true where it belongs to another piece
    if (++w.v == w.v_end) {
      ++w.run;
      enter(w);
      return true;
    }
    if (++w.u == nk) {
      w.u = 0;
      ++w.piece;
      return true;
    }
    return false;
  };

  // fill the ring; a dependent launch copies weights, which the kernel before
  // it does not write, then waits for it before it reads token rows
  enter(in);
  const FtWalk begin = in;
  const int ahead = a.depth - 1;
  if (in.run < runs) weights_of(in);
  for (int i = 0; i < ahead; ++i) {
    if (in.run < runs) {
      copy_w(ring + i * U::BYTES, in.u);
      if (step(in) && in.run < runs) weights_of(in);
    }
    cp_async_commit();
  }
  if (a.dependent && !wait_first) pdl_wait();

  // ---------------------------------------------------------------- products
  FtWalk at = begin;
  int slot_in = ahead, slot_at = 0;
  constexpr bool XREG = NT <= 2;  // token rows held one unit ahead
  uint4 x[NT][2];
  if (at.run < runs) {
    tokens_of(at);
    if (XREG)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) load_x(x[nt], nt, at.u);
  }
  float acc[RT][NT][4];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][nt][c] = 0.0f;
  };
  clear();
  // the partial tile of the piece just finished: its own place in shared
  // memory, or added to the warp's weighted sums per token
  auto flush = [&](int run, int piece) {
    if (combine) {
      int tile, expert, first, count;
      piece_at(run, piece, tile, expert, first, count);
      float* y = red + warp * a.M * 16 * RT;
      __syncwarp();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int m = nt * 8 + 2 * t + c;
          if (m < count) {
            const float w = l.w[first + m];
            float* yt = y + (l.at[first + m] / a.topk) * 16 * RT + g;
#pragma unroll
            for (int i = 0; i < RT; ++i) {
              yt[16 * i] += w * acc[i][nt][c];
              yt[16 * i + 8] += w * acc[i][nt][c + 2];
            }
          }
        }
    } else {
      float4* p = reinterpret_cast<float4*>(red + (size_t)(piece + warp) * (U::PART / 4)) + lane;
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          p[(i * NT + nt) * 32] =
              make_float4(acc[i][nt][0], acc[i][nt][1], acc[i][nt][2], acc[i][nt][3]);
    }
    clear();
  };
  auto multiply = [&](uint32_t slot, const uint4 (&x)[NT][2]) {
    const uint32_t d = slot + lane * 16;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      uint32_t A[4][4];
      if (W4) {
        const uint4 c = lds128(d + U::W + i * 512);
        const uint32_t sc0 = lds32(slot + U::S + i * U::GROUPS * 128 + lane * 4);
        const uint32_t sc1 = G32 ? lds32(slot + U::S + (i * 2 + 1) * 128 + lane * 4) : sc0;
        uint32_t z0l = P::MAGIC + 0x00080008u, z0h = z0l, z1l = z0l, z1h = z0l;
        if (ZP) {
          const int sh = (g & 1) * 16;
          const uint32_t q0 = lds32(slot + U::Z + i * U::GROUPS * 128 + lane * 4) >> sh;
          z0l = P::MAGIC + (q0 & 0xffu) * 0x10001u;
          z0h = P::MAGIC + ((q0 >> 8) & 0xffu) * 0x10001u;
          z1l = z0l;
          z1h = z0h;
          if (G32) {
            const uint32_t q1 = lds32(slot + U::Z + (i * 2 + 1) * 128 + lane * 4) >> sh;
            z1l = P::MAGIC + (q1 & 0xffu) * 0x10001u;
            z1h = P::MAGIC + ((q1 >> 8) & 0xffu) * 0x10001u;
          }
        }
        ft_codes<BF16>(c.x, c.y, z0l, z0h, A[0]);
        ft_codes<BF16>(c.x >> 8, c.y >> 8, z0l, z0h, A[1]);
        ft_codes<BF16>(c.z, c.w, z1l, z1h, A[2]);
        ft_codes<BF16>(c.z >> 8, c.w >> 8, z1l, z1h, A[3]);
        const float s0g = P::lo(sc0), s0h = P::hi(sc0);
        const float s1g = G32 ? P::lo(sc1) : s0g, s1h = G32 ? P::hi(sc1) : s0h;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float p0[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          mma_16816<BF16>(p0, A[0][0], A[0][1], A[0][2], A[0][3], x[nt][0].x, x[nt][0].y);
          mma_16816<BF16>(p0, A[1][0], A[1][1], A[1][2], A[1][3], x[nt][0].z, x[nt][0].w);
          float(&o)[4] = acc[i][nt];
          if (G32) {
            o[0] = fmaf(s0g, p0[0], o[0]);
            o[1] = fmaf(s0g, p0[1], o[1]);
            o[2] = fmaf(s0h, p0[2], o[2]);
            o[3] = fmaf(s0h, p0[3], o[3]);
            p0[0] = p0[1] = p0[2] = p0[3] = 0.0f;
          }
          mma_16816<BF16>(p0, A[2][0], A[2][1], A[2][2], A[2][3], x[nt][1].x, x[nt][1].y);
          mma_16816<BF16>(p0, A[3][0], A[3][1], A[3][2], A[3][3], x[nt][1].z, x[nt][1].w);
          o[0] = fmaf(s1g, p0[0], o[0]);
          o[1] = fmaf(s1g, p0[1], o[1]);
          o[2] = fmaf(s1h, p0[2], o[2]);
          o[3] = fmaf(s1h, p0[3], o[3]);
        }
      } else {
        const uint4 g0 = lds128(d + U::W + i * 2048), g1 = lds128(d + U::W + i * 2048 + 512);
        const uint4 h0 = lds128(d + U::W + i * 2048 + 1024), h1 = lds128(d + U::W + i * 2048 + 1536);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_16816<BF16>(acc[i][nt], g0.x, h0.x, g0.y, h0.y, x[nt][0].x, x[nt][0].y);
          mma_16816<BF16>(acc[i][nt], g0.z, h0.z, g0.w, h0.w, x[nt][0].z, x[nt][0].w);
          mma_16816<BF16>(acc[i][nt], g1.x, h1.x, g1.y, h1.y, x[nt][1].x, x[nt][1].y);
          mma_16816<BF16>(acc[i][nt], g1.z, h1.z, g1.w, h1.w, x[nt][1].z, x[nt][1].w);
        }
      }
    }
  };

  uint16_t* const out = static_cast<uint16_t*>(a.out);
  for (int run = 0; run < runs; ++run) {
    while (at.run == run) {
      cp_async_wait(ahead - 1);
      if (in.run < runs) {
        copy_w(ring + slot_in * U::BYTES, in.u);
        if (step(in) && in.run < runs) weights_of(in);
      }
      cp_async_commit();
      if (++slot_in == a.depth) slot_in = 0;
      const uint32_t slot = ring + slot_at * U::BYTES;
      if (++slot_at == a.depth) slot_at = 0;
      if (!XREG)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) load_x(x[nt], nt, at.u);
      const int piece = at.piece;
      const bool last = step(at);  // of this piece
      if (last && at.run < runs) tokens_of(at);
      if (XREG) {
        uint4 xn[NT][2];
        if (at.run < runs)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) load_x(xn[nt], nt, at.u);
        multiply(slot, x);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          x[nt][0] = xn[nt][0];
          x[nt][1] = xn[nt][1];
        }
      } else {
        multiply(slot, x);
      }
      if (last) flush(run, piece);
    }
    __syncthreads();
    if (combine) {
      // the warps' weighted sums, in warp order
      const int tile = item0 + run;
      for (int i = threadIdx.x; i < a.M * 16 * RT; i += FT_THREADS) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < FT_WARPS; ++w) {
          v += red[w * a.M * 16 * RT + i];
          red[w * a.M * 16 * RT + i] = 0.0f;
        }
        const int m = i / (16 * RT), r = tile * 16 * RT + i % (16 * RT);
        if (r < a.rows) {
          uint16_t* o = out + (int64_t)m * a.rows + r;
          if (SWIGLU_CHECK_PTR(a.dbg, o, 2, a.err)) *o = P::rnd(a.scale * v);
        }
      }
    } else {
      // a tile's partials, in warp order: the warps whose shares meet it
      const int n = pieces_of(run);
      const int64_t total = (int64_t)n * nk;
      const bool gu = a.mode == FT_GATE_UP;
      const int per = (gu ? 8 : 16) * RT;  // outputs of a tile and token
      const int each = per * U::TOKENS;
      for (int i = threadIdx.x; i < n * each; i += FT_THREADS) {
        const int j = i / each, m = (i - j * each) / per, r = i % per;
        int tile, expert, first, count;
        piece_at(run, j, tile, expert, first, count);
        if (m >= count) continue;
        // row r of the tile: 16-row part r / 16 (gate/up: r / 8), row g or g + 8 of it
        const int part = gu ? r >> 3 : r >> 4, rg = r & 7, half = gu ? 0 : (r >> 3) & 1;
        const int at0 = (part * NT + (m >> 3)) * 128 + (rg * 4 + ((m & 7) >> 1)) * 4 + (m & 1) + 2 * half;
        // shares: warp w has [total w / 16, total (w + 1) / 16)
        int w = (int)(((int64_t)j * nk * FT_WARPS) / total);
        while (w + 1 < FT_WARPS && total * (w + 1) / FT_WARPS <= (int64_t)j * nk) ++w;
        float v = 0.0f, v2 = 0.0f;
        for (; w < FT_WARPS && total * w / FT_WARPS < (int64_t)(j + 1) * nk; ++w) {
          if (total * w / FT_WARPS == total * (w + 1) / FT_WARPS) continue;  // an empty share
          const float* p = red + (size_t)(j + w) * (U::PART / 4) + at0;
          v += p[0];
          if (gu) v2 += p[2];
        }
        const int col = tile * per + r;
        if (col >= a.rows) continue;
        uint16_t* o = out + (int64_t)(first + m) * a.rows + col;
        v = gu ? ft_silu(a.scale * v) * v2 : a.scale * v;
        if (SWIGLU_CHECK_PTR(a.dbg, o, 2, a.err)) *o = P::rnd(v);
      }
    }
    __syncthreads();
  }
}

}  // namespace swiglu
