// fewtok.cuh -- what the kernels for a few tokens share: arguments of the
// mixture-of-experts kernels, 16-bit arithmetic, and the experts' token lists.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../csrc/sm103_ptx.cuh"
#include "experts_plan.h"

namespace swiglu {

constexpr int FT_MAX_TOKENS = 64;
constexpr int FT_MAX_EXPERTS = 512;
constexpr int FT_MAX_TOPK = 16;

enum FtMode : int { FT_GATE_UP = 1, FT_COMBINE = 2 };

struct FtArgs {
  int mode;          // FT_GATE_UP: out = rnd(SiLU(scale g) u), a row per assignment;
                     //   FT_COMBINE: out[t] = rnd(scale sum_j w[t, j] v_j) over a token's experts
  int M;             // tokens
  int K;             // contraction, a multiple of 8
  int rows;          // rows of out: hidden units (gate/up) or output features
  int tiles;         // 16-row tiles of one expert's matrix (gate/up: 8 rows of each of two)
  const uint8_t* W;  // packed 4-bit matrices (16-bit ones come by the tensor map)
  int64_t expert_bytes;
  const void* X;     // [*, K]: token rows, or (FT_COMBINE) one row per assignment
  void* out;
  float scale;
  int E, topk;
  const int* idx;    // [M, topk] experts (values outside 0..E-1: none)
  const float* wts;  // [M, topk]
  int first;         // first kernel of a call
  int idx_ready;     // idx was complete before the kernel before this one began
  int inject;        // test hook: no warp's first stage is ever filled
  // shared-memory plan: chunks a warp's ring holds, items of a run, offsets
  int stages, run;
  int list_off, red_off, ring_off;
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
  static __device__ __forceinline__ float lo(uint32_t v) { return __uint_as_float(v << 16); }
  static __device__ __forceinline__ float hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
  static __device__ __forceinline__ uint16_t rnd(float v) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }
};
template <>
struct Ft16<false> {
  static constexpr uint32_t MAGIC = 0x64006400u;  // 1024, 1024
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

// (v & mask) | bits in one instruction
template <uint32_t MASK>
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "n"(MASK), "r"(bits));
  return r;
}

// a - b of both halves
template <bool BF16>
__device__ __forceinline__ uint32_t ft_sub2(uint32_t a, uint32_t b) {
  uint32_t r;
  if (BF16)
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Codes to numbers.  OR-ed into the mantissa of 128 (bf16) or 1024 (fp16) a
// code is a 16-bit number, 128 + q or 1024 + q; the fp16 codes in bits 4..7 can
// stay there, as 1024 + 16 q.  Taking 128 + z or 1024 + z off (the second fp16
// form: multiplied by 1/16 it is 64 + q, and 64 + z goes off in the same
// instruction) leaves the whole number q - z, exactly: every operand and result
// is a whole number that the type holds.
template <bool BF16>
struct W4Off {
  uint32_t a, b;  // 128 + z or 1024 + z, for both halves; fp16: -(64 + z)
  __device__ __forceinline__ explicit W4Off(uint32_t z = 8) {
    a = Ft16<BF16>::MAGIC | z * 0x10001u;
    b = 0xd400d400u | z * 0x100010u;
  }
};
// two elements of each form: the codes in bits 0..3 of v's halves, and those in
// bits 4..7
template <bool BF16>
__device__ __forceinline__ uint32_t w4_first(uint32_t v, const W4Off<BF16>& z) {
  return ft_sub2<BF16>(and_or<0x000f000fu>(v, Ft16<BF16>::MAGIC), z.a);
}
template <bool BF16>
__device__ __forceinline__ uint32_t w4_second(uint32_t v, const W4Off<BF16>& z) {
  if (BF16) return w4_first<BF16>(v >> 4, z);
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;"
      : "=r"(r)
      : "r"(and_or<0x00f000f0u>(v, Ft16<BF16>::MAGIC)), "r"(0x2c002c00u), "r"(z.b));
  return r;
}

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

__device__ __forceinline__ float ft_silu(float g) { return g / (1.0f + __expf(-g)); }

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ float lds32f(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts32(uint32_t a, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}

// 16 bytes through the L1 cache.  Not the read-only path, which asks for data
// that nothing writes while the kernel runs: token rows and router weights may
// be written while its prologue does (before griddepcontrol.wait).
__device__ __forceinline__ uint4 ft_load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
// ---- thread-block clusters
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_store(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

__device__ __forceinline__ float4 cluster_load4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Every launch is a programmatic dependent of the one before it, so that its
// blocks are in place when that one ends.  The first kernel of a call touches
// nothing before then; nor does gate/up after the router, which writes idx.
// Only then may the next kernel start: so the combining kernel, whose idx was
// complete before gate/up went past this point, needs to wait for gate/up only
// before it reads the hidden values, and reads weights at once.
__device__ __forceinline__ bool ft_waits_first(const FtArgs& a) { return a.first || !a.idx_ready; }
__device__ __forceinline__ void ft_begin(const FtArgs& a) {
  if (ft_waits_first(a)) pdl_wait();
  if (a.first && blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;
  pdl_launch_dependents();
}

// The experts' token lists of a call, built by every block for itself in
// shared memory: the valid assignments sorted by (expert, token), and one
// entry per run of at most `per` assignments of one expert.  An expert named
// twice by one token counts once, with the sum of its weights.
struct FtLists {
  unsigned long long* mask;  // [E] tokens of an expert
  int2* entry;               // {expert | count << 16, first position}
  int* start;                // [E] first position of an expert
  int* e;                    // [M * topk] an assignment's expert, as given
  float* we;                 // [M * topk] its weight, as given
  float* w;                  // [M * topk] weight, by position
  uint16_t* at;              // [M * topk] assignment, by position
  int* n;                    // entries
};
__device__ __forceinline__ FtLists ft_lists(uint8_t* p, const FtArgs& a, int per) {
  FtLists l;
  l.n = reinterpret_cast<int*>(p);
  l.mask = reinterpret_cast<unsigned long long*>(p + 16);
  l.entry = reinterpret_cast<int2*>(l.mask + a.E);
  l.start = reinterpret_cast<int*>(l.entry + ft_max_entries(a.M, a.topk, a.E, per));
  l.e = l.start + a.E;
  l.we = reinterpret_cast<float*>(l.e + a.M * a.topk);
  l.w = l.we + a.M * a.topk;
  l.at = reinterpret_cast<uint16_t*>(l.w + a.M * a.topk);
  return l;
}

// Assignment i's expert, or -1 where it is none or an earlier one of the same
// token names the same expert.
__device__ __forceinline__ int ft_assignment(const FtArgs& a, const FtLists& l, int i, int t) {
  const int e = l.e[i];
  if (e < 0 || e >= a.E) return -1;
  for (int q = t * a.topk; q < i; ++q)
    if (l.e[q] == e) return -1;
  return e;
}

// The same for up to 8 tokens and 32 assignments, one a lane of the first warp:
// no passes over shared memory, one barrier (measured: 1.3 us sooner at one
// token and 8 of 64 experts).
__device__ __forceinline__ void ft_build_lists_warp(const FtArgs& a, const FtLists& l) {
  const int total = a.M * a.topk;
  if (threadIdx.x < 32) {
    const int i = threadIdx.x;
    int e = -1;
    float w = 0.0f;
    if (i < total) {
      if (SWIGLU_CHECK_PTR(a.dbg, a.idx + i, 4, a.err)) e = __ldcg(a.idx + i);
      if (a.mode == FT_COMBINE && SWIGLU_CHECK_PTR(a.dbg, a.wts + i, 4, a.err)) w = __ldcg(a.wts + i);
      if (e >= a.E) e = -1;
    }
    const uint32_t named = __ballot_sync(0xffffffffu, e >= 0);
    const uint32_t same = __match_any_sync(0xffffffffu, e) & named;  // lanes with this expert
    const int t = (int)((unsigned)i / (unsigned)a.topk);
    const uint32_t before = (1u << i) - 1, row0 = (1u << (t * a.topk & 31)) - 1;
    const uint32_t row = e >= 0 ? same & ~row0 : 0;  // ... of this token or a later one
    const bool valid = e >= 0 && (row & before) == 0;
    const uint32_t valids = __ballot_sync(0xffffffffu, valid);
    if (a.mode == FT_COMBINE && valids != named) {  // an expert named twice: the sum of its weights
      float sum = 0.0f;
      for (int q = 0; q < total; ++q) {
        const float wq = __shfl_sync(0xffffffffu, w, q);
        if ((row >> q & 1u) && (int)((unsigned)q / (unsigned)a.topk) == t) sum += wq;
      }
      w = sum;
    }
    const bool leads = valid && (same & valids & before) == 0;  // first assignment of its expert
    const uint32_t leaders = __ballot_sync(0xffffffffu, leads);
    int lower = 0, entry = 0;  // assignments of lower experts, and those experts
    for (uint32_t m = valids; m != 0; m &= m - 1) {
      const int q = __ffs(m) - 1;
      const bool less = __shfl_sync(0xffffffffu, e, q) < e;
      lower += less;
      entry += less && (leaders >> q & 1u);
    }
    if (valid) {
      const int p = lower + __popc(same & valids & before);
      l.at[p] = (uint16_t)i;
      l.w[p] = w;
      if (leads) l.entry[entry] = make_int2(e | __popc(same & valids) << 16, lower);
    }
    if (i == 0) *l.n = __popc(leaders);
  }
  __syncthreads();
}

template <int THREADS>
__device__ __forceinline__ void ft_build_lists(const FtArgs& a, const FtLists& l, int per) {
  const int total = a.M * a.topk;
  const bool weights = a.mode == FT_COMBINE;
  if (a.M <= 8 && total <= 32) return ft_build_lists_warp(a, l);
  for (int i = threadIdx.x; i < total; i += THREADS) {
    l.e[i] = SWIGLU_CHECK_PTR(a.dbg, a.idx + i, 4, a.err) ? __ldcg(a.idx + i) : -1;
    if (weights) l.we[i] = SWIGLU_CHECK_PTR(a.dbg, a.wts + i, 4, a.err) ? __ldcg(a.wts + i) : 0.0f;
  }
  for (int e = threadIdx.x; e < a.E; e += THREADS) l.mask[e] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < total; i += THREADS) {
    const int t = i / a.topk, e = ft_assignment(a, l, i, t);
    if (e >= 0) atomicOr(l.mask + e, 1ull << t);
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    int pos = 0, ent = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + threadIdx.x;
      const int n = e < a.E ? __popcll(l.mask[e]) : 0, c = (n + per - 1) / per;
      int sum = n | c << 16;  // inclusive sums over the 32 experts
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, d);
        if ((int)threadIdx.x >= d) sum += up;
      }
      const int p0 = pos + (sum & 0xffff) - n, c0 = ent + (sum >> 16) - c;
      if (e < a.E) l.start[e] = p0;
      for (int q = 0; q < c; ++q)
        l.entry[c0 + q] = make_int2(e | min(per, n - q * per) << 16, p0 + q * per);
      const int all = __shfl_sync(0xffffffffu, sum, 31);
      pos += all & 0xffff;
      ent += all >> 16;
    }
    if (threadIdx.x == 0) *l.n = ent;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < total; i += THREADS) {
    const int t = i / a.topk, e = ft_assignment(a, l, i, t);
    if (e < 0) continue;
    const int p = l.start[e] + __popcll(l.mask[e] & ((1ull << t) - 1));
    l.at[p] = (uint16_t)i;
    if (weights) {
      float w = l.we[i];
      for (int q = i + 1; q < (t + 1) * a.topk; ++q)
        if (l.e[q] == e) w += l.we[q];
      l.w[p] = w;
    }
  }
  __syncthreads();
}

}  // namespace swiglu
