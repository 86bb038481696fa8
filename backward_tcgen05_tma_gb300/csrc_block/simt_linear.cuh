// simt_linear.cuh -- fp32 products with IEEE fp32 FMA on the CUDA cores (never
// TF32), with the linear operators' epilogues:
//
//   C[m, n] = sum_k A(m, k) B(n, k)
//
// Bound by the FMA pipe: 152 SMs x 128 lanes x 2 flops at 1.9 GHz are 74 TFLOP/s.
// Blocks of 256 threads compute 16 TM x 128 tiles, TM x 8 a thread (TM = 8; 2 for
// up to 32 rows), over k in steps of 16 through two shared-memory buffers that
// hold both operands with k outermost.  Two columns share one fma.rn.f32x2, each
// half rounded as an fma of its own, which halves the instructions to issue.  Two
// blocks fit an SM.  The tiles of a last round that would leave many of those
// places empty are split over the contraction, and a second kernel adds the parts
// in order and applies the epilogue.  1999 x 2824 x 1032 (368 tiles of 128 x 128,
// 64 of them split): 272 us, 43 TFLOP/s, 58% of the FMA pipe; 324 with all tiles
// whole, 577 with tiles of 64 x 64.
//
// An operand comes with k contiguous (KC: rows of it are turned on the way to
// shared memory) or with its own index contiguous.
#pragma once

#include "../csrc/simt_gemm.cuh"
#include "act.cuh"
#include "simt_plan.h"

namespace swiglu {

constexpr int SL_THREADS = 256;

struct SlArgs {
  const float* A;
  const float* B;
  int64_t lda, ldb;  // elements between rows of k (KC), or between k
  int M, N, K;
  int m_tiles, n_tiles;
  int whole;         // tiles [0, whole) are taken whole, the others in parts
  int parts;
  int per;           // k of a part, a multiple of SL_BK
  float* part;       // [(tiles - whole) * parts][tile]
  int* clear;        // the error word, cleared by the first kernel of a call, or null
  SimtCheck chk;
};

__device__ __forceinline__ float4 sl_load4(const float* p, const SimtCheck& chk) {
  return SWIGLU_CHECK_PTR(chk.win, p, 16, chk.err) ? *reinterpret_cast<const float4*>(p)
                                                   : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
}
__device__ __forceinline__ void sl_store4(float* p, const float (&v)[4], const SimtCheck& chk) {
  if (SWIGLU_CHECK_PTR(chk.win, p, 16, chk.err))
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// Y = act(acc + bias) + res, Z = acc + bias; four columns at a time
struct SlEpiLinear {
  const float* bias;
  const float* res;
  float* z;
  float* y;
  int64_t ld;
  int act;
  __device__ __forceinline__ void apply(int m, int n, float (&v)[4], const SimtCheck& chk) const {
    const int64_t o = (int64_t)m * ld + n;
    if (bias != nullptr) {
      const float4 b = sl_load4(bias + n, chk);
      v[0] += b.x;
      v[1] += b.y;
      v[2] += b.z;
      v[3] += b.w;
    }
    if (z != nullptr) sl_store4(z + o, v, chk);
    act_switch(act, [&](auto a) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = ActPrecise::value<decltype(a)::value>(v[i]);
    });
    if (res != nullptr) {
      const float4 r = sl_load4(res + o, chk);
      v[0] = __fadd_rn(v[0], r.x);
      v[1] = __fadd_rn(v[1], r.y);
      v[2] = __fadd_rn(v[2], r.z);
      v[3] = __fadd_rn(v[3], r.w);
    }
    sl_store4(y + o, v, chk);
  }
};

// out = acc act'(pre) (pre null: acc), or with `add` out + acc
struct SlEpiGrad {
  const float* pre;
  float* out;
  int64_t ld;
  int act;
  int add;
  __device__ __forceinline__ void apply(int m, int n, float (&v)[4], const SimtCheck& chk) const {
    const int64_t o = (int64_t)m * ld + n;
    if (pre != nullptr) {
      const float4 z4 = sl_load4(pre + o, chk);
      const float z[4] = {z4.x, z4.y, z4.z, z4.w};
      act_switch(act, [&](auto a) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __fmul_rn(v[i], ActPrecise::slope<decltype(a)::value>(z[i]));
      });
    }
    if (add) {
      const float4 h = sl_load4(out + o, chk);
      v[0] = __fadd_rn(v[0], h.x);
      v[1] = __fadd_rn(v[1], h.y);
      v[2] = __fadd_rn(v[2], h.z);
      v[3] = __fadd_rn(v[3], h.w);
    }
    sl_store4(out + o, v, chk);
  }
};

__device__ __forceinline__ uint64_t sl_pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void sl_fma2(uint64_t& c, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a), "l"(b));
}

// One operand's ROWS x 16 tile: fetched to registers, then put as [k][row].
template <int ROWS, bool KC>
struct SlTile {
  static constexpr int LD = ROWS + 4;                    // floats of a k row in shared memory
  static constexpr int QUADS = ROWS * SL_BK / 4;         // 16-byte pieces
  static constexpr int EACH = (QUADS + SL_THREADS - 1) / SL_THREADS;
  float4 v[EACH];
  __device__ __forceinline__ void fetch(const float* p, int64_t ld, int r0, int rows, int k0, int k1,
                                        const SimtCheck& chk) {
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int q = threadIdx.x + i * SL_THREADS;
      const int r = r0 + (KC ? q / (SL_BK / 4) : q % (ROWS / 4) * 4);
      const int k = k0 + (KC ? q % (SL_BK / 4) * 4 : q / (ROWS / 4));
      const float* at = p + (KC ? (int64_t)r * ld + k : (int64_t)k * ld + r);
      bool in = q < QUADS && r < rows && k < k1;
      in = in && SWIGLU_CHECK_PTR(chk.win, at, 16, chk.err);
      // predicated and in its place: a k-tile's arithmetic ahead of its use
      v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      asm volatile(
          "{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %5, 0;\n\t"
          "@p ld.global.v4.f32 {%0, %1, %2, %3}, [%4];\n\t}"
          : "+f"(v[i].x), "+f"(v[i].y), "+f"(v[i].z), "+f"(v[i].w)
          : "l"(at), "r"((int)in));
    }
  }
  __device__ __forceinline__ void put(float* s) const {
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int q = threadIdx.x + i * SL_THREADS;
      if (QUADS % SL_THREADS != 0 && q >= QUADS) break;
      if constexpr (KC) {
        const int r = q / (SL_BK / 4), k = q % (SL_BK / 4) * 4;
        s[k * LD + r] = v[i].x;
        s[(k + 1) * LD + r] = v[i].y;
        s[(k + 2) * LD + r] = v[i].z;
        s[(k + 3) * LD + r] = v[i].w;
      } else {
        *reinterpret_cast<float4*>(s + q / (ROWS / 4) * LD + q % (ROWS / 4) * 4) = v[i];
      }
    }
  }
};

// Tiles go down columns of up to 16 tile rows, so that the blocks that run at one
// time share few columns of B.
__device__ __forceinline__ void sl_tile(const SlArgs& a, int tile, int bm, int& m0, int& n0) {
  const int per_group = 16 * a.n_tiles, grp = tile / per_group, left = tile - grp * per_group;
  const int gh = min(16, a.m_tiles - grp * 16);
  m0 = (grp * 16 + left % gh) * bm;
  n0 = left / gh * SL_BN;
}

template <int TM, bool A_KC, bool B_KC, class Epi>
__global__ void __launch_bounds__(SL_THREADS, 2) simt_linear_kernel(const SlArgs a, const Epi epi) {
  constexpr int BM = 16 * TM;
  using TA = SlTile<BM, A_KC>;
  using TB = SlTile<SL_BN, B_KC>;
  __shared__ __align__(16) float As[2][SL_BK * TA::LD];
  __shared__ __align__(16) float Bs[2][SL_BK * TB::LD];
  if (a.clear != nullptr && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.clear = 0;
  const int split = (int)blockIdx.x - a.whole;  // >= 0: a part of a split tile
  int m0, n0;
  sl_tile(a, split < 0 ? (int)blockIdx.x : a.whole + split / a.parts, BM, m0, n0);
  const int k0 = split < 0 ? 0 : split % a.parts * a.per, k1 = split < 0 ? a.K : min(a.K, k0 + a.per);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  constexpr int AV = TM < 4 ? TM : 4;  // rows of a thread that follow one another
  uint64_t acc[TM][4];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0;
  TA ta;
  TB tb;
  ta.fetch(a.A, a.lda, m0, a.M, k0, k1, a.chk);
  tb.fetch(a.B, a.ldb, n0, a.N, k0, k1, a.chk);
  ta.put(As[0]);
  tb.put(Bs[0]);
  __syncthreads();
  int buf = 0;
  for (int k = k0; k < k1; k += SL_BK) {
    const bool more = k + SL_BK < k1;
    if (more) {
      ta.fetch(a.A, a.lda, m0, a.M, k + SL_BK, k1, a.chk);
      tb.fetch(a.B, a.ldb, n0, a.N, k + SL_BK, k1, a.chk);
    }
#pragma unroll
    for (int kk = 0; kk < SL_BK; ++kk) {
      float av[TM];
      uint64_t bv[4];
      const float* sa = As[buf] + kk * TA::LD + ty * AV;
      const float* sb = Bs[buf] + kk * TB::LD + tx * 4;
#pragma unroll
      for (int i = 0; i < TM; i += AV) {
        if constexpr (AV == 4) {
          const float4 q = *reinterpret_cast<const float4*>(sa + i * 16);
          av[i] = q.x;
          av[i + 1] = q.y;
          av[i + 2] = q.z;
          av[i + 3] = q.w;
        } else {
          const float2 q = *reinterpret_cast<const float2*>(sa);
          av[0] = q.x;
          av[1] = q.y;
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(sb + j * 64);
        bv[2 * j] = q.x;
        bv[2 * j + 1] = q.y;
      }
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const uint64_t aa = sl_pair(av[i], av[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) sl_fma2(acc[i][j], aa, bv[j]);
      }
    }
    if (more) {
      ta.put(As[buf ^ 1]);
      tb.put(Bs[buf ^ 1]);
    }
    __syncthreads();
    buf ^= 1;
  }
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int mt = (i / AV) * 16 * AV + ty * AV + i % AV, m = m0 + mt;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int n = n0 + j * 64 + tx * 4;
      float v[4];
      asm("mov.b64 {%0, %1}, %2;" : "=f"(v[0]), "=f"(v[1]) : "l"(acc[i][2 * j]));
      asm("mov.b64 {%0, %1}, %2;" : "=f"(v[2]), "=f"(v[3]) : "l"(acc[i][2 * j + 1]));
      if (split >= 0)
        sl_store4(a.part + (int64_t)split * (BM * SL_BN) + mt * SL_BN + (n - n0), v, a.chk);
      else if (m < a.M && n < a.N)
        epi.apply(m, n, v, a.chk);
    }
  }
}

// Up to 8 rows of X (ROWS >= M of them, R rows of W a block): the weights' bytes are
// the bound.  A block's 8 warps split k; lanes read 16 bytes of each row, coalesced,
// X from the caches; sums meet over the lanes, then over the warps in order.
// 4096 x 4096, one row, weights in the L2: 52 us in tiles of 32 rows, 6.6 so.
template <int ROWS, class Epi>
__global__ void __launch_bounds__(SL_THREADS) simt_rows_kernel(const SlArgs a, const Epi epi) {
  constexpr int R = ROWS == 8 ? 4 : 8, WARPS = SL_THREADS / 32;
  static_assert(R % 4 == 0, "the epilogue takes four columns");
  __shared__ float sums[WARPS][ROWS][R];
  if (a.clear != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *a.clear = 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * R;
  const int quads = a.K / 4, q0 = (int)((int64_t)quads * warp / WARPS), q1 = (int)((int64_t)quads * (warp + 1) / WARPS);
  float acc[ROWS][R];
#pragma unroll
  for (int m = 0; m < ROWS; ++m)
#pragma unroll
    for (int r = 0; r < R; ++r) acc[m][r] = 0.0f;
#pragma unroll 2
  for (int q = q0 + lane; q < q1; q += 32) {
    float4 w[R], x[ROWS];
#pragma unroll
    for (int r = 0; r < R; ++r)  // (rows past N repeat the last)
      w[r] = sl_load4(a.B + (int64_t)min(n0 + r, a.N - 1) * a.ldb + q * 4, a.chk);
#pragma unroll
    for (int m = 0; m < ROWS; ++m) x[m] = sl_load4(a.A + (int64_t)min(m, a.M - 1) * a.lda + q * 4, a.chk);
#pragma unroll
    for (int m = 0; m < ROWS; ++m)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float v = acc[m][r];
        v = fmaf(x[m].x, w[r].x, v);
        v = fmaf(x[m].y, w[r].y, v);
        v = fmaf(x[m].z, w[r].z, v);
        acc[m][r] = fmaf(x[m].w, w[r].w, v);
      }
  }
#pragma unroll
  for (int m = 0; m < ROWS; ++m)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float v = acc[m][r];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0) sums[warp][m][r] = v;
    }
  __syncthreads();
  const int m = threadIdx.x / (R / 4), c = threadIdx.x % (R / 4) * 4;
  if (m >= ROWS || m >= a.M || n0 + c >= a.N) return;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int w = 0; w < WARPS; ++w)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += sums[w][m][c + i];
  epi.apply(m, n0 + c, v, a.chk);
}

template <int TM, class Epi>
__global__ void __launch_bounds__(256) simt_sum_kernel(const SlArgs a, const Epi epi) {
  constexpr int BM = 16 * TM, QUADS = BM * SL_BN / 4;
  const int t = blockIdx.x;
  int m0, n0;
  sl_tile(a, a.whole + t, BM, m0, n0);
  const int q = blockIdx.y * 256 + threadIdx.x, m = m0 + q / (SL_BN / 4), n = n0 + q % (SL_BN / 4) * 4;
  if (q >= QUADS || m >= a.M || n >= a.N) return;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int p = 0; p < a.parts; ++p) {
    const float4 w = sl_load4(a.part + ((int64_t)t * a.parts + p) * (BM * SL_BN) + q * 4, a.chk);
    v[0] += w.x;
    v[1] += w.y;
    v[2] += w.z;
    v[3] += w.w;
  }
  epi.apply(m, n, v, a.chk);
}

}  // namespace swiglu
