// linear_few.cuh -- Y [M, N] = act(X W^T + bias) + residual for up to 16 tokens
// and 16-bit weights, bound by streaming W from HBM.
//
// mma.sync with W's rows as its M (16 rows a warp at a time) and the tokens as
// its N (NT columns of 8).  The contraction is split into `parts`, one a warp,
// over the blocks of a cluster and over `halves` within a block.  A block keeps
// its parts of the token rows in shared memory and works on all rows of W that
// its cluster takes, so token rows are fetched once per cluster and not with
// every tile of weights.  The warps that work on the same 16 rows send their
// sums, 8 tokens at a time, to one of them (st.async, which carries the data and
// counts it on the receiver's barrier); it adds them in the order of the parts
// and applies the epilogue.
//
// Weights go from global memory to the fragments' registers: the order of k
// within 32 is free as long as both operands share it, so lane (g, t) takes the
// 16 bytes of row g at k = 8 t, which serve two k steps of the instruction.  Two
// chunks of 4 x 32 k take turns, one on its way while the other is used, across
// items.  (A third one meant code for three orders of them, which the compiler
// folded into moves of registers and waits for what they hold.)
//
// Measured, back to back: 2816 x 1024 one token 5.0 us, 2056 x 5640 thirteen 7.5
// (3.1 TB/s), 11008 x 4096 one 20.5 (4.4 TB/s).  At more tokens the products'
// instructions and their latencies bound it.
//
// Each warp's receive buffers are two: what a source sends for a use of one of
// them it sends after it was itself sent to, in between, by a warp that had done
// with the use before last (ownership goes round the parts evenly).
#pragma once

#include "../csrc_serving/fewtok.cuh"
#include "act.cuh"

namespace swiglu {

constexpr int LF_THREADS = 256, LF_WARPS = LF_THREADS / 32;
constexpr int LF_BLOCKS = 4;      // 32-k blocks of a chunk
constexpr int LF_MAX_M = 16;
constexpr int LF_MAX_PARTS = 8;
constexpr int LF_SMEM = 226 * 1024;

struct LfArgs {
  const uint8_t* X;     // [M, K]
  const uint8_t* W;     // [N, K]
  const uint8_t* bias;  // [N] or null
  const uint8_t* res;   // [M, N] or null
  uint8_t* z;           // [M, N] or null
  uint8_t* y;           // [M, N]
  int M, N, K, act;
  int units;            // runs of 16 rows
  int blocks;           // of a cluster; 1 only with one part (st.async is for clusters)
  int halves;           // parts of a block; a power of two, like `blocks`
  int clusters;
  int xstride;          // bytes of a token row in shared memory
  int recv_off;         // receive buffers
  int inject;           // test hook: nothing is sent for the first item
  uint64_t wait_limit_ns;
  int* err;
#ifdef SWIGLU_DEBUG
  DbgWin dbg;           // y, workspace, z, residual, bias, X, W
#endif
};

// Bytes of a warp's receive buffer: a column of 8 tokens x 16 rows from each
// part, of each column that it may own.
__host__ __device__ constexpr int lf_recv(int nt, int parts) { return (nt > parts ? nt : parts) * 512; }

__device__ __forceinline__ void st_async16(uint32_t addr, uint32_t bar, const float (&v)[4]) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%2, %3, %4, %5}, [%1];" ::"r"(addr),
      "r"(bar), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3])
      : "memory");
}

__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

template <bool BF16>
__device__ __forceinline__ float lf_get(const uint8_t* p) {
  const uint16_t v = *reinterpret_cast<const uint16_t*>(p);
  return Ft16<BF16>::lo(v);
}

template <bool BF16, int NT>
__global__ void __launch_bounds__(LF_THREADS, 1) linear_few_kernel(const LfArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint64_t bars[LF_WARPS][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rank = a.blocks > 1 ? (int)cluster_rank() : 0;
  const int parts = a.blocks * a.halves, part = rank * a.halves + warp % a.halves;
  const int plog = __ffs(parts) - 1, hlog = __ffs(a.halves) - 1;
  const int cluster = (int)blockIdx.x / a.blocks;
  const uint32_t sbase = smem_u32(smem);

  if (lane == 0) {
    mbar_init(smem_u32(&bars[warp][0]), 1);
    mbar_init(smem_u32(&bars[warp][1]), 1);
    fence_mbar_init();
  }
  __syncwarp();
  if (a.blocks > 1) cluster_arrive();  // waited for before anything is sent
  pdl_wait();  // launched early: nothing is touched before the kernel before has ended
  pdl_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;

  // the 32-k blocks of this block and of this warp's part, and the warp's items (16 rows of W)
  const int nk = (a.K + 31) / 32;
  const int xb0 = (int)((int64_t)nk * rank / a.blocks), xn = (int)((int64_t)nk * (rank + 1) / a.blocks) - xb0;
  const int kb0 = xb0 + xn * (warp % a.halves) / a.halves;
  const int nkl = xb0 + xn * (warp % a.halves + 1) / a.halves - kb0;
  const int chunks = (nkl + 2 * LF_BLOCKS - 1) / (2 * LF_BLOCKS) * 2;  // in pairs: the last may be empty
  const int groups = LF_WARPS / a.halves;
  const int first = cluster * groups + warp / a.halves, stride = a.clusters * groups;
  const int items = first < a.units ? (a.units - first + stride - 1) / stride : 0;

  // Weights of the next chunk to be fetched: predicated loads, not branches, whose
  // ends would wait for what they loaded.  Rows past N repeat the last one (they
  // are never stored); what lies past the part or past K is not loaded.
  int lu = first, lc = 0;
  const uint8_t *lp = a.W, *lq = a.W;  // rows g and g + 8 of the item, at this lane's k
  auto load_item = [&]() {
    const int64_t k = (int64_t)kb0 * 32 + t * 8;
    lp = a.W + ((int64_t)min(lu * 16 + g, a.N - 1) * a.K + k) * 2;
    lq = a.W + ((int64_t)min(lu * 16 + 8 + g, a.N - 1) * a.K + k) * 2;
  };
  auto fetch = [&](uint4& w, const uint8_t* p, bool want) {
    if (!SWIGLU_CHECK(!want || dbg_in(a.dbg, p, 16), a.err)) want = false;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %5, 0;\n\t"
        "@p ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "+r"(w.x), "+r"(w.y), "+r"(w.z), "+r"(w.w)
        : "l"(p), "r"((int)want));
  };
  const int ragged = a.K & 31;  // of the last block, whole if 0
  // blocks of this part that this lane has all its 8 k of
  const int mine = ragged != 0 && kb0 + nkl == nk && t * 8 >= ragged ? nkl - 1 : nkl;
  auto load = [&](uint4 (&w)[2 * LF_BLOCKS]) {
    const int left = lu < a.units ? mine - lc * LF_BLOCKS : 0;
#pragma unroll
    for (int j = 0; j < LF_BLOCKS; ++j) {
      fetch(w[2 * j], lp + j * 64, j < left);
      fetch(w[2 * j + 1], lq + j * 64, j < left);
    }
    lp += LF_BLOCKS * 64;
    lq += LF_BLOCKS * 64;
    if (++lc == chunks) {
      lc = 0;
      lu += stride;
      load_item();
    }
  };
  uint4 w0[2 * LF_BLOCKS], w1[2 * LF_BLOCKS];
#pragma unroll
  for (int j = 0; j < 2 * LF_BLOCKS; ++j) w0[j] = w1[j] = make_uint4(0u, 0u, 0u, 0u);
  load_item();
  load(w0);
  load(w1);

  // this block's part of the token rows; past K zeros (0 times what lies there may not be 0)
  for (int i = threadIdx.x; i < a.M * xn * 4; i += LF_THREADS) {
    const int m = i / (xn * 4), v = i - m * (xn * 4), k = xb0 * 32 + v * 8;
    const uint32_t dst = sbase + m * a.xstride + v * 16;
    const uint8_t* src = a.X + ((int64_t)m * a.K + k) * 2;
    if (k < a.K && SWIGLU_CHECK_PTR(a.dbg, src, 16, a.err))
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
      asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst), "r"(0u) : "memory");
  }
  asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  if (a.blocks > 1) cluster_wait();  // every block's barriers are set

  uint32_t xa[NT];  // (columns past M repeat the last token; they are never stored)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) xa[nt] = sbase + min(nt * 8 + g, a.M - 1) * a.xstride + (kb0 - xb0) * 64 + t * 16;

  float acc[NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[nt][i] = 0.0f;

  // The epilogue of 16 rows x 8 tokens: v = (row g, tokens 2t, 2t + 1), (row g + 8, ...).
  auto finish = [&](int unit, int nt, float (&v)[4]) {
    const int m0 = nt * 8 + 2 * t, r0 = unit * 16 + g;
    float r[4], b[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = r0 + 8 * h;
      b[h] = a.bias != nullptr && row < a.N && SWIGLU_CHECK_PTR(a.dbg, a.bias + row * 2ll, 2, a.err)
                 ? lf_get<BF16>(a.bias + row * 2ll)
                 : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = m0 + (i & 1), row = r0 + 8 * (i >> 1);
      const int64_t o = ((int64_t)m * a.N + row) * 2;
      const bool in = m < a.M && row < a.N;
      r[i] = a.res != nullptr && in && SWIGLU_CHECK_PTR(a.dbg, a.res + o, 2, a.err) ? lf_get<BF16>(a.res + o) : 0.0f;
      v[i] += b[i >> 1];
      if (a.z != nullptr && in && SWIGLU_CHECK_PTR(a.dbg, a.z + o, 2, a.err))
        *reinterpret_cast<uint16_t*>(a.z + o) = Ft16<BF16>::rnd(v[i]);
    }
    act_switch(a.act, [&](auto f) {
      act_value2<decltype(f)::value>(v[0], v[1]);
      act_value2<decltype(f)::value>(v[2], v[3]);
    });
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = m0 + (i & 1), row = r0 + 8 * (i >> 1);
      const int64_t o = ((int64_t)m * a.N + row) * 2;
      if (m < a.M && row < a.N && SWIGLU_CHECK_PTR(a.dbg, a.y + o, 2, a.err))
        *reinterpret_cast<uint16_t*>(a.y + o) = Ft16<BF16>::rnd(v[i] + r[i]);
    }
  };

  const int recv = lf_recv(NT, parts);
  int uses = 0;       // of this warp's buffers
  bool live = true;   // no wait has run out
  auto flush = [&](int item) {
    const int unit = first + item * stride;
    // column nt of item i belongs to part (i NT + nt + group) mod parts: every
    // part is a receiver equally often, and all know how often each was
    const int rot = (item * NT + (warp >> hlog)) & (parts - 1);
    const bool quiet = a.inject && item == 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int to = (nt + rot) & (parts - 1), slot = nt >> plog;
      const int turn = NT >= parts ? item : (item * NT + nt) >> plog;  // the receiver's uses before
      const int there = (warp & ~(a.halves - 1)) + (to & (a.halves - 1));  // its warp
      const uint32_t at = sbase + a.recv_off + (there * 2 + (turn & 1)) * recv + (slot * parts + part) * 512 + lane * 16;
      if (a.blocks == 1)  // not in a cluster: one part, each lane's own sums
        *reinterpret_cast<float4*>(smem + at - sbase) = make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
      else if (!quiet)
        st_async16(cluster_map(at, to >> hlog), cluster_map(smem_u32(&bars[there][turn & 1]), to >> hlog), acc[nt]);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[nt][i] = 0.0f;
    }
    const int own = (part - rot) & (parts - 1);  // this warp's first column of the item
    if (own >= NT) return;
    const uint32_t bar = smem_u32(&bars[warp][uses & 1]);
    const int cols = NT >= parts ? NT >> plog : 1;
    if (a.blocks > 1) {
      if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(cols * parts * 512));
      __syncwarp();
      const uint32_t parity = (uint32_t)(uses >> 1) & 1u;
      if (live && !mbar_try_wait_cluster(bar, parity)) {
        live = mbar_wait_bounded(bar, parity, a.wait_limit_ns, nullptr, a.err);
        if (live) live = mbar_try_wait_cluster(bar, parity);
      }
      live = __all_sync(0xffffffffu, live);
    }
    if (live) {
      const uint8_t* buf = smem + a.recv_off + (warp * 2 + (uses & 1)) * recv + lane * 16;
#pragma unroll 1
      for (int c = 0; c < cols; ++c) {
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int q = 0; q < parts; ++q) {
          const float4 p = *reinterpret_cast<const float4*>(buf + (c * parts + q) * 512);
          v[0] += p.x;
          v[1] += p.y;
          v[2] += p.z;
          v[3] += p.w;
        }
        finish(unit, own + c * parts, v);
      }
    }
    ++uses;
  };

  int item = 0, cc = 0;
  auto compute = [&](uint4 (&w)[2 * LF_BLOCKS]) {
    const int left = nkl - cc * LF_BLOCKS;
#pragma unroll
    for (int j = 0; j < LF_BLOCKS; ++j) {
      if (j < left) {
        const bool in = j < left - 1 || mine == nkl || left > LF_BLOCKS;  // past K: zeros
        const uint4 lo = w[2 * j], hi = w[2 * j + 1];
        uint4 x[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) x[nt] = lds128(xa[nt] + (cc * LF_BLOCKS + j) * 64);
        const uint32_t a0 = in ? lo.x : 0u, a1 = in ? hi.x : 0u, a2 = in ? lo.y : 0u, a3 = in ? hi.y : 0u;
        const uint32_t a4 = in ? lo.z : 0u, a5 = in ? hi.z : 0u, a6 = in ? lo.w : 0u, a7 = in ? hi.w : 0u;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_16816<BF16>(acc[nt], a0, a1, a2, a3, x[nt].x, x[nt].y);
          mma_16816<BF16>(acc[nt], a4, a5, a6, a7, x[nt].z, x[nt].w);
        }
      }
    }
    ++cc;
  };
  while (item < items) {
    compute(w0);
    load(w0);
    compute(w1);
    load(w1);
    if (cc == chunks) {
      cc = 0;
      flush(item++);
    }
  }
  if (a.blocks > 1) {  // no block goes while another may write to it
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    // After a wait that ran out this warp waited for no more of what it was sent:
    // all of it has been sent by now, and gets the time to land.
    if (!live) {
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 100000) {
      }
    }
  }
}

}  // namespace swiglu
