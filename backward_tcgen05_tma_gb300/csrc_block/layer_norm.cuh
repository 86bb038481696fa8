// layer_norm.cuh -- layer norm over rows of D elements, with the residual sum
// in front of it, and its backward pass with the reduction of the weight's and
// the bias's gradients.
//
//   forward   S = rnd(X + R) or X,  mu = mean S,  rstd = (mean (S - mu)^2 + eps)^-1/2,
//             Y = rnd((S - mu) rstd w + b)
//   backward  h = (S - mu) rstd,  t = dY w,
//             dX = rnd(rstd (t - mean t - h mean(t h)) + dS),
//             dw = sum over rows of dY h,  db = sum over rows of dY
//
// Everything is fp32 between the loads and the one rounding at the end.  The
// variance is the mean of squares about the mean (a second pass over registers),
// not E S^2 - mu^2, which cancels where |mu| is large against the deviation.  The
// mean's sum carries its roundings along: a row of small deviation multiplies
// what is left of them by a large rstd, and the mean of many unlike channels is
// small against their sum of sizes.
//
// Both are bound by memory: every input is read once and every output written
// once.  A row is held by TPR threads, VPT vectors of 16 bytes each.  Measured,
// with the residual: 65536 x 4096 bf16 309 us forward (6.9 TB/s) and 330 us
// backward (6.5 TB/s); 16384 x 1024 fp16 backward without one 27 us (3.7 TB/s: 7
// rows a warp, of which the first has to arrive and the sums to be added up).
//
// Backward is persistent: a block's groups of TPR threads (a warp up to 1024
// 16-bit elements: what bounds short rows is the latency of a row's two sums, so
// many rows are in progress) take rows in turn and keep the gradients of w and b
// of their columns in registers, so that the reduction over rows costs one
// partial row pair per block.  Its rows arrive through a ring in shared memory
// that each thread fills for itself (cp.async): no thread waits for another's
// copies.  (With two vectors a thread, half as many rows in progress, and the
// groups' sums added one group after another, these two cases took 390 and 36
// us.)  Partial sums are added in the order of the groups, then of the blocks: the
// result does not depend on timing.
#pragma once

#include "vec16.cuh"

namespace swiglu {

struct LnFwdArgs {
  const void* x;
  const void* res;   // or null
  const void* w;     // or null: 1
  const void* b;     // or null: 0
  void* s;           // with res: rnd(x + res)
  void* y;
  float* mean;       // or null
  float* rstd;       // or null
  int64_t M;
  int D;
  float eps;
  RowCheck chk;
};

// a + b = sum + err exactly (Knuth's two-sum)
__device__ __forceinline__ float two_sum(float a, float b, float& err) {
  const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
  err = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
  return s;
}

// Sum of v over the TPR threads of a row.  `slots`: TPR / 32 floats that no
// other use of this row's sums touches.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* slots) {
  v = warp_sum(v);
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) slots[(threadIdx.x % TPR) >> 5] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) v += slots[i];
  }
  return v;
}

// The same of v.x + v.y, v.y being what roundings left out of v.x.
template <int TPR>
__device__ __forceinline__ float row_sum_exact(float2 v, float2* slots) {
  float e;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    v.x = two_sum(v.x, __shfl_xor_sync(0xffffffffu, v.x, o), e);
    v.y += e;
  }
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) slots[(threadIdx.x % TPR) >> 5] = v;
    __syncthreads();
    v = slots[0];
#pragma unroll
    for (int i = 1; i < TPR / 32; ++i) {
      v.x = two_sum(v.x, slots[i].x, e);
      v.y += slots[i].y + e;
    }
  }
  return fabsf(v.x) < INFINITY ? v.x + v.y : v.x;  // (an infinity leaves no roundings but NaN)
}

// ROWS rows a block of ROWS * TPR threads (ROWS > 1 only with TPR = 32).
template <class T, int TPR, int VPT, int ROWS>
__global__ void __launch_bounds__(TPR* ROWS) ln_fwd_kernel(const LnFwdArgs a) {
  static_assert(ROWS == 1 || TPR == 32, "several rows a block: one warp each");
  using V = Vec<T>;
  constexpr int N = V::N;
  __shared__ float2 sums[TPR > 32 ? TPR / 32 : 1];
  __shared__ float squares[TPR > 32 ? TPR / 32 : 1];
  pdl_wait();  // launched early: nothing is touched before the kernel before has ended
  pdl_launch_dependents();
  const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
  if (ROWS > 1 && row >= a.M) return;
  const int t = threadIdx.x % TPR, nv = a.D / N;
  const int64_t base = row * a.D;
  float v[VPT][N];
  uint4 rx[VPT], rr[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int at = t + i * TPR;
    rx[i] = rr[i] = make_uint4(0u, 0u, 0u, 0u);
    if (at < nv) {
      const T* px = static_cast<const T*>(a.x) + base + at * N;
      if (row_ok(a.chk, px, 16)) rx[i] = ld_stream(px);
      if (a.res != nullptr) {
        const T* pr = static_cast<const T*>(a.res) + base + at * N;
        if (row_ok(a.chk, pr, 16)) rr[i] = ld_stream(pr);
      }
    }
  }
  float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int at = t + i * TPR;
    V::unpack(rx[i], v[i]);
    if (a.res != nullptr) {
      float r[N];
      V::unpack(rr[i], r);
#pragma unroll
      for (int j = 0; j < N; ++j) v[i][j] += r[j];
      const uint4 w = V::pack(v[i]);
      V::unpack(w, v[i]);  // the norm is that of the rounded sum, which backward sees
      T* ps = static_cast<T*>(a.s) + base + at * N;
      if (at < nv && row_ok(a.chk, ps, 16)) *reinterpret_cast<uint4*>(ps) = w;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float e;
      sum.x = two_sum(sum.x, v[i][j], e);
      sum.y += e;
    }
  }
  const float n = (float)a.D;
  const float mean = row_sum_exact<TPR>(sum, sums) / n;
  float sq = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (t + i * TPR < nv) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        v[i][j] -= mean;
        sq = fmaf(v[i][j], v[i][j], sq);
      }
    }
  const float rstd = 1.0f / sqrtf(row_sum<TPR>(sq, squares) / n + a.eps);
  if (t == 0) {
    if (a.mean != nullptr && row_ok(a.chk, a.mean + row, 4)) a.mean[row] = mean;
    if (a.rstd != nullptr && row_ok(a.chk, a.rstd + row, 4)) a.rstd[row] = rstd;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int at = t + i * TPR;
    if (at >= nv) continue;
    float w[N], b[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      w[j] = 1.0f;
      b[j] = 0.0f;
    }
    const T* pw = static_cast<const T*>(a.w) + at * N;
    const T* pb = static_cast<const T*>(a.b) + at * N;
    if (a.w != nullptr && row_ok(a.chk, pw, 16)) V::unpack(*reinterpret_cast<const uint4*>(pw), w);
    if (a.b != nullptr && row_ok(a.chk, pb, 16)) V::unpack(*reinterpret_cast<const uint4*>(pb), b);
#pragma unroll
    for (int j = 0; j < N; ++j) v[i][j] = fmaf(v[i][j] * rstd, w[j], b[j]);
    T* py = static_cast<T*>(a.y) + base + at * N;
    if (row_ok(a.chk, py, 16)) *reinterpret_cast<uint4*>(py) = V::pack(v[i]);
  }
}

struct LnBwdArgs {
  const void* dy;
  const void* s;
  const void* ds;      // or null
  const void* w;       // or null: 1
  const float* mean;
  const float* rstd;
  void* dx;
  float* part;         // [gridDim.x][2][D]: dw and db of the block's rows
  int64_t M;
  int D;
  int stages;          // of the ring
  int want;            // whether any of dw, db is wanted
  int* err;            // cleared here
  RowCheck chk;
};

constexpr int LNB_THREADS = 512;

// Group barrier 1 + group over its TPR threads.
template <int TPR>
__device__ __forceinline__ void group_bar(int group) {
  if constexpr (TPR > 32) asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(TPR) : "memory");
}

template <class T, int TPR, int VPT, bool DS>
__global__ void __launch_bounds__(LNB_THREADS, 1) ln_bwd_kernel(const LnBwdArgs a) {
  using V = Vec<T>;
  constexpr int N = V::N, GROUPS = LNB_THREADS / TPR, W = TPR / 32, TENS = DS ? 3 : 2;
  constexpr int SLOT = LNB_THREADS * 16;  // one vector of every thread
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float2 slots[2][LNB_THREADS / 32];
  pdl_wait();  // launched early: nothing is touched before the kernel before has ended
  pdl_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;
  const int group = threadIdx.x / TPR, t = threadIdx.x % TPR, nv = a.D / N;
  const int64_t step = (int64_t)gridDim.x * GROUPS;
  const int64_t first = (int64_t)blockIdx.x * GROUPS + group;
  uint8_t* const mine = ring + threadIdx.x * 16;
  auto slot = [&](int stage, int ten, int i) -> uint4* {
    return reinterpret_cast<uint4*>(mine + (size_t)((stage * TENS + ten) * VPT + i) * SLOT);
  };
  auto fetch = [&](int64_t row, int stage) {
    if (row < a.M) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int at = t + i * TPR;
        if (at >= nv) continue;
        const int64_t o = (row * a.D + at * N) * (int64_t)sizeof(T);
        const uint8_t* py = static_cast<const uint8_t*>(a.dy) + o;
        const uint8_t* ps = static_cast<const uint8_t*>(a.s) + o;
        if (row_ok(a.chk, py, 16)) cp16(slot(stage, 0, i), py);
        if (row_ok(a.chk, ps, 16)) cp16(slot(stage, 1, i), ps);
        if constexpr (DS) {
          const uint8_t* pd = static_cast<const uint8_t*>(a.ds) + o;
          if (row_ok(a.chk, pd, 16)) cp16(slot(stage, 2, i), pd);
        }
      }
    }
    cp_commit();  // (an empty group past the last row)
  };
  auto stat = [&](const float* p, int64_t row) {
    return row < a.M && row_ok(a.chk, p + row, 4) ? p[row] : 0.0f;
  };
  // a stage is refilled after the sums of its row are taken, one row ahead of
  // the stages' count: stages - 1 rows are on their way
  const int ahead = a.stages - 1;
  for (int i = 0; i < ahead; ++i) fetch(first + i * step, i);
  uint4 wv[VPT];  // the weight, as it is stored
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int at = t + i * TPR;
    const T* pw = static_cast<const T*>(a.w) + at * N;
    float one[N];
#pragma unroll
    for (int j = 0; j < N; ++j) one[j] = 1.0f;
    wv[i] = V::pack(one);
    if (a.w != nullptr && at < nv && row_ok(a.chk, pw, 16)) wv[i] = *reinterpret_cast<const uint4*>(pw);
  }
  float gw[VPT][N], gb[VPT][N];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) gw[i][j] = gb[i][j] = 0.0f;
  const float inv = 1.0f / (float)a.D;
  float mean = stat(a.mean, first), rstd = stat(a.rstd, first);
  int stage = 0, into = ahead, flip = 0;
  for (int64_t row = first; row < a.M; row += step) {
    fetch(row + ahead * step, into);
    // this row's copies are done when at most `ahead` later groups are not
    switch (ahead) {
      case 0: cp_wait<0>(); break;
      case 1: cp_wait<1>(); break;
      case 2: cp_wait<2>(); break;
      case 3: cp_wait<3>(); break;
      default: cp_wait<4>(); break;
    }
    const float next_mean = stat(a.mean, row + step), next_rstd = stat(a.rstd, row + step);
    float st = 0.0f, sth = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (t + i * TPR >= nv) continue;
      float dy[N], s[N], w[N];
      V::unpack(*slot(stage, 0, i), dy);
      V::unpack(*slot(stage, 1, i), s);
      V::unpack(wv[i], w);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float h = (s[j] - mean) * rstd, tt = dy[j] * w[j];
        st = fmaf(dy[j], w[j], st);
        sth = fmaf(tt, h, sth);
        gw[i][j] = fmaf(dy[j], h, gw[i][j]);
        gb[i][j] += dy[j];
      }
    }
    st = warp_sum(st);
    sth = warp_sum(sth);
    if constexpr (TPR > 32) {
      float2* sl = slots[flip] + group * W;
      if ((t & 31) == 0) sl[t >> 5] = make_float2(st, sth);
      group_bar<TPR>(group);
      st = sth = 0.0f;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float2 p = sl[i];
        st += p.x;
        sth += p.y;
      }
      flip ^= 1;  // the next row's sums: no thread is two rows behind another
    }
    st *= inv;
    sth *= inv;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int at = t + i * TPR;
      if (at >= nv) continue;
      float dy[N], s[N], d[N], w[N];
      V::unpack(*slot(stage, 0, i), dy);
      V::unpack(*slot(stage, 1, i), s);
      V::unpack(wv[i], w);
      if constexpr (DS) V::unpack(*slot(stage, 2, i), d);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float h = (s[j] - mean) * rstd;
        const float g = fmaf(-h, sth, fmaf(dy[j], w[j], -st));
        d[j] = DS ? fmaf(rstd, g, d[j]) : rstd * g;
      }
      T* px = static_cast<T*>(a.dx) + row * a.D + at * N;
      if (row_ok(a.chk, px, 16)) *reinterpret_cast<uint4*>(px) = V::pack(d);
    }
    mean = next_mean;
    rstd = next_rstd;
    if (++stage == a.stages) stage = 0;
    if (++into == a.stages) into = 0;
  }
  cp_wait<0>();
  if (!a.want) return;
  // the block's sums, in shared memory past the ring's use: every group's, element
  // j of the vectors apart so that lanes meet no bank twice, then over the groups
  __syncthreads();
  const int row_floats = N * (nv + 4), slab = 2 * row_floats;
  float* acc = reinterpret_cast<float*>(ring);  // [GROUPS][2][N][nv + 4]
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int at = t + i * TPR;
    if (at >= nv) continue;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      acc[group * slab + j * (nv + 4) + at] = gw[i][j];
      acc[group * slab + row_floats + j * (nv + 4) + at] = gb[i][j];
    }
  }
  __syncthreads();
  float* out = a.part + (int64_t)blockIdx.x * 2 * a.D;
  for (int c = threadIdx.x; c < 2 * a.D; c += LNB_THREADS) {
    const int which = c >= a.D, col = c - (which ? a.D : 0);
    const float* p = acc + which * row_floats + col % N * (nv + 4) + col / N;
    float v = 0.0f;
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) v += p[g * slab];
    if (row_ok(a.chk, out + c, 4)) out[c] = v;
  }
}

}  // namespace swiglu
