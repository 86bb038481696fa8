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
// not E S^2 - mu^2, which cancels where |mu| is large against the deviation; the
// same pass finds what the first sum's roundings left in the mean, which a row
// of small deviation would have multiplied by a large rstd.
//
// Both are bound by memory: every input is read once and every output written
// once.  A row is held by TPR threads, VPT vectors of 16 bytes each.
//
// Backward is persistent: a block's groups of TPR threads take rows in turn and
// keep the gradients of w and b of their columns in registers, so that the
// reduction over rows costs one partial row pair per block.  Its rows arrive
// through a ring in shared memory that each thread fills for itself (cp.async):
// no thread waits for another's copies.  Partial sums are added in the order of
// the groups, then of the blocks: the result does not depend on timing.
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

// Sums of v.x and v.y over the TPR threads of a row.  `slots`: TPR / 32 pairs
// that no other use of this row's sums touches.
template <int TPR>
__device__ __forceinline__ float2 row_sums(float2 v, float2* slots) {
  v.x = warp_sum(v.x);
  v.y = warp_sum(v.y);
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    const int warp = (threadIdx.x % TPR) >> 5;
    if ((threadIdx.x & 31) == 0) slots[warp] = v;
    __syncthreads();
    v = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      v.x += slots[i].x;
      v.y += slots[i].y;
    }
  }
  return v;
}

// ROWS rows a block of ROWS * TPR threads (ROWS > 1 only with TPR = 32).
template <class T, int TPR, int VPT, int ROWS>
__global__ void __launch_bounds__(TPR* ROWS) ln_fwd_kernel(const LnFwdArgs a) {
  static_assert(ROWS == 1 || TPR == 32, "several rows a block: one warp each");
  using V = Vec<T>;
  constexpr int N = V::N;
  __shared__ float2 slots[2][TPR > 32 ? TPR / 32 : 1];
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
  float sum = 0.0f;
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
    for (int j = 0; j < N; ++j) sum += v[i][j];
  }
  const float n = (float)a.D;
  float mean = row_sums<TPR>(make_float2(sum, 0.0f), slots[0]).x / n;
  float2 sq = make_float2(0.0f, 0.0f);  // squares about the mean, and what the mean is off by
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (t + i * TPR < nv) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        v[i][j] -= mean;
        sq.x = fmaf(v[i][j], v[i][j], sq.x);
        sq.y += v[i][j];
      }
    }
  sq = row_sums<TPR>(sq, slots[1]);
  const float off = sq.y / n;
  const float var = sq.x / n - off * off;
  const float rstd = 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + a.eps);
  mean += off;
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
    for (int j = 0; j < N; ++j) v[i][j] = fmaf((v[i][j] - off) * rstd, w[j], b[j]);
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
  float wv[VPT][N];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int at = t + i * TPR;
    const T* pw = static_cast<const T*>(a.w) + at * N;
#pragma unroll
    for (int j = 0; j < N; ++j) wv[i][j] = 1.0f;
    if (a.w != nullptr && at < nv && row_ok(a.chk, pw, 16))
      V::unpack(*reinterpret_cast<const uint4*>(pw), wv[i]);
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
      float dy[N], s[N];
      V::unpack(*slot(stage, 0, i), dy);
      V::unpack(*slot(stage, 1, i), s);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float h = (s[j] - mean) * rstd, tt = dy[j] * wv[i][j];
        st = fmaf(dy[j], wv[i][j], st);
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
      float dy[N], s[N], d[N];
      V::unpack(*slot(stage, 0, i), dy);
      V::unpack(*slot(stage, 1, i), s);
      if constexpr (DS) V::unpack(*slot(stage, 2, i), d);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float h = (s[j] - mean) * rstd;
        const float g = fmaf(-h, sth, fmaf(dy[j], wv[i][j], -st));
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
  // the block's sums: groups in turn, in shared memory (past the ring's use)
  __syncthreads();
  float* acc = reinterpret_cast<float*>(ring);  // [2][D]
  for (int g = 0; g < GROUPS; ++g) {
    if (group == g) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int at = t + i * TPR;
        if (at >= nv) continue;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          float* pw = acc + at * N + j;
          float* pb = pw + a.D;
          *pw = g == 0 ? gw[i][j] : *pw + gw[i][j];
          *pb = g == 0 ? gb[i][j] : *pb + gb[i][j];
        }
      }
    }
    __syncthreads();
  }
  float* out = a.part + (int64_t)blockIdx.x * 2 * a.D;
  for (int c = threadIdx.x * 4; c < 2 * a.D; c += LNB_THREADS * 4)
    if (row_ok(a.chk, out + c, 16))
      *reinterpret_cast<float4*>(out + c) = *reinterpret_cast<const float4*>(acc + c);
}

}  // namespace swiglu
