// column_sums.cuh -- sums over the rows of a matrix: a linear layer's bias
// gradient, taken in the pass that multiplies dY by the activation's
// derivative, and the second half of every such reduction.
//
//   dZ = rnd(dY act'(Z)),   db = sum over rows of dY act'(Z) (not of the rounded dZ)
//
// Bound by memory.  A warp reads 512 contiguous bytes of a row; a block's 8
// warps take the rows of its part in turn, the next ones' loads under way, and its
// sums meet in shared memory; the parts' sums are added by a second kernel in the
// order of the parts.  Measured: 16384 x 2816 fp16 with gelu 52 us (5.3 TB/s; 78
// before activations went in pairs and rows were read ahead), 32768 x 2048 bf16
// without 26 us (5.2 TB/s).  No more registers than it needs: where they filled
// the SM, the products behind it could not start early (20 us of 205).
#pragma once

#include "act.cuh"
#include "vec16.cuh"

namespace swiglu {

struct DactArgs {
  const void* dy;   // [M, N]
  const void* z;    // [M, N], with an activation
  void* dz;         // [M, N], with one
  float* part;      // [gridDim.y][N], or null: no sums
  int64_t M;
  int N;
  int act;
  int* err;         // cleared here
  RowCheck chk;
};

constexpr int DA_THREADS = 256, DA_WARPS = DA_THREADS / 32;

template <class T, bool ACT>
__global__ void __launch_bounds__(DA_THREADS) dact_kernel(const DactArgs a) {
  using V = Vec<T>;
  constexpr int N = V::N, DA_BATCH = ACT ? 2 : 4;  // rows of a warp at a time
  __shared__ float acc[DA_WARPS][32][N + 1];
  pdl_wait();  // launched early: nothing is touched before the kernel before has ended
  pdl_launch_dependents();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.err = 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = (blockIdx.x * 32 + lane) * N;
  const int64_t r0 = a.M * blockIdx.y / gridDim.y, r1 = a.M * (blockIdx.y + 1) / gridDim.y;
  float sum[N];
#pragma unroll
  for (int j = 0; j < N; ++j) sum[j] = 0.0f;
  if (col < a.N) {
    // the next rows' loads are on their way while these are used
    uint4 wy[DA_BATCH], wz[DA_BATCH];
    auto load = [&](int64_t r) {
#pragma unroll
      for (int b = 0; b < DA_BATCH; ++b) {
        const int64_t row = r + b * DA_WARPS, o = row * a.N + col;
        wy[b] = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (ACT) wz[b] = wy[b];
        if (row < r1) {
          const T* py = static_cast<const T*>(a.dy) + o;
          if (row_ok(a.chk, py, 16)) wy[b] = ld_stream(py);
          if constexpr (ACT) {
            const T* pz = static_cast<const T*>(a.z) + o;
            if (row_ok(a.chk, pz, 16)) wz[b] = ld_stream(pz);
          }
        }
      }
    };
    load(r0 + warp);
    for (int64_t r = r0 + warp; r < r1; r += DA_WARPS * DA_BATCH) {
      uint4 cy[DA_BATCH], cz[DA_BATCH];
#pragma unroll
      for (int b = 0; b < DA_BATCH; ++b) {
        cy[b] = wy[b];
        if constexpr (ACT) cz[b] = wz[b];
      }
      load(r + DA_WARPS * DA_BATCH);
#pragma unroll
      for (int b = 0; b < DA_BATCH; ++b) {
        const int64_t row = r + b * DA_WARPS;
        if (row >= r1) break;
        float y[N];
        V::unpack(cy[b], y);
        if constexpr (ACT) {
          float z[N];
          V::unpack(cz[b], z);
          act_switch(a.act, [&](auto t) {
#pragma unroll
            for (int j = 0; j < N; j += 2) {
              if constexpr (N == 4) {
                z[j] = ActPrecise::slope<decltype(t)::value>(z[j]);
                z[j + 1] = ActPrecise::slope<decltype(t)::value>(z[j + 1]);
              } else {
                act_slope2<decltype(t)::value>(z[j], z[j + 1]);
              }
              y[j] = __fmul_rn(y[j], z[j]);
              y[j + 1] = __fmul_rn(y[j + 1], z[j + 1]);
            }
          });
          T* pd = static_cast<T*>(a.dz) + row * a.N + col;
          if (row_ok(a.chk, pd, 16)) *reinterpret_cast<uint4*>(pd) = V::pack(y);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) sum[j] += y[j];
      }
    }
  }
  if (a.part == nullptr) return;
#pragma unroll
  for (int j = 0; j < N; ++j) acc[warp][lane][j] = sum[j];
  __syncthreads();
  for (int c = threadIdx.x; c < 32 * N; c += DA_THREADS) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < DA_WARPS; ++w) v += acc[w][c / N][c % N];
    const int at = blockIdx.x * 32 * N + c;
    float* out = a.part + (int64_t)blockIdx.y * a.N + at;
    if (at < a.N && row_ok(a.chk, out, 4)) *out = v;
  }
}

// out[c] = rnd(sum over p of part[p][c]), or with `add` rnd(out[c] + that sum).
// Columns [0, n) go to out0 and [n, 2n) to out1; a null output takes none.
struct ColumnSumArgs {
  const float* part;  // [parts][cols]
  void* out0;
  void* out1;
  int parts, cols, n;
  int add;
  RowCheck chk;
};

constexpr int CS_COLS = 32;  // columns of a block: 8 quads of columns x 32 shares of the parts

template <class T>
__global__ void __launch_bounds__(256) column_sum_kernel(const ColumnSumArgs a) {
  __shared__ float4 acc[32][8];
  pdl_wait();
  pdl_launch_dependents();
  const int q = threadIdx.x & 7, share = threadIdx.x >> 3;
  const int c = blockIdx.x * CS_COLS + q * 4;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (c < a.cols) {
#pragma unroll 4
    for (int p = share; p < a.parts; p += 32) {
      const float* src = a.part + (int64_t)p * a.cols + c;
      if (!row_ok(a.chk, src, 16)) continue;
      const float4 w = *reinterpret_cast<const float4*>(src);
      v.x += w.x;
      v.y += w.y;
      v.z += w.z;
      v.w += w.w;
    }
  }
  acc[share][q] = v;
  __syncthreads();
  if (threadIdx.x >= CS_COLS) return;
  const int col = blockIdx.x * CS_COLS + threadIdx.x;
  if (col >= a.cols) return;
  float sum = 0.0f;
#pragma unroll
  for (int s = 0; s < 32; ++s) sum += (&acc[s][threadIdx.x >> 2].x)[threadIdx.x & 3];
  T* out = static_cast<T*>(col < a.n ? a.out0 : a.out1);
  if (out == nullptr) return;
  out += col < a.n ? col : col - a.n;
  if (!row_ok(a.chk, out, sizeof(T))) return;
  *out = Vec<T>::round(a.add ? Vec<T>::one(out) + sum : sum);
}

}  // namespace swiglu
