// vec16.cuh -- 16 bytes of a row as fp32 values, for the kernels that go over
// rows: 8 elements of bf16 or fp16, 4 of fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../csrc/sm103_ptx.cuh"

namespace swiglu {

// Debug builds: the error word (null where the call has no workspace) and the
// buffers that the launch may touch; empty in release builds.
struct RowCheck {
#ifdef SWIGLU_DEBUG
  int* err;
  DbgWin win;
#endif
};
__device__ __forceinline__ bool row_ok(const RowCheck& c, const void* p, int64_t bytes) {
#ifdef SWIGLU_DEBUG
  if (dbg_in(c.win, p, bytes)) return true;
  if (c.err != nullptr) dbg_fail(c.err);
  return false;
#else
  (void)c;
  (void)p;
  (void)bytes;
  return true;
#endif
}

template <class T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& w, float (&v)[4]) {
    v[0] = __uint_as_float(w.x);
    v[1] = __uint_as_float(w.y);
    v[2] = __uint_as_float(w.z);
    v[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static __device__ __forceinline__ float round(float v) { return v; }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& w, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = (&w.x)[i];
      v[2 * i] = __uint_as_float(u << 16);
      v[2 * i + 1] = __uint_as_float(u & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
    uint4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      (&w.x)[i] = *reinterpret_cast<uint32_t*>(&h);
    }
    return w;
  }
  static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ __nv_bfloat16 round(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Vec<__half> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& w, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&(&w.x)[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
    uint4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      (&w.x)[i] = *reinterpret_cast<uint32_t*>(&h);
    }
    return w;
  }
  static __device__ __forceinline__ float one(const __half* p) { return __half2float(*p); }
  static __device__ __forceinline__ __half round(float v) { return __float2half_rn(v); }
};

// 16 bytes of global memory that are used once: not kept in L1
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 w;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
               : "l"(p)
               : "memory");
  return w;
}

// 16 bytes, global to shared, asynchronously; each thread waits for its own.
__device__ __forceinline__ void cp16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace swiglu
