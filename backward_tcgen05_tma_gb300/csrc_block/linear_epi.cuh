// linear_epi.cuh -- the epilogues of the linear operators for the tensor-core
// kernels (tc_gemm.cuh, tc2_gemm.cuh).
//
//   forward   z = acc + bias[n],  Z = rnd(z) where it is kept,  Y = rnd(act(z) + R)
//   backward  dX = rnd(acc act'(Xpre)), the gradient of what X = act(Xpre) was made from
//
// Bias, activation and residual meet in fp32 and are rounded once.
#pragma once

#include "../csrc/tc2_gemm.cuh"
#include "act.cuh"

namespace swiglu {

// Row pointers of one 32 x 32 chunk (first row mw, first column nc) of a
// row-major 16-bit matrix; rows past the matrix are null.
__device__ __forceinline__ auto chunk_rows(const TcShape& s, const void* base, int64_t ld, int mw,
                                           int nc) {
  return [=, &s](int r) -> uint8_t* {
    const int m = mw + r;
    return m < s.M ? static_cast<uint8_t*>(const_cast<void*>(base)) + ((int64_t)m * ld + nc) * 2
                   : nullptr;
  };
}

struct EpiLinear {
  struct Params {
    const void* bias;  // [N] or null
    const void* res;   // [M, N] or null
    void* z;           // [M, N] or null
    void* y;           // [M, N]
    int64_t ld;        // elements
    int act;
  };
  template <int BN, bool BF16>
  static __device__ __forceinline__ void run(const Params& p, const TcShape& s, uint32_t tacc,
                                             int m0, int nt, int row, int half, uint8_t* buf) {
    using P = Pack<BF16>;
    const int lane = row & 31;
    const int mw = m0 + (row & ~31);
    const int n0 = nt * BN;
#pragma unroll 1
    for (int c = half * (BN / 64); c < (half + 1) * (BN / 64); ++c) {
      const int nc = n0 + c * 32;
      auto ok = [&](int q) { return nc + q * 8 + 8 <= s.N; };
      uint4 rw[4];
      if (p.res != nullptr)
        warp_load_issue(rw, lane, checked_rows(s, chunk_rows(s, p.res, p.ld, mw, nc), ok), ok);
      uint4 bq[4];
      const uint4* bias = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.bias) +
                                                         (int64_t)nc * 2);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        bq[q] = p.bias != nullptr && ok(q) && SWIGLU_CHECK_PTR(s.dbg, bias + q, 16, s.err)
                    ? bias[q]
                    : make_uint4(0u, 0u, 0u, 0u);
      uint32_t r[32];
      tmem_ld_32x32b_x32(tacc + c * 32, r);
      tmem_ld_wait();
      float v[32];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 b = P::unpack((&bq[i >> 2].x)[i & 3]);
        v[2 * i] = __uint_as_float(r[2 * i]) + b.x;
        v[2 * i + 1] = __uint_as_float(r[2 * i + 1]) + b.y;
      }
      uint32_t w[16];
      if (p.z != nullptr) {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = P::two(v[2 * i], v[2 * i + 1]);
        warp_store_tile(buf, w, lane, checked_rows(s, chunk_rows(s, p.z, p.ld, mw, nc), ok), ok);
      }
      act_switch(p.act, [&](auto a) {
#pragma unroll
        for (int i = 0; i < 32; i += 2) act_value2<decltype(a)::value>(v[i], v[i + 1]);
      });
      if (p.res != nullptr) {
        uint4 rr[4];
        warp_load_finish(buf, rw, lane, rr);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 b = P::unpack((&rr[i >> 2].x)[i & 3]);
          v[2 * i] += b.x;
          v[2 * i + 1] += b.y;
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = P::two(v[2 * i], v[2 * i + 1]);
      warp_store_tile(buf, w, lane, checked_rows(s, chunk_rows(s, p.y, p.ld, mw, nc), ok), ok);
    }
  }
};

// 32 bytes, a whole sector, to or from a lane's own row
__device__ __forceinline__ void st_sector(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void ld_sector(const void* p, uint32_t* w) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}

// The same where rows start on 32 bytes (N a multiple of 16, buffers aligned so):
// a lane stores its own row's sectors whole, straight from its registers.  The
// plain form turns every chunk round through shared memory to that end, and
// stores by TMA wait behind the ring's loads in that unit: 16384 x 2816 x 1024 with
// gelu and Z took 117 us with it (stream-K shares among it), 90 with TMA stores, 80
// with these and launches that overlap (81 to 88 on other boxes).  Without Z it takes
// 12 us less, the rate at which Z's bytes go to memory.
struct EpiLinearSectors {
  using Params = EpiLinear::Params;
  template <int BN, bool BF16>
  static __device__ __forceinline__ void run(const Params& p, const TcShape& s, uint32_t tacc, int m0, int nt,
                                             int row, int half, uint8_t*) {
    using P = Pack<BF16>;
    const int m = m0 + row, n0 = nt * BN;
    constexpr int CH = BN / 64;
    auto at = [&](const void* base, int nc) {
      return static_cast<uint8_t*>(const_cast<void*>(base)) + ((int64_t)m * p.ld + nc) * 2;
    };
#pragma unroll 1
    for (int c = half * CH; c < (half + 1) * CH; ++c) {
      const int nc = n0 + c * 32;
      if (nc >= s.N) return;
      const bool in0 = m < s.M, in1 = m < s.M && nc + 32 <= s.N;  // the row's two sectors
      uint32_t rr[16], w[16];
      uint4 bq[4];
      const uint4* bias = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.bias) + (int64_t)nc * 2);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        bq[q] = p.bias != nullptr && nc + q * 8 + 8 <= s.N && SWIGLU_CHECK_PTR(s.dbg, bias + q, 16, s.err)
                    ? bias[q]
                    : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int i = 0; i < 16; ++i) rr[i] = 0;
      if (p.res != nullptr) {
        if (in0 && SWIGLU_CHECK_PTR(s.dbg, at(p.res, nc), 32, s.err)) ld_sector(at(p.res, nc), rr);
        if (in1 && SWIGLU_CHECK_PTR(s.dbg, at(p.res, nc + 16), 32, s.err)) ld_sector(at(p.res, nc + 16), rr + 8);
      }
      auto store = [&](void* base) {
        if (in0 && SWIGLU_CHECK_PTR(s.dbg, at(base, nc), 32, s.err)) st_sector(at(base, nc), w);
        if (in1 && SWIGLU_CHECK_PTR(s.dbg, at(base, nc + 16), 32, s.err)) st_sector(at(base, nc + 16), w + 8);
      };
      uint32_t r[32];
      tmem_ld_32x32b_x32(tacc + c * 32, r);
      tmem_ld_wait();
      float v[32];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 b = P::unpack((&bq[i >> 2].x)[i & 3]);
        add2(F2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), F2(b.x, b.y)).get(v[2 * i], v[2 * i + 1]);
      }
      if (p.z != nullptr) {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = P::two(v[2 * i], v[2 * i + 1]);
        store(p.z);
      }
      act_switch(p.act, [&](auto a) {
#pragma unroll
        for (int i = 0; i < 32; i += 2) act_value2<decltype(a)::value>(v[i], v[i + 1]);
      });
      if (p.res != nullptr) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 b = P::unpack(rr[i]);
          add2(F2(v[2 * i], v[2 * i + 1]), F2(b.x, b.y)).get(v[2 * i], v[2 * i + 1]);
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = P::two(v[2 * i], v[2 * i + 1]);
      store(p.y);
    }
  }
};

struct EpiDAct {
  struct Params {
    const void* pre;  // [M, N]
    void* out;        // [M, N]
    int64_t ld;       // elements
    int act;
  };
  template <int BN, bool BF16>
  static __device__ __forceinline__ void run(const Params& p, const TcShape& s, uint32_t tacc,
                                             int m0, int nt, int row, int half, uint8_t* buf) {
    using P = Pack<BF16>;
    const int lane = row & 31;
    const int mw = m0 + (row & ~31);
    const int n0 = nt * BN;
    constexpr int CH = BN / 64;
    uint4 zw[4];  // the next chunk's
    auto issue = [&](int c) {
      const int nc = n0 + c * 32;
      auto ok = [&](int q) { return nc + q * 8 + 8 <= s.N; };
      warp_load_issue(zw, lane, checked_rows(s, chunk_rows(s, p.pre, p.ld, mw, nc), ok), ok);
    };
    issue(half * CH);
#pragma unroll 1
    for (int c = half * CH; c < (half + 1) * CH; ++c) {
      const int nc = n0 + c * 32;
      auto ok = [&](int q) { return nc + q * 8 + 8 <= s.N; };
      uint4 zr[4];
      warp_load_finish(buf, zw, lane, zr);
      if (c + 1 < (half + 1) * CH) issue(c + 1);
      uint32_t r[32];
      tmem_ld_32x32b_x32(tacc + c * 32, r);
      tmem_ld_wait();
      uint32_t w[16];
      act_switch(p.act, [&](auto a) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float2 z = P::unpack((&zr[i >> 2].x)[i & 3]);
          act_slope2<decltype(a)::value>(z.x, z.y);
          w[i] = P::two(__uint_as_float(r[2 * i]) * z.x, __uint_as_float(r[2 * i + 1]) * z.y);
        }
      });
      warp_store_tile(buf, w, lane, checked_rows(s, chunk_rows(s, p.out, p.ld, mw, nc), ok), ok);
    }
  }
};

}  // namespace swiglu
