// w4_layout.cuh -- 4-bit weights: rounding 16-bit weights to codes and group
// scales, laying codes out for the few-token kernels, and expanding them.
//
// A packed matrix [R, K] is a run of 16-row tiles (a gate/up pair: 8 rows of
// Wg and the 8 rows of Wu of the same hidden units), in three parts:
//   codes   tile x ceil(K/64) blocks of 512 bytes; lane l = 4 g + t of a warp
//           has 16 bytes at 16 l: word 2 c + h holds, of rows g and g + 8, the
//           k = 32 c + 8 t + 4 h + {0..3} of the block's 64: nibbles 0, 4, 2, 6
//           are row g's, 1, 5, 3, 7 row g + 8's;
//   scales  tile x groups x 16, 16-bit, rows in the order 0, 8, 1, 9, ...;
//   zeros   (with zero points) tile x groups x 16 bytes in the same order.
// Rows past R have scale 0 and code = zero point; k past K has code 8.
#pragma once

#include "fewtok.cuh"

namespace swiglu {

struct W4Geom {
  int64_t N;      // rows of the matrix (gate/up: 2H)
  int K, group_log2, groups, zeros, gate_up;
  int blocks;     // 64-k blocks of a row
  int tiles;      // 16-row tiles
  int64_t scales_off, zeros_off, bytes;  // of one packed matrix
};

__host__ __device__ inline W4Geom w4_geom(int64_t N, int64_t K, int group_log2, int zeros,
                                          int gate_up) {
  W4Geom w;
  w.N = N;
  w.K = (int)K;
  w.group_log2 = group_log2;
  w.groups = (int)((K + (1 << group_log2) - 1) >> group_log2);
  w.zeros = zeros;
  w.gate_up = gate_up;
  w.blocks = (int)((K + 63) >> 6);
  w.tiles = (int)(gate_up ? (N / 2 + 7) / 8 : (N + 15) / 16);
  w.scales_off = (int64_t)w.tiles * w.blocks * 512;
  w.zeros_off = w.scales_off + (int64_t)w.tiles * w.groups * 32;
  w.bytes = w.zeros_off + (zeros ? (int64_t)w.tiles * w.groups * 16 : 0);
  return w;
}

// Row of the matrix that row r (0..15) of a tile holds, or -1 past its end.
__device__ __forceinline__ int64_t w4_row(const W4Geom& w, int tile, int r) {
  if (w.gate_up) {
    const int64_t u = (int64_t)tile * 8 + (r & 7);
    return u < w.N / 2 ? u + (r >= 8 ? w.N / 2 : 0) : -1;
  }
  const int64_t n = (int64_t)tile * 16 + r;
  return n < w.N ? n : -1;
}

// One thread per 16 bytes of a matrix's packed codes, then per scale.
__global__ void w4_pack_kernel(W4Geom w, int64_t experts, const uint8_t* codes,
                               const uint16_t* scales, const uint8_t* zeros, uint8_t* packed) {
  const int64_t nc = (int64_t)w.tiles * w.blocks * 32, ns = (int64_t)w.tiles * w.groups * 16;
  const int64_t total = (nc + ns) * experts;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t e = i / (nc + ns), j = i - e * (nc + ns);
    uint8_t* out = packed + e * w.bytes;
    if (j < nc) {
      const int lane = (int)(j & 31), g = lane >> 2, t = lane & 3;
      const int b = (int)((j >> 5) % w.blocks), tile = (int)((j >> 5) / w.blocks);
      const int64_t r0 = w4_row(w, tile, g), r1 = w4_row(w, tile, g + 8);
      uint32_t o[4];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int k = b * 64 + c * 32 + t * 8;
        uint32_t v0 = 0x88888888u, v1 = 0x88888888u;  // 8 codes of each row, nibble n = k + n
        if (k < w.K) {
          const int64_t half = w.K / 2;
          if (r0 >= 0) v0 = *reinterpret_cast<const uint32_t*>(codes + (e * w.N + r0) * half + k / 2);
          if (r1 >= 0) v1 = *reinterpret_cast<const uint32_t*>(codes + (e * w.N + r1) * half + k / 2);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t a = v0 >> (16 * h), q = v1 >> (16 * h);
          o[2 * c + h] = (a & 15u) | (q & 15u) << 4 | ((a >> 8) & 15u) << 8 | ((q >> 8) & 15u) << 12 |
                         ((a >> 4) & 15u) << 16 | ((q >> 4) & 15u) << 20 |
                         ((a >> 12) & 15u) << 24 | ((q >> 12) & 15u) << 28;
        }
      }
      reinterpret_cast<uint4*>(out)[j] = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
      const int64_t q = j - nc;
      const int slot = (int)(q & 15), gr = (int)((q >> 4) % w.groups),
                tile = (int)((q >> 4) / w.groups);
      const int64_t r = w4_row(w, tile, (slot >> 1) + 8 * (slot & 1));
      const int64_t src = (e * w.N + r) * w.groups + gr;
      reinterpret_cast<uint16_t*>(out + w.scales_off)[q] = r >= 0 ? scales[src] : 0;
      if (w.zeros) out[w.zeros_off + q] = r >= 0 ? zeros[src] & 15u : 8u;
    }
  }
}

// W[n, k] = rnd(s (q - z)), one thread per 16 bytes of packed codes; s (q - z)
// is exact in fp32 (12 + 4 bits), so each weight is rounded once.
template <bool BF16>
__global__ void w4_unpack_kernel(W4Geom w, int64_t experts, const uint8_t* packed, uint16_t* W) {
  const int64_t nc = (int64_t)w.tiles * w.blocks * 32, total = nc * experts;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t e = i / nc, j = i - e * nc;
    const uint8_t* in = packed + e * w.bytes;
    const int lane = (int)(j & 31), g = lane >> 2, t = lane & 3;
    const int b = (int)((j >> 5) % w.blocks), tile = (int)((j >> 5) / w.blocks);
    const uint4 v = reinterpret_cast<const uint4*>(in)[j];
    const uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int k = b * 64 + c * 32 + t * 8;
      if (k >= w.K) continue;
      const int64_t gi = (int64_t)tile * w.groups + (k >> w.group_log2);
#pragma unroll
      for (int hi = 0; hi < 2; ++hi) {
        const int64_t r = w4_row(w, tile, g + 8 * hi);
        if (r < 0) continue;
        const uint16_t sb = reinterpret_cast<const uint16_t*>(in + w.scales_off)[gi * 16 + g * 2 + hi];
        const float s = Ft16<BF16>::lo(sb);
        const int z = w.zeros ? in[w.zeros_off + gi * 16 + g * 2 + hi] : 8;
        uint32_t o[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t x = word[2 * c + h] >> (4 * hi);
          // nibbles 0, 4 are k + {0, 1}; 2, 6 are k + {2, 3}
          o[2 * h] = Ft16<BF16>::rnd(s * (float)((int)(x & 15u) - z)) |
                     (uint32_t)Ft16<BF16>::rnd(s * (float)((int)((x >> 16) & 15u) - z)) << 16;
          o[2 * h + 1] = Ft16<BF16>::rnd(s * (float)((int)((x >> 8) & 15u) - z)) |
                         (uint32_t)Ft16<BF16>::rnd(s * (float)((int)((x >> 24) & 15u) - z)) << 16;
        }
        *reinterpret_cast<uint4*>(W + (e * w.N + r) * w.K + k) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

// Rounds rows of 16-bit weights to codes with one scale per group: a thread
// takes 8 weights, the 4, 8 or 16 threads of a group meet by shuffles.
//   without zero points  s = rnd(max |w| / 7),               q = clamp(rint(w / s) + 8)
//   with                 s = rnd((max(w, 0) - min(w, 0)) / 15), z = clamp(rint(-min(w, 0) / s)),
//                        q = clamp(rint(w / s) + z)
// clamp: to 0..15; a scale that rounds to 0 gives q = z (= 8): weights of 0.
template <bool BF16>
__global__ void w4_quantize_kernel(int64_t N, int K, int group_log2, int groups, const uint16_t* W,
                                   uint8_t* codes, uint16_t* scales, uint8_t* zeros) {
  const int lanes = 1 << (group_log2 - 3);            // threads of a group
  const int64_t per_row = (int64_t)groups * lanes, total = N * per_row;
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  // whole warps stay in the loop together: the shuffles need every lane
  for (int64_t base = blockIdx.x * (int64_t)blockDim.x + (threadIdx.x & ~31); base < total;
       base += step) {
    const int64_t i = base + (threadIdx.x & 31);
    const bool in_row = i < total;
    const int64_t n = in_row ? i / per_row : 0;
    const int k = in_row ? (int)(i - n * per_row) * 8 : 0;
    const bool in = in_row && k < K;
    float w[8];
    float lo = 0.0f, hi = 0.0f;
    if (in) {
      const uint4 v = *reinterpret_cast<const uint4*>(W + n * K + k);
      const uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[2 * j] = Ft16<BF16>::lo(word[j]);
        w[2 * j + 1] = Ft16<BF16>::hi(word[j]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        lo = fminf(lo, w[j]);
        hi = fmaxf(hi, w[j]);
      }
    }
    for (int d = 1; d < lanes; d <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, d));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
    }
    if (!in) continue;
    const uint16_t sb = Ft16<BF16>::rnd(zeros ? __fdiv_rn(hi - lo, 15.0f) : __fdiv_rn(fmaxf(hi, -lo), 7.0f));
    const float s = Ft16<BF16>::lo(sb);
    float z = 8.0f;
    if (zeros && s != 0.0f) z = fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.0f), 15.0f);
    uint32_t o = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float q = s != 0.0f ? fminf(fmaxf(rintf(__fdiv_rn(w[j], s)) + z, 0.0f), 15.0f) : z;
      o |= (uint32_t)(int)q << (4 * j);
    }
    *reinterpret_cast<uint32_t*>(codes + (n * K + k) / 2) = o;
    if (k % (1 << group_log2) == 0) {
      const int64_t at = n * groups + (k >> group_log2);
      scales[at] = sb;
      if (zeros) zeros[at] = (uint8_t)(int)z;
    }
  }
}

}  // namespace swiglu
