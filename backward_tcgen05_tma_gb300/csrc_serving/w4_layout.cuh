// w4_layout.cuh -- 4-bit weights: rounding 16-bit weights to codes and group
// scales, laying codes out for the few-token kernels, and expanding them.
//
// A packed matrix [R, K] is a run of 16-row tiles (a gate/up pair: 8 rows of
// Wg and the 8 rows of Wu of the same hidden units), each a run of records of
// 64 k, each
//   codes   512 bytes; lane l = 4 g + t of a warp has 16 bytes at 16 l: word
//           2 c + r holds the k = 32 c + 8 t + {0..7} of row g + 8 r: k + 0, 4,
//           2, 6 in nibbles 0..3, k + 1, 5, 3, 7 in nibbles 4..7;
//   scales  one set of 16 (groups of 32: two, one per half), 16-bit, rows in
//           the order 0, 8, 1, 9, ...; a scale of a group of 128 is in both of
//           the group's records, so that a record is all a unit needs (3% more
//           bytes, one address);
//   zeros   (with zero points) as many sets of 16 bytes, in the same order.
// Rows past R have scale 0; k past K have code 8, and scale 0 in a half of its
// own.
// Codes and scales in one record cost the readers one address and one copy; with
// scales in an array of their own w4_stream.cuh spent 47 us on what now takes 22.
// These kernels run once per checkpoint, bound by memory or by their byte
// gathers: 11008 x 4096 in groups of 128 round in 75 us (113 MB, 1.5 TB/s), pack
// in 19 us (47 MB, 2.4 TB/s) and expand in 25 us (113 MB, 4.5 TB/s).
#pragma once

#include "fewtok.cuh"

namespace swiglu {

struct W4Geom {
  int64_t N;      // rows of the matrix (gate/up: 2H)
  int K, group_log2, groups, zeros, gate_up;
  int blocks;     // records of a tile
  int tiles;      // 16-row tiles
  int sets;       // scale sets of a record
  int record;     // bytes
  int64_t bytes;  // of one packed matrix
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
  w.sets = group_log2 == 5 ? 2 : 1;
  w.record = 512 + w.sets * (zeros ? 48 : 32);
  w.bytes = (int64_t)w.tiles * w.blocks * w.record;
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

// The nibble of elements 2 n (and, 4 further on, 2 n + 1) of a word's 8: the
// first four elements lie where one mask finds them, the others where the
// other does, so that each meets two neighbouring registers of token elements.
__host__ __device__ constexpr int w4_nibble(int n) { return n == 1 ? 2 : n == 2 ? 1 : n; }

// One warp per record of the packed copy.
__global__ void w4_pack_kernel(W4Geom w, int64_t experts, const uint8_t* codes,
                               const uint16_t* scales, const uint8_t* zeros, uint8_t* packed) {
  const int64_t per = (int64_t)w.tiles * w.blocks, total = per * experts;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; i < total; i += warps) {
    const int64_t e = i / per, j = i - e * per;
    const int tile = (int)(j / w.blocks), b = (int)(j - (int64_t)tile * w.blocks);
    uint8_t* out = packed + e * w.bytes + j * w.record;
    uint32_t o[4];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int64_t row = w4_row(w, tile, g + 8 * r);
        const int k = b * 64 + c * 32 + t * 8;
        uint32_t v = 0x88888888u;  // nibble n: element k + n
        if (k < w.K && row >= 0)
          v = *reinterpret_cast<const uint32_t*>(codes + ((e * w.N + row) * w.K + k) / 2);
        uint32_t x = 0;
#pragma unroll
        for (int n = 0; n < 4; ++n) {  // elements 2 n and 2 n + 1
          const int at = 4 * w4_nibble(n);
          x |= ((v >> (8 * n)) & 15u) << at | ((v >> (8 * n + 4)) & 15u) << (16 + at);
        }
        o[2 * c + r] = x;
      }
    reinterpret_cast<uint4*>(out)[lane] = make_uint4(o[0], o[1], o[2], o[3]);
    if (lane < 16 * w.sets) {
      const int slot = lane & 15, h = lane >> 4;
      const int64_t row = w4_row(w, tile, (slot >> 1) + 8 * (slot & 1));
      const int gr = (b * 64 + h * 32) >> w.group_log2;
      const bool in = row >= 0 && gr < w.groups;
      const int64_t src = (e * w.N + row) * w.groups + gr;
      reinterpret_cast<uint16_t*>(out + 512)[lane] = in ? scales[src] : 0;
      if (w.zeros) out[512 + 32 * w.sets + lane] = in ? zeros[src] & 15u : 8u;
    }
  }
}

// W[n, k] = rnd(s (q - z)), one warp per record; s (q - z) is exact in fp32
// (12 + 4 bits), so each weight is rounded once.
template <bool BF16>
__global__ void w4_unpack_kernel(W4Geom w, int64_t experts, const uint8_t* packed, uint16_t* W) {
  const int64_t per = (int64_t)w.tiles * w.blocks, total = per * experts;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; i < total; i += warps) {
    const int64_t e = i / per, j = i - e * per;
    const int tile = (int)(j / w.blocks), b = (int)(j - (int64_t)tile * w.blocks);
    const uint8_t* in = packed + e * w.bytes + j * w.record;
    const uint4 v = reinterpret_cast<const uint4*>(in)[lane];
    const uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int64_t row = w4_row(w, tile, g + 8 * r);
        const int k = b * 64 + c * 32 + t * 8, set = w.sets == 2 ? c : 0;
        if (k >= w.K || row < 0) continue;
        const float s = Ft16<BF16>::lo(reinterpret_cast<const uint16_t*>(in + 512)[set * 16 + g * 2 + r]);
        const int z = w.zeros ? in[512 + 32 * w.sets + set * 16 + g * 2 + r] : 8;
        uint32_t o[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const uint32_t x = word[2 * c + r] >> (4 * w4_nibble(n));
          o[n] = Ft16<BF16>::rnd(s * (float)((int)(x & 15u) - z)) |
                 (uint32_t)Ft16<BF16>::rnd(s * (float)((int)((x >> 16) & 15u) - z)) << 16;
        }
        *reinterpret_cast<uint4*>(W + (e * w.N + row) * w.K + k) = make_uint4(o[0], o[1], o[2], o[3]);
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
