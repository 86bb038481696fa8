// tc_host.cuh -- host side of the tensor-core GEMMs: tensor maps, the stream-K
// plans, and the launches of the kernels in tc_gemm.cuh, tc2_gemm.cuh,
// ng_gemm.cuh and simt_gemm.cuh, for the translation units that use them.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>
#include <mutex>
#include <utility>

#include "../csrc_serving/host_shared.h"
#include "ng_gemm.cuh"
#include "simt_gemm.cuh"
#include "tc2_gemm.cuh"
#include "tc_gemm.cuh"
#include "tc_plan.h"

namespace swiglu {

constexpr size_t WS_HEADER = 256;  // error word + reserved
constexpr int TC_STAGES = 4;
constexpr int TC_BN = 256;
constexpr int TC2_STAGES = 6;

// Debug builds (SWIGLU_DEBUG): the buffers (base, bytes) a launch may touch
// with plain loads and stores, its output first; the kernels check every
// such access against them.  Release builds carry no windows.
using Win = std::pair<const void*, size_t>;

template <class T>
inline void set_windows(T& args, std::initializer_list<Win> wins) {
#ifdef SWIGLU_DEBUG
  args.dbg = host::windows(wins);
#else
  (void)args;
  (void)wins;
#endif
}

inline SimtCheck simt_check(int* err, std::initializer_list<Win> wins) {
  SimtCheck c;
#ifdef SWIGLU_DEBUG
  c.err = err;
  c.win = host::windows(wins);
#else
  (void)err;
  (void)wins;
#endif
  return c;
}

// ---------------------------------------------------------------------------
// driver entry point for tensor-map encoding (no link-time libcuda dependency)
// ---------------------------------------------------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn get_encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

inline int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

// 2-D tiled map over a row-major matrix [outer][inner] (inner contiguous) with
// a row stride in bytes; 128-byte swizzle unless given; out-of-range elements
// read as 0 (and are not written by a store).
inline bool encode_2d(CUtensorMap* tm, bool bf16, const void* base, uint64_t inner, uint64_t outer,
               uint64_t row_stride_bytes, uint32_t box_inner, uint32_t box_outer,
               CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  EncodeTiledFn enc = get_encode_fn();
  if (enc == nullptr) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {row_stride_bytes};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t estr[2] = {1, 1};
  return enc(tm, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
             const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Wgu [2H][D] seen as [2][H][D]: one box brings rows j0.. of Wg and of Wu
// (depth 2), or of one of them (depth 1: the two CTAs of a pair each bring one).
inline bool encode_gateup(CUtensorMap* tm, bool bf16, const void* Wgu, uint64_t D, uint64_t H,
                   uint32_t rows, uint32_t depth = 2) {
  EncodeTiledFn enc = get_encode_fn();
  if (enc == nullptr) return false;
  cuuint64_t dims[3] = {D, H, 2};
  cuuint64_t strides[2] = {D * 2, H * D * 2};
  cuuint32_t box[3] = {64, rows, depth};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(tm, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
             const_cast<void*>(Wgu), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// K-major operand: rows of K elements, box {64, rows_per_tile}.
inline bool map_kmajor(CUtensorMap* tm, bool bf16, const void* base, int64_t K, int64_t rows, int64_t ld,
                uint32_t box_rows) {
  return encode_2d(tm, bf16, base, (uint64_t)K, (uint64_t)rows, (uint64_t)ld * 2, 64, box_rows);
}

// MN-major operand stored [K][MN]: boxes {64 MN, 64 K}.
inline bool map_mnmajor(CUtensorMap* tm, bool bf16, const void* base, int64_t MN, int64_t K, int64_t ld) {
  return encode_2d(tm, bf16, base, (uint64_t)MN, (uint64_t)K, (uint64_t)ld * 2, 64, 64);
}

// ---------------------------------------------------------------------------
// stream-K hybrid for the tensor-core kernels
// ---------------------------------------------------------------------------
// Workspace of a training call: [0, 256) header (error word), then the
// shared-tile counters, then the fp32 partial tiles.
constexpr size_t TC_SK_COUNTER_BYTES = 1024;  // up to 256 shared tiles
constexpr int TC_SK_MAX_SMS = 256;

// Workspace bytes left for stream-K partial tiles after the header and the
// tile counters.
inline size_t part_capacity(size_t ws_bytes) {
  const size_t fixed = WS_HEADER + TC_SK_COUNTER_BYTES;
  return ws_bytes > fixed ? ws_bytes - fixed : 0;
}

inline size_t tc_part_bytes(const TcPlan& p, int64_t bn = TC_BN) {
  return p.sk_tiles ? (size_t)p.grid * p.seg_max * TC_BM * bn * 4 : 0;
}

// 512-column pair tiles for the weight-gradient and dX GEMMs (use_wide)
constexpr int TC2_WIDE_BN = 512;
constexpr int64_t TC2_WIDE_MIN_K = 16384;

inline int tc_nsm() {
  const int n = sm_count();
  return n < 1 ? 1 : (n > TC_SK_MAX_SMS ? TC_SK_MAX_SMS : n);
}

// 512-column pair tiles (one accumulator, no epilogue overlap) for an
// M x N GEMM over K: by size, where the main loop dwarfs a tile's epilogue
// (K >= 16384) and every pair gets at least two whole tiles.  Measured at
// B=8 S=8192 D=4096 H=11008: dWd 3.74 -> 3.61, dWgu 7.46 -> 6.96, dX 7.17
// -> 6.88 ms; at S=4096 D=2048 H=5632 dWgu 0.975 -> 0.897 ms, while dX
// (K = 11264) and dWd (88 tiles for 76 pairs) were slower, which the rule
// leaves on 256-column tiles.
inline bool use_wide(bool pairs, int64_t M, int64_t N, int64_t K) {
  const int mode = host::wide_tiles();
  if (!pairs || mode == 0) return false;
  if (mode == 2) return true;
  const int64_t tiles = ((M + TC2_BM - 1) / TC2_BM) * ((N + TC2_WIDE_BN - 1) / TC2_WIDE_BN);
  return K >= TC2_WIDE_MIN_K && tiles >= 2 * (int64_t)host::pair_units();
}

// Whether one GEMM runs on SM pairs.  Measured per kernel on GB300: pairs
// win when the main loop dominates -- long K and several rounds of tiles, or
// the very long K of the weight gradients -- while short-K GEMMs with heavy
// epilogues or few tiles run faster on single SMs (the pair's fixed costs and
// its coupled epilogues are not amortised).
inline bool use_pairs(int64_t Mg, int64_t N, int64_t n_per_tile, int64_t K) {
  const int mode = host::cta_pairs();
  if (mode == 0 || host::pair_units() < 1) return false;
  if (mode == 2) return true;
  // pairs once every pair gets at least one of their 256-row tiles and the
  // 256-row tiles add no padding beyond the 128-row ones; measured per GEMM
  // at B=8, S=2048-8192 (D = 1024-4096): as fast or faster on pairs for
  // every GEMM there, including the short contractions (gate/up and dX at
  // D = 1024: 0.151 vs 0.171 and 0.126 vs 0.143 ms); no-grad calls with
  // 65-128 or 384 tokens, whose pair tiles would be partly empty, are 3% and
  // 11% faster on single SMs
  const int64_t pair_tiles = ((Mg + TC2_BM - 1) / TC2_BM) * ((N + n_per_tile - 1) / n_per_tile);
  const bool no_pad = (Mg + TC2_BM - 1) / TC2_BM * TC2_BM == (Mg + TC_BM - 1) / TC_BM * TC_BM;
  const int64_t kb = (K + TC_BK - 1) / TC_BK;
  return (kb >= 16 && no_pad && pair_tiles >= (int64_t)host::pair_units()) || kb >= 256;
}

// part_cap: workspace bytes available for stream-K partial tiles; a GEMM
// whose plan needs more runs whole tiles only (same results within
// rounding, without the last round's balancing).
// units: CTAs or pairs to plan for, 0 for all that the device holds.
inline TcShape make_shape(int64_t M, int64_t N, int64_t K, int64_t n_per_tile, int* err, bool pairs,
                   size_t part_cap, int units = 0) {
  TcShape s;
  s.M = (int)M;
  s.N = (int)N;
  s.K = (int)K;
  const int64_t bm = pairs ? TC2_BM : TC_BM;
  s.m_tiles = (int)((M + bm - 1) / bm);
  s.n_tiles = (int)((N + n_per_tile - 1) / n_per_tile);
  s.k_blocks = (int)((K + TC_BK - 1) / TC_BK);
  s.group_m = 16;
  s.wait_limit_ns = host::wait_limit_ns();
  s.err = err;
  s.inject_stall = host::take_stall() ? 1 : 0;
  // the workspace (whose first word is err) carries the stream-K scratch
  s.early = s.clear_err = 0;
  s.units = units > 0 ? units : pairs ? host::pair_units() : tc_nsm();
  const TcPlan p = tc_plan((int64_t)s.m_tiles * s.n_tiles, s.k_blocks, s.units);
  s.sk_tiles = p.sk_tiles;
  s.seg_max = p.seg_max;
  if (tc_part_bytes(p, n_per_tile) * (pairs ? 2 : 1) > part_cap) {
    s.sk_tiles = 0;
    s.seg_max = 1;
  }
  s.counters = reinterpret_cast<int*>(reinterpret_cast<char*>(err) + WS_HEADER);
  s.part = reinterpret_cast<float*>(reinterpret_cast<char*>(err) + WS_HEADER + TC_SK_COUNTER_BYTES);
  return s;
}

// CTAs (or pairs) to launch: the stream-K plan's grid, or one per tile up to
// s.units when the GEMM runs whole tiles only.
inline int launch_units(const TcShape& s) {
  const int64_t tiles = (int64_t)s.m_tiles * s.n_tiles;
  if (s.sk_tiles) return tc_plan(tiles, s.k_blocks, s.units).grid;
  return (int)(tiles < s.units ? tiles : s.units);
}

// The same for a GEMM of a linear layer, shared or not by what it costs.  A shared
// tile's partial sums (128 KB a CTA) go out and come back, the last CTA of a tile
// reading everyone's; a k-block takes 0.34 us.  Measured at 16384 x 2816 x 1024 on
// pairs (whole tiles, shared ones): forward, 16 k-blocks, 9.26 rounds: 86 and 109
// us; dX, 44 k-blocks, 3.37 rounds: 67 and 77; dW, 256 k-blocks, 0.58 rounds: 87
// and 77; 32768 x 2048 x 5632: dW, 512 k-blocks, 2.3 rounds: 499 and 455.  So the
// last round is shared where it leaves 74 k-blocks' time of every CTA idle, and
// fewer tiles than CTAs go to as many CTAs each as makes their parts, and the
// reading of them (about 8 k-blocks each), shortest together.
inline TcShape linear_plan(int64_t M, int64_t N, int64_t K, int64_t n_per_tile, int* err, bool pairs,
                           size_t part_cap) {
  const int all = pairs ? host::pair_units() : tc_nsm();
  const int64_t bm = pairs ? TC2_BM : TC_BM, kb = (K + TC_BK - 1) / TC_BK;
  const int64_t tiles = ((M + bm - 1) / bm) * ((N + n_per_tile - 1) / n_per_tile);
  if (tiles >= all) {
    const int64_t idle = (all - tiles % all) % all;  // CTAs without a tile in the last round
    return make_shape(M, N, K, n_per_tile, err, pairs, idle * kb >= 74 * (int64_t)all ? part_cap : 0);
  }
  int64_t best = kb, units = tiles;
  for (int64_t s = 2; (s - 1) * tiles < all; ++s) {
    // (parts that are no whole share of a tile give it one more reader's sums to read)
    const bool even = s * tiles <= all;
    const int64_t u = even ? s * tiles : all, cost = kb * tiles / u + 18 + 8 * (even ? s : s + 1);
    if (cost < best) {
      best = cost;
      units = u;
    }
  }
  return make_shape(M, N, K, n_per_tile, err, pairs, units > tiles ? part_cap : 0, (int)units);
}
// first: the first kernel of its call.
inline TcShape linear_shape(int64_t M, int64_t N, int64_t K, int64_t n_per_tile, int* err, bool pairs,
                            size_t part_cap, bool first) {
  TcShape s = linear_plan(M, N, K, n_per_tile, err, pairs, part_cap);
  s.early = 1;
  s.clear_err = first ? 1 : 0;
  return s;
}

// The training kernels are launched in plain stream order (the linear layers'
// set s.early): with a static round-robin tile split, a programmatic dependent whose CTAs start late on
// SMs still held by the predecessor's last wave also finishes late (measured
// slower than plain order).
template <int AM, int BMODE, bool BF16, class Epi>
cudaError_t launch_tc(int kid, const CUtensorMap& ta, const CUtensorMap& tb, const TcShape& s,
                      const typename Epi::Params& ep, cudaStream_t st) {
  auto kern = tc_gemm_kernel<TC_BN, TC_STAGES, AM, BMODE, BF16, Epi>;
  constexpr int smem = TcSmem<TC_BN, TC_STAGES>::DYN_BYTES;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int grid = launch_units(s);
  host::Prof prof(kid, st);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(TC_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = s.early && !host::profiling() ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kern, ta, tb, s, ep);
  host::count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

// The pair kernel: clusters of two CTAs on the two SMs of a TPC.
// tg, tu: the TMA dG/dU epilogue's maps of G and U (other epilogues: unused)
template <int AM, int BMODE, bool BF16, class Epi, int BN = TC2_BN>
cudaError_t launch_tc2(int kid, const CUtensorMap& ta, const CUtensorMap& tb, const TcShape& s,
                       const typename Epi::Params& ep, cudaStream_t st,
                       const CUtensorMap* tg = nullptr, const CUtensorMap* tu = nullptr) {
  // the TMA dG/dU epilogue's slots (GU_SLOTS x 4 KB per epilogue warp) take
  // the room of GU_SLOTS - 1 ring stages; 512-column tiles (48 KB stages)
  // keep four
  constexpr bool gu = epi_tma_gu<Epi>::value;
  constexpr int stages = BN > 256 ? 4 : (gu ? TC2_STAGES + 1 - GU_SLOTS : TC2_STAGES);
  auto kern = tc2_gemm_kernel<stages, AM, BMODE, BF16, Epi, BN>;
  constexpr int smem = Tc2Smem<stages, gu, BN>::DYN_BYTES;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int units = launch_units(s);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * units));
  cfg.blockDim = dim3(TC_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = s.early && !host::profiling() ? 2 : 1;
  host::Prof prof(kid, st);
  e = cudaLaunchKernelEx(&cfg, kern, ta, tb, s, ep, tg != nullptr ? *tg : ta,
                         tu != nullptr ? *tu : tb);
  host::count_launch();
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

template <int AM, int BMODE, bool BF16, class Epi>
cudaError_t launch_gemm(bool pairs, int kid, const CUtensorMap& ta, const CUtensorMap& tb,
                        const TcShape& s, const typename Epi::Params& ep, cudaStream_t st) {
  return pairs ? launch_tc2<AM, BMODE, BF16, Epi>(kid, ta, tb, s, ep, st)
               : launch_tc<AM, BMODE, BF16, Epi>(kid, ta, tb, s, ep, st);
}

template <bool DUAL, class Epi>
cudaError_t launch_simt(int kid, SimtOperand A, SimtOperand B, SimtOperand B2, int64_t M,
                        int64_t N, int64_t K, const Epi& epi, const SimtCheck& chk,
                        cudaStream_t st) {
  dim3 grid((unsigned)((N + SG_BN - 1) / SG_BN), (unsigned)((M + SG_BM - 1) / SG_BM));
  host::Prof prof(kid, st);
  simt_gemm_kernel<DUAL, Epi>
      <<<grid, SG_THREADS, 0, st>>>(A, B, B2, (int)M, (int)N, (int)K, epi, chk);
  host::count_launch();
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// few-token kernels
// ---------------------------------------------------------------------------
constexpr int NG_MAX_M = 64;
constexpr int NG_MAX_CTAS = 256;  // stream-K CTAs per launch (one per SM, capped)

// CTAs, stream-K tiles and partial slots per CTA of one GEMM over at most
// `grid` CTAs.  With tiles >= CTAs, all but (tiles mod CTAs) tiles are taken
// whole, the same number per CTA; with fewer k-blocks than CTAs to share, the
// count shrinks so that every sharing CTA owns at least one.
inline void ng_split(int tiles, int kb, int grid, int& ctas, int& sk_tiles, int& seg_max) {
  int64_t c = grid < 1 ? 1 : grid;
  sk_tiles = tiles >= c ? (int)(tiles % c) : tiles;
  const int64_t total = (int64_t)sk_tiles * kb;
  if (total > 0 && c > total && tiles < c) c = total;
  ctas = (int)c;
  const int64_t range = total > 0 ? (total + c - 1) / c : 0;
  seg_max = (int)((range + kb - 1) / kb) + 1;
}

inline int ng_max_grid() {
  const int nsm = sm_count();
  return nsm < 1 ? 1 : (nsm < NG_MAX_CTAS ? nsm : NG_MAX_CTAS);
}

inline void ng_grid(int tiles, int kb, int& ctas, int& sk_tiles, int& seg_max) {
  ng_split(tiles, kb, ng_max_grid(), ctas, sk_tiles, seg_max);
}
template <int NT, bool GATE_UP, bool BF16, bool PACKED = false>
cudaError_t launch_ng(int kid, const CUtensorMap& tw, const CUtensorMap& tx, NgArgs a,
                      cudaStream_t st) {
  auto kern = ng_gemm_kernel<NT, GATE_UP, BF16, PACKED>;
  constexpr int smem = NgSmem<NT>::DYN_BYTES;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  int grid = 1;
  ng_grid(a.tiles, a.kb_tile, grid, a.sk_tiles, a.seg_max);
  a.ctas = grid;
  host::Prof prof(kid, st);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(NG_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  // the down kernel overlaps its prologue and weight prefetch with gate/up's tail
  // (per-kernel event timing would serialise the two, so it is not used then)
  const bool pdl = a.dependent && !host::profiling();
  if (!pdl) a.dependent = 0;
  cfg.attrs = pdl ? attr : nullptr;
  cfg.numAttrs = pdl ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kern, tw, tx, a);
  host::count_launch();
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace swiglu
