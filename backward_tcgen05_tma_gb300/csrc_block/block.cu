// block.cu -- C ABI of the operators around an MLP in a transformer block
// (include/swiglu_mlp.h): layer norm, and linear layers with bias, activation
// and residual.  Argument checks, plans and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/swiglu_mlp.h"
#include "../csrc/tc_host.cuh"
#include "column_sums.cuh"
#include "layer_norm.cuh"
#include "linear_epi.cuh"
#include "linear_few.cuh"
#include "linear_mid.cuh"
#include "simt_linear.cuh"
#include "simt_plan.h"

using namespace swiglu;

namespace {

constexpr int64_t LN_MAX_D = 16384;            // a row fits the registers of a block
constexpr int64_t MAX_ROWS = 0x7fffffffLL - 256;  // the kernels' 32-bit row and column indexes
constexpr size_t FIXED = WS_HEADER + TC_SK_COUNTER_BYTES;  // error word and counters of shared tiles
static_assert(TC_SK_MAX_SMS * 4 <= TC_SK_COUNTER_BYTES, "fewer tiles are shared than there are SMs to share them");

swiglu_status status_of(cudaError_t e) { return e == cudaSuccess ? SWIGLU_OK : SWIGLU_ERR_CUDA; }

size_t bytes_of(swiglu_dtype dt) { return dt == SWIGLU_F32_IEEE ? 4 : 2; }

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// Needed pointers are not null; all of them, given or null, are aligned.
swiglu_status check_ptrs(std::initializer_list<const void*> needed,
                         std::initializer_list<const void*> optional = {}) {
  for (const void* p : needed)
    if (p == nullptr) return SWIGLU_ERR_INVALID_ARG;
  for (const void* p : needed)
    if (misaligned(p)) return SWIGLU_ERR_ALIGNMENT;
  for (const void* p : optional)
    if (misaligned(p)) return SWIGLU_ERR_ALIGNMENT;
  return SWIGLU_OK;
}

swiglu_status check_dtype(swiglu_dtype dt) {
  return dt == SWIGLU_BF16 || dt == SWIGLU_F16 || dt == SWIGLU_F32_IEEE ? SWIGLU_OK
                                                                        : SWIGLU_ERR_INVALID_ARG;
}

swiglu_status check_ws(const void* ws, size_t bytes, size_t need) {
  if (ws == nullptr || bytes < need) return SWIGLU_ERR_WORKSPACE;
  return misaligned(ws) ? SWIGLU_ERR_ALIGNMENT : SWIGLU_OK;
}

int nsm() { return host::sms() > 0 ? host::sms() : 1; }

RowCheck row_check(void* ws, std::initializer_list<Win> wins) {
  RowCheck c;
#ifdef SWIGLU_DEBUG
  c.err = static_cast<int*>(ws);
  c.win = host::windows(wins);
#else
  (void)ws;
  (void)wins;
#endif
  return c;
}

// The dynamic shared memory of a kernel, raised once per device.
template <auto KERNEL>
cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load() & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit);
  return e;
}

// A launch that may start while the kernel before it on the stream ends; the
// kernels wait for it before they touch anything.
template <class... P, class... A>
cudaError_t launch(int id, void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                   A... args) {
  host::Prof prof(id, st);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  // per-kernel event timing would serialise the launches, so no overlap then
  cfg.attrs = attr;
  cfg.numAttrs = host::profiling() ? 0 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  host::count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

// f(a value of the storage type)
template <class F>
auto by_type(swiglu_dtype dt, F f) {
  if (dt == SWIGLU_BF16) return f(__nv_bfloat16{});
  if (dt == SWIGLU_F16) return f(__half{});
  return f(float{});
}

// ---------------------------------------------------------------------------
// layer norm
// ---------------------------------------------------------------------------
swiglu_status check_ln(int64_t M, int64_t D, swiglu_dtype dt) {
  swiglu_status st = check_dtype(dt);
  if (st != SWIGLU_OK) return st;
  if (M < 0 || D <= 0) return SWIGLU_ERR_INVALID_ARG;
  if (D % (16 / (int64_t)bytes_of(dt)) != 0) return SWIGLU_ERR_ALIGNMENT;
  return M > MAX_ROWS || D > LN_MAX_D ? SWIGLU_ERR_UNSUPPORTED : SWIGLU_OK;
}

template <class T>
cudaError_t ln_forward(const LnFwdArgs& a, cudaStream_t st) {
  const int nv = a.D / Vec<T>::N;
  auto rows4 = [&](auto k) { return launch(host::K_LN, k, dim3((unsigned)((a.M + 3) / 4)), 128, 0, st, a); };
  auto row = [&](auto k, int tpr) { return launch(host::K_LN, k, dim3((unsigned)a.M), tpr, 0, st, a); };
  if (nv <= 32) return rows4(ln_fwd_kernel<T, 32, 1, 4>);
  if (nv <= 64) return rows4(ln_fwd_kernel<T, 32, 2, 4>);
  if (nv <= 128) return rows4(ln_fwd_kernel<T, 32, 4, 4>);
  if (nv <= 256) return row(ln_fwd_kernel<T, 128, 2, 1>, 128);
  if (nv <= 512) return row(ln_fwd_kernel<T, 128, 4, 1>, 128);
  if (nv <= 1024) return row(ln_fwd_kernel<T, 256, 4, 1>, 256);
  if (nv <= 2048) return row(ln_fwd_kernel<T, 512, 4, 1>, 512);
  return row(ln_fwd_kernel<T, 1024, 4, 1>, 1024);
}

// Threads of a row in the backward pass: four vectors each as far as a block has
// threads for it.
int lnb_tpr(int nv) {
  int t = 32;
  while (t < LNB_THREADS && t * 4 < nv) t *= 2;
  return t;
}
int lnb_grid(int64_t M, int64_t D, swiglu_dtype dt) {
  const int groups = LNB_THREADS / lnb_tpr((int)(D * (int64_t)bytes_of(dt) / 16));
  return (int)std::min<int64_t>((M + groups - 1) / groups, nsm());
}
size_t ln_part_bytes(int64_t M, int64_t D, swiglu_dtype dt) {
  return (size_t)lnb_grid(M, D, dt) * 2 * D * 4;
}

constexpr int LNB_SMEM = 200 * 1024;

template <class T, int TPR, int VPT, bool DS>
cudaError_t ln_backward(LnBwdArgs a, int grid, cudaStream_t st) {
  constexpr auto kern = ln_bwd_kernel<T, TPR, VPT, DS>;
  constexpr int stage = (DS ? 3 : 2) * VPT * LNB_THREADS * 16;
  a.stages = std::min(5, LNB_SMEM / stage);
  // the ring, and then the groups' sums in its place
  constexpr int groups = LNB_THREADS / TPR, n = Vec<T>::N;
  const int smem = std::max(a.stages * stage, groups * 2 * (a.D + 4 * n) * 4);
  const cudaError_t e = allow_smem<kern>(LNB_SMEM);
  if (e != cudaSuccess) return e;
  return launch(host::K_DLN, kern, dim3((unsigned)grid), LNB_THREADS, (size_t)smem, st, a);
}

template <class T, int TPR, int VPT>
cudaError_t ln_backward(const LnBwdArgs& a, int grid, cudaStream_t st) {
  return a.ds != nullptr ? ln_backward<T, TPR, VPT, true>(a, grid, st)
                         : ln_backward<T, TPR, VPT, false>(a, grid, st);
}

template <class T>
cudaError_t ln_backward(const LnBwdArgs& a, int grid, cudaStream_t st) {
  const int nv = a.D / Vec<T>::N;
  if (nv <= 32) return ln_backward<T, 32, 1>(a, grid, st);
  if (nv <= 64) return ln_backward<T, 32, 2>(a, grid, st);
  switch (lnb_tpr(nv)) {
    case 32: return ln_backward<T, 32, 4>(a, grid, st);
    case 64: return ln_backward<T, 64, 4>(a, grid, st);
    case 128: return ln_backward<T, 128, 4>(a, grid, st);
    case 256: return ln_backward<T, 256, 4>(a, grid, st);
  }
  if (nv <= 2048) return ln_backward<T, 512, 4>(a, grid, st);
  if constexpr (sizeof(T) == 4) return ln_backward<T, 512, 8>(a, grid, st);
  return cudaErrorInvalidConfiguration;
}

// out0, out1 = sums of the parts' columns [0, n) and [n, cols)
cudaError_t column_sums(const float* part, int parts, int cols, void* out0, void* out1, int n, int add,
                        swiglu_dtype dt, void* ws, size_t ws_bytes, cudaStream_t st) {
  ColumnSumArgs a = {part, out0, out1, parts, cols, n, add, {}};
  const size_t e = bytes_of(dt);
  a.chk = row_check(ws, {{out0 != nullptr ? out0 : out1, (size_t)n * e}, {out1, out1 ? (size_t)(cols - n) * e : 0},
                         {ws, ws_bytes}});
  const dim3 grid((unsigned)((cols + CS_COLS - 1) / CS_COLS));
  return by_type(dt, [&](auto t) {
    return launch(host::K_COLUMN_SUMS, column_sum_kernel<decltype(t)>, grid, 256, 0, st, a);
  });
}

// ---------------------------------------------------------------------------
// linear
// ---------------------------------------------------------------------------
// 16-bit products that linear_mid_kernel takes (fewer tokens: the streaming form where
// it fits), those of some size only while they have too few tiles of 256 x 256 for the
// pairs of SMs.  Measured in us, this form first, the GEMM of large tiles after it:
// 11008 x 4096 128 tokens 22, 35, 512 tokens 38, 48, 768 tokens 57, 48; 4096 x 11008
// 768 tokens 56, 81; 32768 x 4096 256 tokens 63, 56; 2816 x 1024 128 tokens 7.5, 14.2,
// 1024 tokens 10.5, 14.2.
bool mid_tokens(int64_t M, int64_t N, int64_t K) {
  if (M <= 64) return true;
  if (host::cta_pairs() == 2) return false;  // pairs asked for, whatever the size
  return M <= 1024 && ((double)M * N * K < 0x1p35 || (M + 255) / 256 * ((N + 255) / 256) < nsm() / 2);
}

swiglu_status check_linear(int64_t M, int64_t N, int64_t K, int act, swiglu_dtype dt) {
  swiglu_status st = check_dtype(dt);
  if (st != SWIGLU_OK) return st;
  if (M < 0 || N <= 0 || K <= 0 || act < SWIGLU_ACT_NONE || act > SWIGLU_ACT_SILU)
    return SWIGLU_ERR_INVALID_ARG;
  const int64_t unit = 16 / (int64_t)bytes_of(dt);
  if (N % unit != 0 || K % unit != 0) return SWIGLU_ERR_ALIGNMENT;
  if (M > MAX_ROWS || N > MAX_ROWS || K > MAX_ROWS) return SWIGLU_ERR_UNSUPPORTED;
  // tiles (of 64 x 64 at least) are counted in 32 bits
  auto tiles = [](int64_t a, int64_t b) { return ((a + 63) / 64) * ((b + 63) / 64); };
  return std::max({tiles(M, N), tiles(M, K), tiles(N, K)}) > 0x7fffffffLL ? SWIGLU_ERR_UNSUPPORTED
                                                                         : SWIGLU_OK;
}

// Partial-tile bytes of one GEMM [Mg, N] over K on the tensor cores, either
// form; without a device the bound for any GPU of up to 256 SMs.
size_t gemm_part_bytes(int64_t Mg, int64_t N, int64_t K, bool may_be_wide) {
  if (host::sms() < 1) return (size_t)2 * TC_SK_MAX_SMS * TC_BM * (may_be_wide ? TC2_WIDE_BN : TC_BN) * 4;
  const int64_t kb = (K + TC_BK - 1) / TC_BK, nt = (N + TC_BN - 1) / TC_BN, rows2 = (Mg + TC2_BM - 1) / TC2_BM;
  const int units = host::pair_units();
  size_t best = tc_part_bytes(tc_plan(((Mg + TC_BM - 1) / TC_BM) * nt, kb, tc_nsm()));
  if (units >= 1) {
    best = std::max(best, 2 * tc_part_bytes(tc_plan(rows2 * nt, kb, units)));
    if (may_be_wide)
      best = std::max(best, 2 * tc_part_bytes(tc_plan(rows2 * ((N + TC2_WIDE_BN - 1) / TC2_WIDE_BN), kb, units),
                                              TC2_WIDE_BN));
  }
  return best;
}

// Parts of the rows whose column sums are taken apart, in the pass over dY:
// about four blocks on each SM.
int dact_parts(int64_t M, int64_t N, swiglu_dtype dt) {
  const int64_t strips = (N * (int64_t)bytes_of(dt) + 511) / 512;
  const int64_t most = (M + 2 * DA_WARPS - 1) / (2 * DA_WARPS);
  const int64_t want = (4 * (int64_t)(host::sms() > 0 ? host::sms() : TC_SK_MAX_SMS) + strips - 1) / strips;
  return (int)std::max<int64_t>(1, std::min(want, most));
}

size_t sl_bytes(int64_t M, int64_t N, int64_t K) {
  if (host::sms() < 1) return (size_t)8 * TC_SK_MAX_SMS * 128 * SL_BN * 4;
  const SlPlan p = sl_plan(M, N, K, nsm());
  return (size_t)p.split() * p.parts * 16 * p.tm * SL_BN * 4;
}

size_t linear_bwd_bytes(int64_t M, int64_t N, int64_t K, swiglu_dtype dt) {
  size_t n = (size_t)dact_parts(M, N, dt) * N * 4;
  if (dt == SWIGLU_F32_IEEE) {
    n = std::max({n, sl_bytes(N, K, M), sl_bytes(M, K, N)});
  } else {
    n = std::max(n, gemm_part_bytes(N, K, M, true));
    n = std::max(n, gemm_part_bytes(M, K, N, true));
  }
  return FIXED + n;
}

// Clusters of `split` blocks of a kernel that fit the device at once, kept per
// device and size.
template <auto KERNEL>
int few_clusters(int split) {
  static std::atomic<int> known[64][4];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
  std::atomic<int>& at = known[dev][split == 1 ? 0 : split == 2 ? 1 : split == 4 ? 2 : 3];
  int n = at.load();
  if (n > 0) return n;
  n = nsm() / split;
  if (split > 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(n * split));
    cfg.blockDim = dim3(LF_THREADS);
    cfg.dynamicSmemBytes = LF_SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)split, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int q = 0;
    if (cudaOccupancyMaxActiveClusters(&q, KERNEL, &cfg) == cudaSuccess && q > 0) n = std::min(n, q);
    cudaGetLastError();  // a failed query is not an error of the call
  }
  at.store(n = std::max(n, 1));
  return n;
}

struct StreamPlan {
  int nt, blocks, halves, xstride, recv_off, smem;
  bool fits;
};
// Up to 16 tokens.  Clusters of 4 blocks, whose warps in pairs split the contraction 8
// ways, as they reach every SM (38 clusters; of 8 blocks 15 fit, 120 SMs); of 8 where a
// quarter of the token rows does not fit a block, and linear_mid.cuh's form where an
// eighth does not.  Measured in us, this form first, 8 and 16 tokens:
//   11008 x 4096   20.0, 23.0   20.8, 20.5
//   4096 x 4096    10.4, 11.0   10.8, 10.8
//   2816 x 1024     5.6, 5.9     5.7, 5.9
// (at 32 tokens 23.6, 19.7 and 12.1, 10.3: it is for 16 at most)
StreamPlan stream_plan(int64_t M, int64_t N, int64_t K) {
  StreamPlan p = {};
  if (M > LF_MAX_M) return p;
  p.nt = M <= 8 ? 1 : 2;
  const int64_t nk = (K + 31) / 32;
  int parts = LF_MAX_PARTS;
  while (parts > nk) parts /= 2;
  for (p.blocks = std::min(parts, 4); p.blocks <= parts; p.blocks *= 2) {
    p.halves = parts / p.blocks;
    const int64_t per = (nk + p.blocks - 1) / p.blocks;
    // rows an odd number of 64 bytes apart: 8 lanes' 16-byte reads of two rows meet no bank twice
    const int64_t xs = (per | 1) * 64, bytes = M * xs + (int64_t)LF_WARPS * 2 * lf_recv(p.nt, parts);
    if (bytes > LF_SMEM) continue;
    p.fits = true;
    p.xstride = (int)xs;
    p.recv_off = (int)(M * xs);
    p.smem = (int)bytes;
    break;
  }
  return p;
}

template <bool BF16, int NT>
cudaError_t linear_stream(const StreamPlan& p, LfArgs a, cudaStream_t st) {
  constexpr auto kern = linear_few_kernel<BF16, NT>;
  cudaError_t e = allow_smem<kern>(LF_SMEM);
  if (e != cudaSuccess) return e;
  a.blocks = p.blocks;
  a.halves = p.halves;
  a.xstride = p.xstride;
  a.recv_off = p.recv_off;
  a.units = (a.N + 15) / 16;
  const int groups = LF_WARPS / p.halves;
  a.clusters = std::min(few_clusters<kern>(p.blocks), (a.units + groups - 1) / groups);
  a.inject = host::take_stall() ? 1 : 0;
  host::Prof prof(host::K_LINEAR_FEW, st);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.clusters * p.blocks));
  cfg.blockDim = dim3(LF_THREADS);
  cfg.dynamicSmemBytes = (size_t)p.smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int n = 0;
  // per-kernel event timing would serialise the launches, so no overlap then
  if (!host::profiling()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (p.blocks > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n++].val.clusterDim = {(unsigned)p.blocks, 1, 1};
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  e = cudaLaunchKernelEx(&cfg, kern, a);
  host::count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

// How linear_mid_kernel takes a product: weight rows of a tile, blocks of a cluster
// and the ring of a block (two blocks an SM, or one with a larger ring), by the
// least of a time's estimate in us.
struct MidPlan {
  int bn, split, stages, ring, smem;
};
MidPlan mid_plan_of(int mt, int64_t M, int64_t N, int64_t K) {
  MidPlan best = {};
  double least = 1e300;
  const int64_t kb = (K + TC_BK - 1) / TC_BK, m_tiles = (M + mt - 1) / mt;
  const double hbm = (double)(N * K + M * K + M * N) * 2 / 6.4e6;
  for (int two = 1; two >= 0; --two)
    for (int split = 1; split <= 4 && split <= kb; split *= 2)
      for (int bn = 16 * split; bn <= 256 && (bn < N + 16 || bn == 16 * split); bn += 16) {
        const int stages = std::min<int>(LM_MAX_STAGES, (two ? 108 : 200) * 1024 / ((mt + bn) * 128));
        const int each = (bn / 16 + split - 1) / split;
        const int ring = std::max(lm_ring(mt, bn, stages), split > 1 ? split * each * 8192 : 0);
        const int smem = ring + LM_BARS + 1024;
        if (stages < 3 || smem > (two ? 113 : 227) * 1024) continue;
        // clusters of 4 do not reach every SM
        const double sms = (split == 4 ? 0.85 : 1.0) * nsm();
        const double blocks = (double)(m_tiles * ((N + bn - 1) / bn) * split);
        const double steps = (double)((kb + split - 1) / split), kbytes = (mt + bn) * 0.125;
        // a block takes a step of k in 0.28 us or more, an SM 140 KB a us
        const double rounds = std::ceil(blocks / ((two ? 2 : 1) * sms));
        const double chain = rounds * steps * std::max(0.28, kbytes / (two ? 75 : 115));
        const double sm = std::ceil(blocks / sms) * steps * kbytes / 140;
        double t = std::max(hbm, std::max(chain, sm)) + (rounds - 1) * (two ? 4 : 5) + 0.25 * each;
        if (split > 1) t += 1.5 + (double)mt * bn * (two ? 8 : 4) / 6e4;  // the parts' way through DSMEM
        if (t < least) {
          least = t;
          best = {bn, split, stages, ring, smem};
        }
      }
  return best;
}

// The same for sizes that this thread asked for lately: 7 us of a call's host time.
MidPlan mid_plan(int mt, int64_t M, int64_t N, int64_t K) {
  struct Known {
    int64_t M, N, K;
    int mt, sms;
    MidPlan plan;
  };
  static thread_local Known known[32] = {};
  Known& k = known[(uint64_t)(M * 7 + N * 31 + K * 13) / 8 % 32];
  if (k.M != M || k.N != N || k.K != K || k.mt != mt || k.sms != nsm()) k = {M, N, K, mt, nsm(), mid_plan_of(mt, M, N, K)};
  return k.plan;
}

template <bool BF16, int MT>
cudaError_t linear_mid(const void* X, const void* W, LmArgs a, int64_t K, cudaStream_t st) {
  constexpr auto kern = linear_mid_kernel<BF16, MT>;
  cudaError_t e = allow_smem<kern>(227 * 1024);
  if (e != cudaSuccess) return e;
  const MidPlan p = mid_plan(MT, a.M, a.N, K);
  a.kb = (int)((K + TC_BK - 1) / TC_BK);
  a.m_tiles = (a.M + MT - 1) / MT;
  a.split = p.split;
  a.bn = p.bn;
  a.stages = p.stages;
  a.ring = p.ring;
  a.x_rows = a.m_tiles > 1 ? MT : std::min((a.M + 7) / 8 * 8, MT);
  a.inject = host::take_stall() ? 1 : 0;
  CUtensorMap tx, tw;
  if (!map_kmajor(&tx, BF16, X, K, a.M, K, a.x_rows) || !map_kmajor(&tw, BF16, W, K, a.N, K, p.bn))
    return cudaErrorInvalidValue;
  host::Prof prof(host::K_LINEAR_FEW, st);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.m_tiles * ((a.N + p.bn - 1) / p.bn) * p.split));
  cfg.blockDim = dim3(LM_THREADS);
  cfg.dynamicSmemBytes = (size_t)p.smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int n = 0;
  // per-kernel event timing would serialise the launches, so no overlap then
  if (!host::profiling()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (p.split > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n++].val.clusterDim = {(unsigned)p.split, 1, 1};
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  e = cudaLaunchKernelEx(&cfg, kern, tx, tw, a);
  host::count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool BF16>
cudaError_t linear_forward(const void* X, const void* W, const EpiLinear::Params& ep, int64_t M, int64_t N,
                           int64_t K, int* err, size_t ws_bytes, cudaStream_t st) {
  const Win y{ep.y, (size_t)(M * N * 2)}, z{ep.z, ep.z ? (size_t)(M * N * 2) : 0},
      res{ep.res, ep.res ? (size_t)(M * N * 2) : 0}, bias{ep.bias, ep.bias ? (size_t)N * 2 : 0}, w{err, ws_bytes};
  const StreamPlan sp = stream_plan(M, N, K);
  if (sp.fits) {
    LfArgs a = {};
    a.X = static_cast<const uint8_t*>(X);
    a.W = static_cast<const uint8_t*>(W);
    a.bias = static_cast<const uint8_t*>(ep.bias);
    a.res = static_cast<const uint8_t*>(ep.res);
    a.z = static_cast<uint8_t*>(ep.z);
    a.y = static_cast<uint8_t*>(ep.y);
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.act = ep.act;
    a.wait_limit_ns = host::wait_limit_ns();
    a.err = err;
    set_windows(a, {y, w, z, res, bias, {X, (size_t)(M * K * 2)}, {W, (size_t)(N * K * 2)}});
    return sp.nt == 1 ? linear_stream<BF16, 1>(sp, a, st) : linear_stream<BF16, 2>(sp, a, st);
  }
  if (mid_tokens(M, N, K)) {
    LmArgs a = {};
    a.M = (int)M;
    a.N = (int)N;
    a.bias = static_cast<const uint8_t*>(ep.bias);
    a.res = static_cast<const uint8_t*>(ep.res);
    a.z = static_cast<uint8_t*>(ep.z);
    a.y = static_cast<uint8_t*>(ep.y);
    a.act = ep.act;
    a.wait_limit_ns = host::wait_limit_ns();
    a.err = err;
    set_windows(a, {y, w, z, res, bias});
    return M <= 64 ? linear_mid<BF16, 64>(X, W, a, K, st) : linear_mid<BF16, 128>(X, W, a, K, st);
  }
  const bool pairs = use_pairs(M, N, TC_BN, K);
  CUtensorMap tx, tw;
  if (!map_kmajor(&tx, BF16, X, K, M, K, TC_BM) || !map_kmajor(&tw, BF16, W, K, N, K, pairs ? 128 : TC_BN))
    return cudaErrorInvalidValue;
  TcShape s = linear_shape(M, N, K, TC_BN, err, pairs, part_capacity(ws_bytes), true);
  set_windows(s, {y, w, z, res, bias});
  const auto whole = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 31u) == 0; };
  if (N % 16 == 0 && whole(ep.y) && whole(ep.z) && whole(ep.res))
    return launch_gemm<LOAD_KMAJOR, LOAD_KMAJOR, BF16, EpiLinearSectors>(pairs, host::K_LINEAR, tx, tw, s, ep, st);
  return launch_gemm<LOAD_KMAJOR, LOAD_KMAJOR, BF16, EpiLinear>(pairs, host::K_LINEAR, tx, tw, s, ep, st);
}

// dX = rnd(G W act'(Xpre)), G [M, N], W [N, K]
template <bool BF16>
cudaError_t linear_dx(const void* G, const void* W, const EpiDAct::Params& ep, int64_t M, int64_t N,
                      int64_t K, int* err, size_t ws_bytes, bool first, cudaStream_t st) {
  const bool pairs = use_pairs(M, K, TC_BN, N);
  CUtensorMap tg, tw;
  if (!map_kmajor(&tg, BF16, G, N, M, N, TC_BM) || !map_mnmajor(&tw, BF16, W, K, N, K))
    return cudaErrorInvalidValue;
  TcShape s = linear_shape(M, K, N, TC_BN, err, pairs, part_capacity(ws_bytes), first);
  set_windows(s, {{ep.out, (size_t)(M * K * 2)}, {err, ws_bytes}, {ep.pre, (size_t)(M * K * 2)}});
  return launch_gemm<LOAD_KMAJOR, LOAD_MNMAJOR, BF16, EpiDAct>(pairs, host::K_LINEAR_DX, tg, tw, s, ep, st);
}

template <class Epi>
cudaError_t simt_rows(int id, const SlArgs& a, const Epi& epi, cudaStream_t st) {
  host::Prof prof(id, st);
  const unsigned n8 = (unsigned)((a.N + 7) / 8), n4 = (unsigned)((a.N + 3) / 4);
  if (a.M == 1)
    simt_rows_kernel<1, Epi><<<n8, SL_THREADS, 0, st>>>(a, epi);
  else if (a.M == 2)
    simt_rows_kernel<2, Epi><<<n8, SL_THREADS, 0, st>>>(a, epi);
  else if (a.M <= 4)
    simt_rows_kernel<4, Epi><<<n8, SL_THREADS, 0, st>>>(a, epi);
  else
    simt_rows_kernel<8, Epi><<<n4, SL_THREADS, 0, st>>>(a, epi);
  host::count_launch();
  return cudaGetLastError();
}

template <bool A_KC, bool B_KC, class Epi>
cudaError_t simt_product(int id, const float* A, int64_t lda, const float* B, int64_t ldb, int64_t M, int64_t N,
                         int64_t K, const Epi& epi, void* ws, bool first, std::initializer_list<Win> wins,
                         cudaStream_t st) {
  const SlPlan p = sl_plan(M, N, K, nsm());
  const int split = p.split();
  SlArgs a = {A, B, lda, ldb, (int)M, (int)N, (int)K, p.m_tiles, p.n_tiles, p.whole, p.parts, p.per,
              reinterpret_cast<float*>(static_cast<char*>(ws) + FIXED), first ? static_cast<int*>(ws) : nullptr, {}};
#ifdef SWIGLU_DEBUG
  // where all tiles are split, the partial sums take the output's place in the first kernel
  Win with[DBG_WINS];
  const int nw = (int)(std::copy(wins.begin(), wins.end(), with) - with);
  with[nw] = Win{a.part, (size_t)split * p.parts * 16 * p.tm * SL_BN * 4};
  if (p.whole == 0 && !(A_KC && B_KC && M <= 8)) std::swap(with[0], with[nw]);
  a.chk.err = static_cast<int*>(ws);
  a.chk.win = host::windows(with, nw + 1);
#else
  (void)wins;
#endif
  if constexpr (A_KC && B_KC) {
    if (M <= 8) return simt_rows(id, a, epi, st);
  }
  const dim3 grid((unsigned)(p.whole + split * p.parts));
  {
    host::Prof prof(id, st);
    if (p.tm == 2)
      simt_linear_kernel<2, A_KC, B_KC, Epi><<<grid, SL_THREADS, 0, st>>>(a, epi);
    else
      simt_linear_kernel<8, A_KC, B_KC, Epi><<<grid, SL_THREADS, 0, st>>>(a, epi);
    host::count_launch();
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || split == 0) return e;
#ifdef SWIGLU_DEBUG
  if (p.whole == 0) std::swap(with[0], with[nw]);
  a.chk.win = host::windows(with, nw + 1);
#endif
  host::Prof prof(id, st);
  const dim3 sums((unsigned)split, (unsigned)(16 * p.tm * SL_BN / 4 / 256));
  if (p.tm == 2)
    simt_sum_kernel<2, Epi><<<sums, 256, 0, st>>>(a, epi);
  else
    simt_sum_kernel<8, Epi><<<sums, 256, 0, st>>>(a, epi);
  host::count_launch();
  return cudaGetLastError();
}

}  // namespace

extern "C" {

swiglu_status swiglu_mlp_layer_norm_fwd(const void* X, const void* residual, const void* weight,
                                        const void* bias, void* S, void* Y, float* mean, float* rstd,
                                        int64_t M, int64_t D, float eps, swiglu_dtype dtype, void* ws,
                                        size_t ws_bytes, void* stream) {
  host::reset_launches();
  swiglu_status st = check_ln(M, D, dtype);
  if (st != SWIGLU_OK) return st;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return SWIGLU_ERR_INVALID_ARG;
  if (ws != nullptr && (st = check_ws(ws, ws_bytes, WS_HEADER)) != SWIGLU_OK) return st;
  if (M == 0) return SWIGLU_OK;
  if ((st = check_ptrs({X, Y}, {residual, weight, bias, S, mean, rstd})) != SWIGLU_OK) return st;
  if ((residual == nullptr) != (S == nullptr)) return SWIGLU_ERR_INVALID_ARG;
  const size_t n = (size_t)(M * D) * bytes_of(dtype), d = (size_t)D * bytes_of(dtype);
  LnFwdArgs a = {X, residual, weight, bias, S, Y, mean, rstd, M, (int)D, eps, {}};
  a.chk = row_check(ws, {{Y, n}, {X, n}, {residual, residual ? n : 0}, {S, S ? n : 0}, {weight, weight ? d : 0}, {bias, bias ? d : 0},
                         {mean, mean ? (size_t)M * 4 : 0}, {rstd, rstd ? (size_t)M * 4 : 0}});
  return status_of(by_type(dtype, [&](auto t) { return ln_forward<decltype(t)>(a, static_cast<cudaStream_t>(stream)); }));
}

size_t swiglu_mlp_layer_norm_workspace_bytes(int64_t M, int64_t D, swiglu_dtype dtype) {
  if (check_ln(M, D, dtype) != SWIGLU_OK) return 0;
  if (host::sms() < 1) return FIXED + (size_t)TC_SK_MAX_SMS * 2 * D * 4;
  return FIXED + ln_part_bytes(M, D, dtype);
}

swiglu_status swiglu_mlp_layer_norm_bwd(const void* dY, const void* S, const void* weight,
                                        const float* mean, const float* rstd, const void* dS, void* dX,
                                        void* dweight, void* dbias, int64_t M, int64_t D, int accumulate,
                                        swiglu_dtype dtype, void* ws, size_t ws_bytes, void* stream) {
  host::reset_launches();
  swiglu_status st = check_ln(M, D, dtype);
  if (st != SWIGLU_OK) return st;
  if (accumulate != 0 && accumulate != 1) return SWIGLU_ERR_INVALID_ARG;
  if ((st = check_ws(ws, ws_bytes, swiglu_mlp_layer_norm_workspace_bytes(M, D, dtype))) != SWIGLU_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t d = (size_t)D * bytes_of(dtype), n = (size_t)M * d;
  if ((st = check_ptrs({}, {weight, dS, dweight, dbias})) != SWIGLU_OK) return st;
  if (M == 0) {  // an empty batch adds nothing
    cudaError_t e = cudaSuccess;
    if (!accumulate && dweight != nullptr) e = cudaMemsetAsync(dweight, 0, d, s);
    if (!accumulate && dbias != nullptr && e == cudaSuccess) e = cudaMemsetAsync(dbias, 0, d, s);
    return status_of(e);
  }
  if ((st = check_ptrs({dY, S, mean, rstd, dX})) != SWIGLU_OK) return st;
  LnBwdArgs a = {};
  a.err = static_cast<int*>(ws);
  a.dy = dY;
  a.s = S;
  a.ds = dS;
  a.w = weight;
  a.mean = mean;
  a.rstd = rstd;
  a.dx = dX;
  a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + FIXED);
  a.M = M;
  a.D = (int)D;
  a.want = dweight != nullptr || dbias != nullptr;
  const int grid = lnb_grid(M, D, dtype);
  a.chk = row_check(ws, {{dX, n}, {ws, ws_bytes}, {dY, n}, {S, n}, {dS, dS ? n : 0}, {weight, weight ? d : 0}, {mean, (size_t)M * 4}, {rstd, (size_t)M * 4}});
  st = status_of(by_type(dtype, [&](auto t) { return ln_backward<decltype(t)>(a, grid, s); }));
  if (st != SWIGLU_OK || !a.want) return st;
  return status_of(column_sums(a.part, grid, 2 * (int)D, dweight, dbias, (int)D, accumulate, dtype, ws, ws_bytes, s));
}

size_t swiglu_mlp_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, swiglu_dtype dtype, int op) {
  if (check_linear(M, N, K, 0, dtype) != SWIGLU_OK || (op != SWIGLU_OP_FWD && op != SWIGLU_OP_BWD)) return 0;
  if (op == SWIGLU_OP_BWD) return linear_bwd_bytes(M, N, K, dtype);
  if (dtype == SWIGLU_F32_IEEE) return FIXED + (M <= 8 ? 0 : sl_bytes(M, N, K));
  if (mid_tokens(M, N, K)) return FIXED;
  return FIXED + gemm_part_bytes(M, N, K, false);
}

swiglu_status swiglu_mlp_linear_fwd(const void* X, const void* W, const void* bias, const void* residual,
                                    void* Z, void* Y, int64_t M, int64_t N, int64_t K,
                                    swiglu_activation act, swiglu_dtype dtype, void* ws, size_t ws_bytes,
                                    void* stream) {
  host::reset_launches();
  swiglu_status st = check_linear(M, N, K, act, dtype);
  if (st != SWIGLU_OK) return st;
  st = check_ws(ws, ws_bytes, swiglu_mlp_linear_workspace_bytes(M, N, K, dtype, SWIGLU_OP_FWD));
  if (st != SWIGLU_OK) return st;
  if (M == 0) return SWIGLU_OK;
  if ((st = check_ptrs({X, W, Y}, {bias, residual, Z})) != SWIGLU_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int* err = static_cast<int*>(ws);
  if (dtype == SWIGLU_F32_IEEE) {
    const SlEpiLinear epi{(const float*)bias, (const float*)residual, (float*)Z, (float*)Y, N, act};
    const size_t mn = (size_t)(M * N * 4);
    return status_of(simt_product<true, true>(
        host::K_SIMT_LINEAR, (const float*)X, K, (const float*)W, K, M, N, K, epi, ws, true,
        {{Y, mn}, {X, (size_t)(M * K * 4)}, {W, (size_t)(N * K * 4)}, {bias, bias ? (size_t)N * 4 : 0},
         {residual, residual ? mn : 0}, {Z, Z ? mn : 0}}, s));
  }
  const EpiLinear::Params ep{bias, residual, Z, Y, N, act};
  return status_of(dtype == SWIGLU_BF16 ? linear_forward<true>(X, W, ep, M, N, K, err, ws_bytes, s)
                                        : linear_forward<false>(X, W, ep, M, N, K, err, ws_bytes, s));
}

swiglu_status swiglu_mlp_linear_bwd(const void* dY, const void* X, const void* W, const void* Z,
                                    swiglu_activation act, const void* X_pre, swiglu_activation x_act,
                                    void* dZ, void* dX, void* dW, void* dbias, int64_t M, int64_t N,
                                    int64_t K, int accumulate, swiglu_dtype dtype, void* ws,
                                    size_t ws_bytes, void* stream) {
  host::reset_launches();
  swiglu_status st = check_linear(M, N, K, act, dtype);
  if (st == SWIGLU_OK) st = check_linear(M, N, K, x_act, dtype);
  if (st != SWIGLU_OK) return st;
  if (accumulate != 0 && accumulate != 1) return SWIGLU_ERR_INVALID_ARG;
  st = check_ws(ws, ws_bytes, swiglu_mlp_linear_workspace_bytes(M, N, K, dtype, SWIGLU_OP_BWD));
  if (st != SWIGLU_OK) return st;
  const int64_t e = (int64_t)bytes_of(dtype);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((st = check_ptrs({}, {Z, X_pre, dZ, dX, dW, dbias})) != SWIGLU_OK) return st;
  if (M == 0) {  // an empty batch adds nothing
    cudaError_t c = cudaSuccess;
    if (!accumulate && dW != nullptr) c = cudaMemsetAsync(dW, 0, (size_t)(N * K * e), s);
    if (!accumulate && dbias != nullptr && c == cudaSuccess) c = cudaMemsetAsync(dbias, 0, (size_t)(N * e), s);
    return status_of(c);
  }
  if ((st = check_ptrs({dY})) != SWIGLU_OK) return st;
  if (act != SWIGLU_ACT_NONE && (st = check_ptrs({Z, dZ})) != SWIGLU_OK) return st;
  if (dX != nullptr && (st = check_ptrs({W})) != SWIGLU_OK) return st;
  if (dX != nullptr && x_act != SWIGLU_ACT_NONE && (st = check_ptrs({X_pre})) != SWIGLU_OK) return st;
  if (dW != nullptr && (st = check_ptrs({X})) != SWIGLU_OK) return st;
  int* err = static_cast<int*>(ws);
  const size_t mn = (size_t)(M * N * e), mk = (size_t)(M * K * e), nk = (size_t)(N * K * e);
  const void* G = dY;
  bool first = true;  // the next kernel clears the error word
  if (act != SWIGLU_ACT_NONE || dbias != nullptr) {
    const bool has = act != SWIGLU_ACT_NONE;
    float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + FIXED);
    const int parts = dact_parts(M, N, dtype);
    DactArgs a = {dY, has ? Z : nullptr, has ? dZ : nullptr, dbias != nullptr ? part : nullptr, M, (int)N, act, err, {}};
    a.chk = row_check(ws, {{has ? dZ : ws, has ? mn : ws_bytes}, {ws, ws_bytes}, {dY, mn}, {Z, has ? mn : 0}});
    const dim3 grid((unsigned)((N * e + 511) / 512), (unsigned)parts);
    cudaError_t c = by_type(dtype, [&](auto t) {
      return launch(host::K_DACT, has ? dact_kernel<decltype(t), true> : dact_kernel<decltype(t), false>, grid,
                    DA_THREADS, 0, s, a);
    });
    if (c == cudaSuccess && dbias != nullptr)
      c = column_sums(part, parts, (int)N, dbias, nullptr, (int)N, accumulate, dtype, ws, ws_bytes, s);
    if (c != cudaSuccess) return SWIGLU_ERR_CUDA;
    if (has) G = dZ;
    first = false;
  }
  if (dtype == SWIGLU_F32_IEEE) {
    const float *g = (const float*)G, *x = (const float*)X, *w = (const float*)W;
    if (dW != nullptr) {
      const SlEpiGrad epi{nullptr, (float*)dW, K, 0, accumulate};
      if (simt_product<false, false>(host::K_SIMT_LINEAR_DW, g, N, x, K, N, K, M, epi, ws, first,
                                     {{dW, nk}, {G, mn}, {X, mk}}, s) != cudaSuccess)
        return SWIGLU_ERR_CUDA;
    }
    if (dX != nullptr) {
      first = first && dW == nullptr;
      const bool pre = x_act != SWIGLU_ACT_NONE;
      const SlEpiGrad epi{pre ? (const float*)X_pre : nullptr, (float*)dX, K, x_act, 0};
      if (simt_product<true, false>(host::K_SIMT_LINEAR_DX, g, N, w, K, M, K, N, epi, ws, first,
                                    {{dX, mk}, {G, mn}, {W, nk}, {X_pre, pre ? mk : 0}}, s) != cudaSuccess)
        return SWIGLU_ERR_CUDA;
    }
    return SWIGLU_OK;
  }
  const bool bf = dtype == SWIGLU_BF16;
  if (dW != nullptr &&
      host::gemm_dw(host::K_LINEAR_DW, bf, G, X, dW, M, N, K, accumulate, err, ws_bytes, first, s) != cudaSuccess)
    return SWIGLU_ERR_CUDA;
  first = first && dW == nullptr;
  if (dX != nullptr) {
    const EpiDAct::Params ep{X_pre, dX, K, x_act};
    const cudaError_t c = x_act == SWIGLU_ACT_NONE ? host::gemm_dx(host::K_LINEAR_DX, bf, G, W, dX, M, N, K, err, ws_bytes, first, s)
                          : bf ? linear_dx<true>(G, W, ep, M, N, K, err, ws_bytes, first, s)
                               : linear_dx<false>(G, W, ep, M, N, K, err, ws_bytes, first, s);
    if (c != cudaSuccess) return SWIGLU_ERR_CUDA;
  }
  return SWIGLU_OK;
}

}  // extern "C"
