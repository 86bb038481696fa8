// serving.cu -- C ABI of the few-token serving operators
// (include/swiglu_mlp.h): 4-bit weights and mixture-of-experts layers.
// Argument checks, shared-memory plans and launches.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/swiglu_mlp.h"
#include "experts.cuh"
#include "experts_plan.h"
#include "fewtok.cuh"
#include "host_shared.h"
#include "moe_route.cuh"
#include "w4_layout.cuh"
#include "w4_stream.cuh"
#include "w4_tensor.cuh"

using namespace swiglu;

namespace {

#ifdef SWIGLU_DEBUG
#define SET_WINDOWS(args, ...) (args).dbg = host::windows(__VA_ARGS__)
#else
#define SET_WINDOWS(args, ...) (void)0
#endif

// Sizes up to which the kernels' 32-bit indexes hold, with their last tiles'
// overhang: rows of a matrix, its contraction (byte offsets within one tile's
// records: K / 64 of 608 bytes), and the sizes of a mixture's experts (items:
// up to 640 entries of H / 8 or D / 16 tiles; chunks of a run times warps).
constexpr int64_t MAX_ROWS = 0x7fffffffLL - 256, MAX_K = 1LL << 27, MAX_EXPERT = 1LL << 24;
constexpr size_t HEADER = 256;  // workspace header: the error word

swiglu_status status_of(cudaError_t e) { return e == cudaSuccess ? SWIGLU_OK : SWIGLU_ERR_CUDA; }

bool sixteen_bit(swiglu_dtype dt) { return dt == SWIGLU_BF16 || dt == SWIGLU_F16; }

swiglu_status check_dtype(swiglu_dtype dt) {
  return sixteen_bit(dt) ? SWIGLU_OK : dt == SWIGLU_F32_IEEE ? SWIGLU_ERR_UNSUPPORTED : SWIGLU_ERR_INVALID_ARG;
}

swiglu_status check_ptrs(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (p == nullptr) return SWIGLU_ERR_INVALID_ARG;
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) & 15u) return SWIGLU_ERR_ALIGNMENT;
  return SWIGLU_OK;
}

int log2_group(int group) { return group == 32 ? 5 : group == 64 ? 6 : group == 128 ? 7 : -1; }

// One 4-bit matrix [N, K]: sizes, group and zero-point flag.
swiglu_status check_w4(int64_t E, int64_t N, int64_t K, int group, int zeros) {
  if (E <= 0 || N <= 0 || K <= 0) return SWIGLU_ERR_INVALID_ARG;
  if (log2_group(group) < 0 || (zeros != 0 && zeros != 1)) return SWIGLU_ERR_INVALID_ARG;
  if (K % 8 != 0) return SWIGLU_ERR_ALIGNMENT;
  if (E > MAX_ROWS || N > MAX_ROWS || K > MAX_K) return SWIGLU_ERR_UNSUPPORTED;
  return SWIGLU_OK;
}

swiglu_status check_ws(const void* ws, size_t bytes, size_t need) {
  if (ws == nullptr || bytes < need) return SWIGLU_ERR_WORKSPACE;
  return (reinterpret_cast<uintptr_t>(ws) & 15u) ? SWIGLU_ERR_ALIGNMENT : SWIGLU_OK;
}

struct Muls {
  float gate = 1.0f, down = 1.0f;
};
swiglu_status read_muls(const swiglu_mlp_options* o, Muls* m) {
  if (o == nullptr) return SWIGLU_OK;
  if (!std::isfinite(o->gate_multiplier) || !std::isfinite(o->down_multiplier) || o->accumulate != 0)
    return SWIGLU_ERR_INVALID_ARG;
  m->gate = o->gate_multiplier;
  m->down = o->down_multiplier;
  return SWIGLU_OK;
}

// The dynamic shared memory of a kernel, raised once per device.
template <auto KERNEL>
cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load() & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit);
  return e;
}

constexpr int WS_SMEM = 224 * 1024;

template <bool BF16, bool W4, int NT, bool G32, bool ZP>
cudaError_t launch_experts(host::ServingKernel id, const CUtensorMap& tm, FtArgs a,
                           cudaStream_t st) {
  using S = WxShape<W4, NT, G32, ZP>;
  constexpr auto kern = experts_kernel<BF16, W4, NT, G32, ZP>;
  cudaError_t e = allow_smem<kern>(WX_SMEM_MOST);
  if (e != cudaSuccess) return e;
  const bool combine = a.mode == FT_COMBINE;
  const int nsm = host::sms() > 0 ? host::sms() : 1;
  const int64_t items =
      combine ? a.tiles : (int64_t)a.tiles * ft_max_entries(a.M, a.topk, a.E, S::TOKENS);
  const int grid = (int)(items < nsm ? items : nsm);
  const int64_t most = (items + grid - 1) / grid;  // items of a block
  const WxPlan plan = wx_plan(S::WARPS, NT, S::STAGE, combine, a.M, a.topk, a.E, most);
  if (plan.stages < 2) return cudaErrorInvalidConfiguration;
  a.run = plan.run;
  a.list_off = plan.list_off;
  a.red_off = plan.red_off;
  a.ring_off = plan.ring_off;
  a.stages = plan.stages;
  a.wait_limit_ns = host::wait_limit_ns();
  a.inject = host::take_stall() ? 1 : 0;
  host::Prof prof(id, st);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(S::WARPS * 32);
  cfg.dynamicSmemBytes = plan.bytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  // per-kernel event timing would serialise the launches, so no overlap then
  cfg.attrs = attr;
  cfg.numAttrs = host::profiling() ? 0 : 1;
  e = cudaLaunchKernelEx(&cfg, kern, tm, a);
  host::count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

// nt: 8-token columns of a pass over an expert's weights
template <bool BF16, int NT>
cudaError_t launch_experts(host::ServingKernel id, const CUtensorMap& tm, const FtArgs& a,
                           const swiglu_mlp_w4_format* f, cudaStream_t st) {
  if (f == nullptr) return launch_experts<BF16, false, NT, false, false>(id, tm, a, st);
  if (f->group == 32)
    return f->zeros ? launch_experts<BF16, true, NT, true, true>(id, tm, a, st)
                    : launch_experts<BF16, true, NT, true, false>(id, tm, a, st);
  return f->zeros ? launch_experts<BF16, true, NT, false, true>(id, tm, a, st)
                  : launch_experts<BF16, true, NT, false, false>(id, tm, a, st);
}

cudaError_t launch_experts(host::ServingKernel id, const CUtensorMap& tm, const FtArgs& a, int nt,
                           const swiglu_mlp_w4_format* f, swiglu_dtype dt, cudaStream_t st) {
  if (dt == SWIGLU_BF16)
    return nt == 1 ? launch_experts<true, 1>(id, tm, a, f, st) : launch_experts<true, 2>(id, tm, a, f, st);
  return nt == 1 ? launch_experts<false, 1>(id, tm, a, f, st) : launch_experts<false, 2>(id, tm, a, f, st);
}

// Clusters of `size` blocks of a kernel that fit the device at once (a cluster
// lies within a GPU processing cluster), cached per kernel and size.
template <auto KERNEL>
int max_clusters(int size, int threads, int smem) {
  static std::atomic<int> known[4];  // sizes 1, 2, 4, 8
  const int at = size == 1 ? 0 : size == 2 ? 1 : size == 4 ? 2 : 3;
  int n = known[at].load();
  if (n > 0) return n;
  const int nsm = host::sms() > 0 ? host::sms() : 1;
  n = nsm / size;
  if (size > 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(nsm / size * size));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)size, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int q = 0;
    if (cudaOccupancyMaxActiveClusters(&q, KERNEL, &cfg) == cudaSuccess && q > 0) n = q;
    cudaGetLastError();  // a failed query is not an error of the call
  }
  if (n < 1) n = 1;
  known[at].store(n);
  return n;
}

// One product with packed 4-bit weights: the shared-memory plan and the launch.
// The contraction is split over the smallest cluster whose blocks can each hold
// their part of the tokens' rows beside a ring of two stages; the largest one
// goes through its part in phases.
template <bool BF16, int RT, int NT, bool G32, bool ZP>
cudaError_t launch_ws(host::ServingKernel id, WsArgs a, int tiles16, cudaStream_t st) {
  using S = WsShape<RT, NT, G32, ZP>;
  constexpr auto kern = w4_stream_kernel<BF16, RT, NT, G32, ZP>;
  cudaError_t e = allow_smem<kern>(WS_SMEM);
  if (e != cudaSuccess) return e;
  auto up = [](int v) { return (v + 127) & ~127; };
  const int tiles = (tiles16 + RT - 1) / RT;
  a.tiles16 = tiles16;
  const int nk = (a.K + 63) / 64, rows = a.M < S::TOKENS ? a.M : S::TOKENS;
  constexpr int ring = S::WARPS * S::STAGE;
  int clusters = 0;
  auto plan = [&](int split, int phases) {
    const int most = max_clusters<kern>(split, S::WARPS * 32, WS_SMEM);
    clusters = tiles < most ? tiles : most;
    a.split = split;
    a.tile_quot = tiles / clusters;
    a.tile_rem = tiles % clusters;
    const int per = a.tile_quot + (a.tile_rem != 0);
    a.run = per < S::RUN ? per : S::RUN;
    a.phase_units = ((nk + split - 1) / split + phases - 1) / phases;
    if (phases > 1) a.phase_units = (a.phase_units + S::UNITS - 1) / S::UNITS * S::UNITS;
    if (a.phase_units > WS_SMEM / 128) return false;  // no row of them fits, nor its offsets 32 bits
    a.part_off = up(rows * S::xrow(a.phase_units));
    a.tile_off = up(a.part_off + (a.run + S::WARPS - 1) * S::PART);
    a.phased = phases > 1;
    a.ring_off = up(a.tile_off + (a.phased ? a.run * S::PART : 0));
    a.stages = a.ring_off < WS_SMEM ? (WS_SMEM - a.ring_off) / ring : 0;
    return a.stages >= 2;
  };
  bool fits = false;
  for (int split = 1; !fits && split <= 8 && split <= nk; split *= 2) fits = plan(split, 1);
  for (int phases = 2, split = a.split; !fits; ++phases) {
    if (a.phase_units <= S::UNITS) return cudaErrorInvalidConfiguration;
    fits = plan(split, phases);
  }
  if (a.stages > WS_MAX_STAGES) a.stages = WS_MAX_STAGES;
  a.wait_limit_ns = host::wait_limit_ns();
  a.inject = host::take_stall() ? 1 : 0;
  host::Prof prof(id, st);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * a.split));
  cfg.blockDim = dim3(S::WARPS * 32);
  cfg.dynamicSmemBytes = a.ring_off + a.stages * ring;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int n = 0;
  // per-kernel event timing would serialise the launches, so no overlap then
  if (!host::profiling()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (a.split > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n++].val.clusterDim = {(unsigned)a.split, 1, 1};
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  e = cudaLaunchKernelEx(&cfg, kern, a);
  host::count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

// The tensor-core form: its split over the blocks and its part of the workspace
// (header, counters of gate/up and of down, partial tiles).
constexpr size_t WT_COUNTERS = 2 * WT_MAX_SHARED * 4;
struct WtPlan {
  int grid, sk_tiles, sharers, seg_max;
};
int wt_columns(int64_t M) { return M <= 32 ? 32 : M <= 48 ? 48 : 64; }
// Which form a product takes.  With 33 to 64 tokens w4_stream.cuh would read the
// weights twice.  Up to 32 both read them once; it starts up faster, and is bound
// by products and shared-memory reads that grow with rows x K x tokens, in steps
// (clusters, columns).  Measured in us, w4_stream.cuh first, groups of 128:
//   tokens  8192 x 4096  4096 x 11008  8192 x 8192  22016 x 4096  14336 x 8192
//     17    14.5, 17.8    18.0, 20.6    23.4, 24.0   28.9, 30.4    38.6, 31.9
//     24    14.7, 17.8    22.1, 20.7    33.4, 24.0   35.9, 30.4    54.3, 31.9
//     32    16.1, 17.8    22.3, 20.7    33.2, 24.0   35.6, 30.7    54.2, 32.0
// In groups of 32 the tensor core needs an accumulator per 32 k and comes into its
// own later:
//     24    15.3, 21.5    23.0, 26.0    34.3, 31.8   37.0, 41.3    56.4, 45.2
// Where this takes the slower one of the two it costs 5 to 12% as a rule, and
// at worst 20% (20 tokens, 40000 x 2048) or, in groups of 32 with zero points,
// 29% (32 tokens, 2048 x 40000).
constexpr int64_t WT_MIN_PRODUCTS = (int64_t)21 << 26;
bool wt_serves(int64_t M, int64_t tiles16, int64_t K, int group_log2) {
  const int64_t least = group_log2 == 5 ? 2 * WT_MIN_PRODUCTS : WT_MIN_PRODUCTS;
  return M > 32 || (M > 16 && tiles16 * 16 * K >= least / M);
}
WtPlan wt_plan(int tiles, int nk) {
  const int nsm = host::sms() > 0 ? host::sms() : 1, spt = (nk + WT_KB - 1) / WT_KB;
  WtPlan p;
  // whole tiles where every block gets one; the others' stages are shared evenly
  p.sk_tiles = tiles >= nsm ? tiles % nsm : tiles;
  const int64_t total = (int64_t)p.sk_tiles * spt;
  p.grid = tiles < nsm && total < nsm ? (int)total : nsm;
  p.sharers = total < p.grid ? (int)total : p.grid;
  const int64_t range = p.sharers > 0 ? (total + p.sharers - 1) / p.sharers : 0;
  p.seg_max = (int)((range + spt - 1) / spt) + 1;
  return p;
}
size_t wt_workspace(int64_t M, int64_t tiles16, int64_t K) {
  if (M > FT_MAX_TOKENS || !wt_serves(M, tiles16, K, 7)) return HEADER;  // whatever the groups
  const WtPlan p = wt_plan((int)((tiles16 + 7) / 8), (int)((K + 63) / 64));
  return HEADER + WT_COUNTERS + (size_t)p.grid * p.seg_max * wt_columns(M) * 512;
}

template <bool BF16, int NT, bool G32, bool ZP>
cudaError_t launch_wt(host::ServingKernel id, const WsArgs& s, int pair, int tiles16,
                      cudaStream_t st) {
  using S = WtShape<NT, G32, ZP>;
  constexpr auto kern = w4_tensor_kernel<BF16, NT, G32, ZP>;
  constexpr int fixed = WT_OUT + 1024;
  cudaError_t e = allow_smem<kern>(WS_SMEM);
  if (e != cudaSuccess) return e;
  CUtensorMap tw, tx;
  const int nk = (s.K + 63) / 64;
  // token rows: in whole 64-k blocks as [K / 64][M][64], one box a stage, else
  // as [M][K] with boxes of one block
  if (!host::encode_records(&tw, s.W, S::RECORD, nk, tiles16, WT_KB, 8) ||
      !(s.K % 64 == 0 ? host::encode_blocks(&tx, BF16, s.X, s.K, s.M, NT, WT_KB)
                      : host::encode_3d(&tx, BF16, s.X, s.K, s.M, 1, 64, NT, 1)))
    return cudaErrorInvalidValue;
  const int tiles = (tiles16 + 7) / 8;
  const WtPlan p = wt_plan(tiles, nk);
  char* ws = reinterpret_cast<char*>(s.err);
  WtArgs a = {};
  a.gate_up = s.gate_up;
  a.M = s.M;
  a.K = s.K;
  a.rows = s.rows;
  a.tiles16 = tiles16;
  a.tiles = tiles;
  a.sk_tiles = p.sk_tiles;
  a.sharers = p.sharers;
  a.seg_max = p.seg_max;
  a.pair = pair;
  a.W = s.W;
  a.out = s.out;
  a.scale = s.scale;
  a.first = s.first;
  a.stages = (WS_SMEM - fixed) / S::STAGE < WT_MAX_STAGES ? (WS_SMEM - fixed) / S::STAGE : WT_MAX_STAGES;
  a.counters = reinterpret_cast<int*>(ws + HEADER) + (s.gate_up ? 0 : WT_MAX_SHARED);
  a.part = reinterpret_cast<float*>(ws + HEADER + WT_COUNTERS);
  a.wait_limit_ns = host::wait_limit_ns();
  a.err = s.err;
  a.inject = host::take_stall() ? 1 : 0;
#ifdef SWIGLU_DEBUG
  a.dbg = s.dbg;
#endif
  host::Prof prof(id, st);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.grid);
  cfg.blockDim = dim3(WT_THREADS);
  cfg.dynamicSmemBytes = fixed + a.stages * S::STAGE;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  // per-kernel event timing would serialise the launches, so no overlap then
  cfg.attrs = attr;
  cfg.numAttrs = host::profiling() ? 0 : 1;
  e = cudaLaunchKernelEx(&cfg, kern, tw, tx, a);
  host::count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool BF16, bool G32, bool ZP>
cudaError_t launch_wt(host::ServingKernel id, const WsArgs& s, int pair, int tiles16,
                      cudaStream_t st) {
  const int nt = wt_columns(s.M);
  if (nt == 32) return launch_wt<BF16, 32, G32, ZP>(id, s, pair, tiles16, st);
  if (nt == 48) return launch_wt<BF16, 48, G32, ZP>(id, s, pair, tiles16, st);
  return launch_wt<BF16, 64, G32, ZP>(id, s, pair, tiles16, st);
}

// Token columns of a pass: 8, 16 or 32.
template <bool BF16, bool G32, bool ZP>
cudaError_t launch_ws(host::ServingKernel id, const WsArgs& a, int tiles16, cudaStream_t st) {
  if (a.M <= 8) return launch_ws<BF16, 1, 1, G32, ZP>(id, a, tiles16, st);
  if (a.M <= 16) return launch_ws<BF16, 2, 2, G32, ZP>(id, a, tiles16, st);
  return launch_ws<BF16, 2, 4, G32, ZP>(id, a, tiles16, st);
}

template <bool BF16>
cudaError_t launch_ws(host::ServingKernel id, const WsArgs& a, const W4Geom& w, cudaStream_t st) {
  if (wt_serves(a.M, w.tiles, a.K, w.group_log2)) {
    const int pair = w.group_log2 == 7 ? 2 : 1;
    if (w.sets == 2)
      return w.zeros ? launch_wt<BF16, true, true>(id, a, pair, w.tiles, st)
                     : launch_wt<BF16, true, false>(id, a, pair, w.tiles, st);
    return w.zeros ? launch_wt<BF16, false, true>(id, a, pair, w.tiles, st)
                   : launch_wt<BF16, false, false>(id, a, pair, w.tiles, st);
  }
  if (w.sets == 2)
    return w.zeros ? launch_ws<BF16, true, true>(id, a, w.tiles, st)
                   : launch_ws<BF16, true, false>(id, a, w.tiles, st);
  return w.zeros ? launch_ws<BF16, false, true>(id, a, w.tiles, st)
                 : launch_ws<BF16, false, false>(id, a, w.tiles, st);
}

cudaError_t launch_ws(host::ServingKernel id, const WsArgs& a, const W4Geom& w, swiglu_dtype dt,
                      cudaStream_t st) {
  return dt == SWIGLU_BF16 ? launch_ws<true>(id, a, w, st) : launch_ws<false>(id, a, w, st);
}


int grid_for(int64_t threads) {
  const int64_t want = (threads + 255) / 256, most = (int64_t)(host::sms() > 0 ? host::sms() : 1) * 8;
  return (int)(want < 1 ? 1 : want < most ? want : most);
}

size_t moe_inner_bytes(int64_t T, int64_t H, int topk) {
  return ((size_t)T * (size_t)topk * (size_t)H * 2 + 255) & ~(size_t)255;
}

// Sizes, types and formats of a mixture-of-experts layer.
swiglu_status check_moe(int64_t T, int64_t D, int64_t H, int64_t E, int64_t topk,
                        const swiglu_mlp_w4_format* f, swiglu_dtype dt) {
  const swiglu_status st = check_dtype(dt);
  if (st != SWIGLU_OK) return st;
  if (T < 0 || D <= 0 || H <= 0 || E <= 0 || topk <= 0 || topk > E) return SWIGLU_ERR_INVALID_ARG;
  if (f != nullptr && (log2_group(f->group) < 0 || (f->zeros != 0 && f->zeros != 1)))
    return SWIGLU_ERR_INVALID_ARG;
  if (D % 8 != 0 || H % 8 != 0) return SWIGLU_ERR_ALIGNMENT;
  if (T > FT_MAX_TOKENS || E > FT_MAX_EXPERTS || topk > FT_MAX_TOPK || D > MAX_EXPERT ||
      H > MAX_EXPERT)
    return SWIGLU_ERR_UNSUPPORTED;
  return SWIGLU_OK;
}

// 8-token columns per pass over an expert's weights: an expert meets T topk / E
// tokens on average, and one with more takes several passes.  16 columns cost
// 16-bit experts little more than 8 (64 experts, 8 of them per token, D = 2048,
// H = 1024: at 64 tokens 166 against 219 us, at 16 tokens 135 against 130),
// 4-bit ones, bound by issue slots, 1.6 times as much (64 tokens: 133 against
// 117 us).
int moe_columns(int64_t T, int64_t E, int64_t topk, bool w4) {
  if (T <= 8) return 1;
  return (w4 ? T * topk <= 12 * E : 3 * T * topk <= 8 * E) ? 1 : 2;
}

// The experts of a layer: gate/up over the active experts' rows into the
// assignments' hidden values (workspace), then down and the weighted sums.
swiglu_status run_experts(const void* X, const int* idx, const float* wts, const void* Wgu,
                          const void* Wd, void* Y, int T, int D, int H, int E, int topk,
                          const swiglu_mlp_w4_format* f, swiglu_dtype dt, const Muls& mu, char* ws,
                          size_t ws_bytes, bool after_router, cudaStream_t st) {
  (void)ws_bytes;
  void* A = ws + HEADER + WT_COUNTERS;  // past the counters of the products above
  const bool w4 = f != nullptr, bf = dt == SWIGLU_BF16;
  const W4Geom gu = w4 ? w4_geom(2 * (int64_t)H, D, log2_group(f->group), f->zeros, 1) : W4Geom{};
  const W4Geom dn = w4 ? w4_geom(D, H, log2_group(f->group), f->zeros, 0) : W4Geom{};
  CUtensorMap tgu = {}, tdn = {};
  // one box: 64 k of 8 rows of an expert's Wg and the same 8 of its Wu, or of
  // 16 rows of its Wd
  if (!w4 && (!host::encode_3d(&tgu, bf, Wgu, D, H, 2 * (int64_t)E, 64, 8, 2) ||
              !host::encode_3d(&tdn, bf, Wd, H, D, E, 64, 16, 1)))
    return SWIGLU_ERR_CUDA;
  FtArgs a = {};
  a.mode = FT_GATE_UP;
  a.M = T;
  a.K = D;
  a.rows = H;
  a.tiles = H / 8;
  a.W = static_cast<const uint8_t*>(Wgu);
  a.expert_bytes = gu.bytes;
  a.X = X;
  a.out = A;
  a.scale = mu.gate;
  a.E = E;
  a.topk = topk;
  a.idx = idx;
  a.wts = wts;
  a.first = after_router ? 0 : 1;
  a.err = reinterpret_cast<int*>(ws);
  const int nt = moe_columns(T, E, topk, w4);
  SET_WINDOWS(a, {{ws, ws_bytes},
                  {idx, (size_t)T * topk * 4},
                  {wts, (size_t)T * topk * 4},
                  {X, (size_t)T * D * 2}});
  if (launch_experts(w4 ? host::SK_MOE_W4_GATE_UP : host::SK_MOE_GATE_UP, tgu, a, nt, f, dt, st) !=
      cudaSuccess)
    return SWIGLU_ERR_CUDA;
  a.mode = FT_COMBINE;
  a.K = H;
  a.rows = D;
  a.tiles = (D + 15) / 16;
  a.W = static_cast<const uint8_t*>(Wd);
  a.expert_bytes = dn.bytes;
  a.X = A;
  a.out = Y;
  a.scale = mu.down;
  a.first = 0;
  a.idx_ready = 1;
  SET_WINDOWS(a, {{Y, (size_t)T * D * 2},
                  {idx, (size_t)T * topk * 4},
                  {wts, (size_t)T * topk * 4},
                  {ws, ws_bytes}});
  return status_of(launch_experts(w4 ? host::SK_MOE_W4_DOWN : host::SK_MOE_DOWN, tdn, a, nt, f, dt, st));
}

swiglu_status run_route(const void* X, const void* Wr, int* idx, float* wts, int T, int D, int E,
                        int topk, int norm, float scale, swiglu_dtype dt, int* err,
                        cudaStream_t st) {
  RtArgs a = {};
  a.X = static_cast<const uint8_t*>(X);
  a.Wr = static_cast<const uint8_t*>(Wr);
  a.idx = idx;
  a.wts = wts;
  a.M = T;
  a.D = D;
  a.E = E;
  a.topk = topk;
  a.norm = norm;
  a.scale = scale;
  a.err = err;
  SET_WINDOWS(a, {{idx, (size_t)T * topk * 4},
                  {wts, (size_t)T * topk * 4},
                  {X, (size_t)T * D * 2},
                  {Wr, (size_t)E * D * 2}});
  const int blocks = (E + 7) / 8 < RT_CLUSTER ? (E + 7) / 8 : RT_CLUSTER;
  a.per_block = (E + blocks - 1) / blocks;
  host::Prof prof(host::SK_MOE_ROUTE, st);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((T + RT_TOKENS - 1) / RT_TOKENS * blocks));
  cfg.blockDim = dim3(RT_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)blocks, 1, 1};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = host::profiling() ? 1 : 2;
  const bool bf = dt == SWIGLU_BF16;
  cudaError_t e =
      E <= 64 ? cudaLaunchKernelEx(&cfg, bf ? route_kernel<true, 2> : route_kernel<false, 2>, a)
      : E <= 128 ? cudaLaunchKernelEx(&cfg, bf ? route_kernel<true, 4> : route_kernel<false, 4>, a)
                 : cudaLaunchKernelEx(&cfg, bf ? route_kernel<true, 16> : route_kernel<false, 16>, a);
  host::count_launch();
  return status_of(e != cudaSuccess ? e : cudaGetLastError());
}

}  // namespace

extern "C" {

size_t swiglu_mlp_w4_packed_bytes(int64_t E, int64_t N, int64_t K, int group, int zeros,
                                  int gate_up) {
  if (check_w4(E, N, K, group, zeros) != SWIGLU_OK || (gate_up && N % 16 != 0)) return 0;
  return (size_t)(w4_geom(N, K, log2_group(group), zeros, gate_up ? 1 : 0).bytes) * (size_t)E;
}

swiglu_status swiglu_mlp_w4_quantize(const void* W, void* codes, void* scales, void* zeros,
                                     int64_t N, int64_t K, int group, swiglu_dtype dtype,
                                     void* stream) {
  host::reset_launches();
  swiglu_status st = check_dtype(dtype);
  if (st != SWIGLU_OK) return st;
  st = check_w4(1, N, K, group, zeros != nullptr);
  if (st != SWIGLU_OK) return st;
  if ((st = check_ptrs({W, codes, scales})) != SWIGLU_OK) return st;
  if (reinterpret_cast<uintptr_t>(zeros) & 15u) return SWIGLU_ERR_ALIGNMENT;
  const int lg = log2_group(group), groups = (int)((K + group - 1) / group);
  const int grid = grid_for(N * ((int64_t)groups << (lg - 3)));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto k = dtype == SWIGLU_BF16 ? w4_quantize_kernel<true> : w4_quantize_kernel<false>;
  k<<<grid, 256, 0, s>>>(N, (int)K, lg, groups, static_cast<const uint16_t*>(W),
                         static_cast<uint8_t*>(codes), static_cast<uint16_t*>(scales),
                         static_cast<uint8_t*>(zeros));
  host::count_launch();
  return status_of(cudaGetLastError());
}

swiglu_status swiglu_mlp_w4_pack(const void* codes, const void* scales, const void* zeros,
                                 void* packed, int64_t E, int64_t N, int64_t K, int group,
                                 int gate_up, swiglu_dtype dtype, void* stream) {
  host::reset_launches();
  swiglu_status st = check_dtype(dtype);
  if (st != SWIGLU_OK) return st;
  st = check_w4(E, N, K, group, zeros != nullptr);
  if (st != SWIGLU_OK) return st;
  if (gate_up && N % 16 != 0) return SWIGLU_ERR_ALIGNMENT;
  if ((st = check_ptrs({codes, scales, packed})) != SWIGLU_OK) return st;
  if (reinterpret_cast<uintptr_t>(zeros) & 15u) return SWIGLU_ERR_ALIGNMENT;
  const W4Geom w = w4_geom(N, K, log2_group(group), zeros != nullptr, gate_up ? 1 : 0);
  const int grid = grid_for((int64_t)w.tiles * w.blocks * 32 * E);
  w4_pack_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(
      w, E, static_cast<const uint8_t*>(codes), static_cast<const uint16_t*>(scales),
      static_cast<const uint8_t*>(zeros), static_cast<uint8_t*>(packed));
  host::count_launch();
  return status_of(cudaGetLastError());
}

swiglu_status swiglu_mlp_w4_unpack(const void* packed, void* W, int64_t E, int64_t N, int64_t K,
                                   int group, int zeros, int gate_up, swiglu_dtype dtype,
                                   void* stream) {
  host::reset_launches();
  swiglu_status st = check_dtype(dtype);
  if (st != SWIGLU_OK) return st;
  st = check_w4(E, N, K, group, zeros);
  if (st != SWIGLU_OK) return st;
  if (gate_up && N % 16 != 0) return SWIGLU_ERR_ALIGNMENT;
  if ((st = check_ptrs({packed, W})) != SWIGLU_OK) return st;
  const W4Geom w = w4_geom(N, K, log2_group(group), zeros, gate_up ? 1 : 0);
  const int grid = grid_for((int64_t)w.tiles * w.blocks * 32 * E);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto k = dtype == SWIGLU_BF16 ? w4_unpack_kernel<true> : w4_unpack_kernel<false>;
  k<<<grid, 256, 0, s>>>(w, E, static_cast<const uint8_t*>(packed), static_cast<uint16_t*>(W));
  host::count_launch();
  return status_of(cudaGetLastError());
}

size_t swiglu_mlp_w4_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return N <= 0 || K <= 0 ? HEADER : wt_workspace(M, (N + 15) / 16, K);
}

size_t swiglu_mlp_fwd_nograd_w4_workspace_bytes(int64_t M, int64_t D, int64_t H) {
  if (D <= 0 || H <= 0) return HEADER;
  const size_t a = wt_workspace(M, (H + 7) / 8, D), b = wt_workspace(M, (D + 15) / 16, H);
  return a > b ? a : b;
}

swiglu_status swiglu_mlp_w4_linear(const void* X, const void* packed, void* Y, int64_t M, int64_t N,
                                   int64_t K, int group, int zeros, swiglu_dtype dtype, void* ws,
                                   size_t ws_bytes, void* stream) {
  host::reset_launches();
  swiglu_status st = check_dtype(dtype);
  if (st != SWIGLU_OK) return st;
  if (M < 0) return SWIGLU_ERR_INVALID_ARG;
  st = check_w4(1, N, K, group, zeros);
  if (st != SWIGLU_OK) return st;
  if (M > FT_MAX_TOKENS) return SWIGLU_ERR_UNSUPPORTED;
  if ((st = check_ws(ws, ws_bytes, swiglu_mlp_w4_workspace_bytes(M, N, K))) != SWIGLU_OK) return st;
  if (M == 0) return SWIGLU_OK;
  if ((st = check_ptrs({X, packed, Y})) != SWIGLU_OK) return st;
  const W4Geom w = w4_geom(N, K, log2_group(group), zeros, 0);
  WsArgs a = {};
  a.M = (int)M;
  a.K = (int)K;
  a.rows = (int)N;
  a.W = static_cast<const uint8_t*>(packed);
  a.X = X;
  a.out = Y;
  a.scale = 1.0f;
  a.first = 1;
  a.err = static_cast<int*>(ws);
  SET_WINDOWS(a, {{Y, (size_t)(M * N * 2)}, {X, (size_t)(M * K * 2)}, {packed, (size_t)w.bytes},
                  {ws, ws_bytes}});
  return status_of(launch_ws(host::SK_W4_LINEAR, a, w, dtype,
                             static_cast<cudaStream_t>(stream)));
}

swiglu_status swiglu_mlp_fwd_nograd_w4(const void* X, const void* Wgu, const void* Wd, void* Y,
                                       void* A, int64_t M, int64_t D, int64_t H, int group,
                                       int zeros, swiglu_dtype dtype,
                                       const swiglu_mlp_options* options, void* ws,
                                       size_t ws_bytes, void* stream) {
  host::reset_launches();
  Muls mu;
  swiglu_status st = read_muls(options, &mu);
  if (st != SWIGLU_OK) return st;
  if ((st = check_dtype(dtype)) != SWIGLU_OK) return st;
  if (M < 0) return SWIGLU_ERR_INVALID_ARG;
  if ((st = check_w4(1, D, H, group, zeros)) != SWIGLU_OK) return st;
  if (D % 8 != 0) return SWIGLU_ERR_ALIGNMENT;
  if (M > FT_MAX_TOKENS || D > MAX_K) return SWIGLU_ERR_UNSUPPORTED;
  if ((st = check_ws(ws, ws_bytes, swiglu_mlp_fwd_nograd_w4_workspace_bytes(M, D, H))) != SWIGLU_OK)
    return st;
  if (M == 0) return SWIGLU_OK;
  if ((st = check_ptrs({X, Wgu, Wd, Y, A})) != SWIGLU_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const W4Geom gu = w4_geom(2 * H, D, log2_group(group), zeros, 1);
  WsArgs a = {};
  a.gate_up = 1;
  a.M = (int)M;
  a.K = (int)D;
  a.rows = (int)H;
  a.W = static_cast<const uint8_t*>(Wgu);
  a.X = X;
  a.out = A;
  a.scale = mu.gate;
  a.first = 1;
  a.err = static_cast<int*>(ws);
  SET_WINDOWS(a, {{A, (size_t)(M * H * 2)}, {X, (size_t)(M * D * 2)}, {Wgu, (size_t)gu.bytes},
                  {ws, ws_bytes}});
  if (launch_ws(host::SK_W4_GATE_UP, a, gu, dtype, s) != cudaSuccess)
    return SWIGLU_ERR_CUDA;
  const W4Geom dn = w4_geom(D, H, log2_group(group), zeros, 0);
  a.gate_up = 0;
  a.K = (int)H;
  a.rows = (int)D;
  a.W = static_cast<const uint8_t*>(Wd);
  a.X = A;
  a.out = Y;
  a.scale = mu.down;
  a.first = 0;
  SET_WINDOWS(a, {{Y, (size_t)(M * D * 2)}, {A, (size_t)(M * H * 2)}, {Wd, (size_t)dn.bytes},
                  {ws, ws_bytes}});
  return status_of(launch_ws(host::SK_W4_DOWN, a, dn, dtype, s));
}

size_t swiglu_mlp_moe_workspace_bytes(int64_t T, int64_t D, int64_t H, int64_t E, int topk) {
  (void)D;
  (void)E;
  if (T < 0 || H <= 0 || topk <= 0) return 0;
  return HEADER + WT_COUNTERS + moe_inner_bytes(T, H, topk);
}

swiglu_status swiglu_mlp_moe_route(const void* X, const void* Wr, int32_t* idx, float* weights,
                                   int64_t T, int64_t D, int64_t E, int topk, int norm_topk,
                                   float route_scale, swiglu_dtype dtype, void* stream) {
  host::reset_launches();
  swiglu_status st = check_moe(T, D, 8, E, topk, nullptr, dtype);
  if (st != SWIGLU_OK) return st;
  if ((norm_topk != 0 && norm_topk != 1) || !std::isfinite(route_scale))
    return SWIGLU_ERR_INVALID_ARG;
  if (T == 0) return SWIGLU_OK;
  if ((st = check_ptrs({X, Wr, idx, weights})) != SWIGLU_OK) return st;
  return run_route(X, Wr, idx, weights, (int)T, (int)D, (int)E, topk, norm_topk, route_scale, dtype,
                   nullptr, static_cast<cudaStream_t>(stream));
}

swiglu_status swiglu_mlp_moe_experts(const void* X, const int32_t* idx, const float* weights,
                                     const void* Wgu, const void* Wd, void* Y, int64_t T, int64_t D,
                                     int64_t H, int64_t E, int topk,
                                     const swiglu_mlp_w4_format* format, swiglu_dtype dtype,
                                     const swiglu_mlp_options* options, void* ws, size_t ws_bytes,
                                     void* stream) {
  host::reset_launches();
  Muls mu;
  swiglu_status st = read_muls(options, &mu);
  if (st != SWIGLU_OK) return st;
  if ((st = check_moe(T, D, H, E, topk, format, dtype)) != SWIGLU_OK) return st;
  if ((st = check_ws(ws, ws_bytes, swiglu_mlp_moe_workspace_bytes(T, D, H, E, topk))) != SWIGLU_OK)
    return st;
  if (T == 0) return SWIGLU_OK;
  if ((st = check_ptrs({X, idx, weights, Wgu, Wd, Y})) != SWIGLU_OK) return st;
  return run_experts(X, idx, weights, Wgu, Wd, Y, (int)T, (int)D, (int)H, (int)E, topk, format, dtype,
                     mu, static_cast<char*>(ws), ws_bytes, false, static_cast<cudaStream_t>(stream));
}

swiglu_status swiglu_mlp_moe_fwd_nograd(const void* X, const void* Wr, const void* Wgu,
                                        const void* Wd, void* Y, int32_t* idx, float* weights,
                                        int64_t T, int64_t D, int64_t H, int64_t E, int topk,
                                        int norm_topk, float route_scale,
                                        const swiglu_mlp_w4_format* format, swiglu_dtype dtype,
                                        const swiglu_mlp_options* options, void* ws,
                                        size_t ws_bytes, void* stream) {
  host::reset_launches();
  Muls mu;
  swiglu_status st = read_muls(options, &mu);
  if (st != SWIGLU_OK) return st;
  if ((st = check_moe(T, D, H, E, topk, format, dtype)) != SWIGLU_OK) return st;
  if ((norm_topk != 0 && norm_topk != 1) || !std::isfinite(route_scale))
    return SWIGLU_ERR_INVALID_ARG;
  if ((st = check_ws(ws, ws_bytes, swiglu_mlp_moe_workspace_bytes(T, D, H, E, topk))) != SWIGLU_OK)
    return st;
  if (T == 0) return SWIGLU_OK;
  if ((st = check_ptrs({X, Wr, Wgu, Wd, Y, idx, weights})) != SWIGLU_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = run_route(X, Wr, idx, weights, (int)T, (int)D, (int)E, topk, norm_topk, route_scale, dtype,
                 static_cast<int*>(ws), s);
  if (st != SWIGLU_OK) return st;
  return run_experts(X, idx, weights, Wgu, Wd, Y, (int)T, (int)D, (int)H, (int)E, topk, format, dtype,
                     mu, static_cast<char*>(ws), ws_bytes, true, s);
}

}  // extern "C"
