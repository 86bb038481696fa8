// host_shared.h -- the process-wide host state of the library (wait limit,
// stall injection, launch count, per-kernel timing, debug windows), defined in
// csrc/swiglu_mlp.cu and used by every translation unit that launches kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <initializer_list>
#include <utility>

#include "../csrc/sm103_ptx.cuh"

namespace swiglu {
namespace host {

// Kernel ids of the per-kernel timing (swiglu_mlp_profile_read).
enum KernelId : int {
  K_GATE_UP = 0, K_DOWN, K_DGU, K_DWD, K_DWGU, K_DX, K_GATE_UP_NOGRAD, K_DOWN_NOGRAD,
  K_SIMT_GATE_UP, K_SIMT_DOWN, K_SIMT_DGU, K_SIMT_DWD, K_SIMT_DWGU, K_SIMT_DX, K_NG_GATE_UP,
  K_NG_DOWN, K_NG_FUSED,
  // few-token serving
  SK_W4_LINEAR, SK_W4_GATE_UP, SK_W4_DOWN, SK_MOE_ROUTE, SK_MOE_GATE_UP, SK_MOE_DOWN,
  SK_MOE_W4_GATE_UP, SK_MOE_W4_DOWN,
  // layer norm and linear
  K_LN, K_DLN, K_LINEAR, K_LINEAR_FEW, K_SIMT_LINEAR, K_DACT, K_COLUMN_SUMS, K_LINEAR_DW,
  K_LINEAR_DX, K_SIMT_LINEAR_DW, K_SIMT_LINEAR_DX,
  K_COUNT
};
using ServingKernel = KernelId;

uint64_t wait_limit_ns();
bool take_stall();       // true for the launch that swiglu_mlp_inject_stall_once chose
void reset_launches();   // at the start of an entry point
void count_launch();
int sms();               // SMs of the current device
bool profiling();
int cta_pairs();         // swiglu_mlp_set_cta_pairs, swiglu_mlp_set_wide_tiles
int wide_tiles();
// Pairs of SMs that can hold a pair kernel's cluster at once (each TPC whose
// two SMs are both usable), queried once per device.
int pair_units();

// The plain GEMMs of a backward pass over M tokens, bf16 or fp16: dW [N, K] =
// G^T X, or with `accumulate` dW + that product; dX [M, K] = G W.  G [M, N], X
// [M, K] and W [N, K] are contiguous; err: the workspace, whose error word the
// `first` kernel of a call clears and whose counters are zero between kernels.
cudaError_t gemm_dw(int id, bool bf16, const void* G, const void* X, void* dW, int64_t M, int64_t N,
                    int64_t K, int accumulate, int* err, size_t ws_bytes, bool first, cudaStream_t st);
cudaError_t gemm_dx(int id, bool bf16, const void* G, const void* W, void* dX, int64_t M, int64_t N,
                    int64_t K, int* err, size_t ws_bytes, bool first, cudaStream_t st);

// Tensor map of a 16-bit array [n2][n1][n0] (n0 contiguous) with boxes of
// b2 x b1 x b0 elements, 128-byte swizzle; elements outside read as 0.
bool encode_3d(CUtensorMap* tm, bool bf16, const void* base, int64_t n0, int64_t n1, int64_t n2,
               int b0, int b1, int b2);
// The same array [rows][K], K a multiple of 64, seen as [K / 64][rows][64]:
// boxes of `blocks` 64-element blocks of `brows` rows.
bool encode_blocks(CUtensorMap* tm, bool bf16, const void* base, int64_t K, int64_t rows, int brows,
                   int blocks);
// Records of `record` bytes (a multiple of 16), [n2][n1] of them, with boxes of
// b2 x b1 records, no swizzle.
bool encode_records(CUtensorMap* tm, const void* base, int record, int64_t n1, int64_t n2, int b1,
                    int b2);

// Brackets one launch with events while per-kernel timing is enabled.
class Prof {
 public:
  Prof(int id, cudaStream_t st);
  ~Prof();
  Prof(const Prof&) = delete;
  Prof& operator=(const Prof&) = delete;

 private:
  cudaStream_t st_;
  cudaEvent_t end_ = nullptr;
};

#ifdef SWIGLU_DEBUG
DbgWin windows(std::initializer_list<std::pair<const void*, size_t>> wins);
DbgWin windows(const std::pair<const void*, size_t>* wins, int n);
#endif

}  // namespace host
}  // namespace swiglu
