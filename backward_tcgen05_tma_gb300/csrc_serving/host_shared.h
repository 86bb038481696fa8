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

// Kernel ids of the per-kernel timing (swiglu_mlp_profile_read), after those
// of the training and dense no-grad kernels.
enum ServingKernel : int {
  SK_W4_LINEAR = 0, SK_W4_GATE_UP, SK_W4_DOWN, SK_MOE_ROUTE, SK_MOE_GATE_UP, SK_MOE_DOWN,
  SK_MOE_W4_GATE_UP, SK_MOE_W4_DOWN, SK_COUNT
};

uint64_t wait_limit_ns();
bool take_stall();       // true for the launch that swiglu_mlp_inject_stall_once chose
void reset_launches();   // at the start of an entry point
void count_launch();
int sms();               // SMs of the current device
bool profiling();

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
  Prof(ServingKernel id, cudaStream_t st);
  ~Prof();
  Prof(const Prof&) = delete;
  Prof& operator=(const Prof&) = delete;

 private:
  cudaStream_t st_;
  cudaEvent_t end_ = nullptr;
};

#ifdef SWIGLU_DEBUG
DbgWin windows(std::initializer_list<std::pair<const void*, size_t>> wins);
#endif

}  // namespace host
}  // namespace swiglu
