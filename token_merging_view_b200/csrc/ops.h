// Host-side pieces shared by the operators around the layer (attention over
// key ranges, rotary positions, gated norms): error reporting, argument
// checks, and the state their kernels report through.
#pragma once
#include <cuda_runtime.h>

#include <atomic>

#include "../../include/httm.h"
#include "internal.h"

namespace httm {

// Defined with the plan's entry points: records a CUDA error for
// httm_last_cuda_error(); turns a launch error (and, with HTTM_SYNC_CHECK=1,
// a device fault) into a status.
httm_status cuda_fail(cudaError_t e, const char* where);
cudaError_t checked(cudaError_t e, cudaStream_t s);

// The operators' device state on the current device (nullptr on failure).
// Its status word gathers HTTM_DEV_* bits until httm_ops_device_status().
DevState* ops_state();

// SMs of a B200: sizes of grids and splits are chosen for it on the host, so
// that workspace sizes need no device.
constexpr int kSMs = 148;

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// One view with its extents, strides normalised: the stride of an extent of
// 1 is 0.
struct View {
  char* data;
  int64_t sb, sh, st;   // strides in elements over batch, heads, tokens
};

inline View normal_view(const httm_view& v, int64_t batch, int64_t heads, int64_t tokens) {
  return View{static_cast<char*>(v.data), batch > 1 ? v.batch : 0, heads > 1 ? v.head : 0, tokens > 1 ? v.token : 0};
}

// An output whose rows of `inner` channels overlap each other is refused:
// taken in order of stride, each stride must clear the extent of the
// smaller ones.  All strides are non-negative here.
inline bool disjoint(const View& v, int64_t batch, int64_t heads, int64_t tokens, int64_t inner) {
  int64_t st[3] = {v.sb, v.sh, v.st}, n[3] = {batch, heads, tokens};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (st[j] < st[i]) {
        int64_t t = st[i]; st[i] = st[j]; st[j] = t;
        t = n[i]; n[i] = n[j]; n[j] = t;
      }
  int64_t span = inner;
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;
    if (st[i] < span) return false;
    span += st[i] * (n[i] - 1);
  }
  return true;
}

// A kernel whose warps exchange registers (setmaxnreg) waits forever if it
// was launched with fewer than it hands out: checked against what the
// compiler gave it, until that once succeeded.
template <auto kKernel>
inline cudaError_t check_registers(int threads, int total) {
  static std::atomic<bool> enough{false};
  if (enough.load(std::memory_order_relaxed)) return cudaSuccess;
  cudaFuncAttributes at;
  const cudaError_t e = cudaFuncGetAttributes(&at, kKernel);
  if (e != cudaSuccess) return e;
  if (at.numRegs * threads < total) return cudaErrorInvalidConfiguration;
  enough.store(true, std::memory_order_relaxed);
  return cudaSuccess;
}

#define HTTM_TRY(expr)                   \
  do {                                   \
    const httm_status t_ = (expr);       \
    if (t_ != HTTM_OK) return t_;        \
  } while (0)

#define HTTM_OPS_LAUNCH(expr, s)                              \
  do {                                                        \
    const cudaError_t e_ = ::httm::checked((expr), (s));      \
    if (e_ != cudaSuccess) return ::httm::cuda_fail(e_, #expr); \
  } while (0)

}  // namespace httm
