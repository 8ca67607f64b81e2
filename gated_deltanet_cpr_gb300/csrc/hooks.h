// hooks.h -- the profiling hook, the wait-timeout test hook and the NVTX ranges of the C-ABI entry points.
#pragma once

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "../../include/gdn_cpr.h"

namespace gdn {

// set by gdn_cpr_set_profile for the calling thread
extern thread_local gdn_cpr_profile* t_profile;
// set by gdn_cpr_test_wait_timeout for the calling thread: calls left whose first CTA gives up a wait
// that nothing completes
extern thread_local int32_t t_wait_fault;
// one such call, where it has a wait to give up
inline int take_wait_fault(bool has_one) {
  if (!has_one || t_wait_fault <= 0) return 0;
  --t_wait_fault;
  return 1;
}

// NVTX range over one entry point (host-side markers for profilers such as Nsight; no
// effect without a tool attached).
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

// Stage boundaries of one call: the profiling hook's events and kernel counts, and a nested
// NVTX range per stage (names[i] is stage i + 1; NULL-terminated).
struct Stages {
  cudaStream_t st;
  const char* const* names;
  int next = 0;
  bool open = false;
  Stages(cudaStream_t s, const char* const* stage_names) : st(s), names(stage_names) {
    if (t_profile) t_profile->stages = 0;
    mark(0);
  }
  ~Stages() {
    if (open) nvtxRangePop();
  }
  Stages(const Stages&) = delete;
  Stages& operator=(const Stages&) = delete;
  // a kernel launched at the start of the first stage (counted, no event of its own)
  void count(int kernels) {
    if (t_profile) t_profile->kernels += kernels;
  }
  void mark(int kernels) {
    if (open) nvtxRangePop();
    open = names && names[next] != nullptr;
    if (open) nvtxRangePushA(names[next]);
    if (!t_profile) {
      ++next;
      return;
    }
    t_profile->kernels += kernels;
    if (next < t_profile->n_events && next < 16 && t_profile->events[next]) {
      cudaEventRecord(static_cast<cudaEvent_t>(t_profile->events[next]), st);
      t_profile->stages = next + 1;
    }
    ++next;
  }
};

}  // namespace gdn
