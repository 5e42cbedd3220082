// api_util.cuh -- host helpers shared by the files that define the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>
#include <stdint.h>

#include "../../include/up.h"

namespace up {

// A named NVTX range around each public call's host work (argument checks and
// launches), so a timeline profiler shows the calls of a step; without a
// profiler attached a push or pop is a check of a null hook.
struct CallRange {
    explicit CallRange(const char *name) { nvtxRangePushA(name); }
    ~CallRange() { nvtxRangePop(); }
    CallRange(const CallRange &) = delete;
    CallRange &operator=(const CallRange &) = delete;
};

inline size_t align256(size_t v) { return (v + 255) & ~size_t(255); }
inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// SM count and error word of the current device, and the bound of the kernels'
// spin-waits (see up_set_wait_limit).
struct DeviceInfo {
    int sms;
    unsigned int *err;
    long long wait_limit;
};
up_status device_info(DeviceInfo *out);

}  // namespace up
