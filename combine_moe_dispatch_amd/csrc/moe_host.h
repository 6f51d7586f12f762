// Host helpers shared by the C entry points (moe_ep.hip, moe_ops.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <rocprofiler-sdk-roctx/roctx.h>

#include "moe_ep.h"

namespace moe {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int from_hip(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// A ROCTX range around one call of the C ABI (shown by rocprofv3
// --marker-trace; a few tens of nanoseconds when no tool listens).
struct CallRange {
    explicit CallRange(const char* name) { roctxRangePushA(name); }
    ~CallRange() { roctxRangePop(); }
    CallRange(const CallRange&) = delete;
    CallRange& operator=(const CallRange&) = delete;
};

}  // namespace moe
