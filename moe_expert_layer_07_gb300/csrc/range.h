// NVTX ranges of the entry points.
#pragma once

#include <nvtx3/nvToolsExt.h>

namespace moe {

// An NVTX range around each entry point (and each step of the layer call),
// so that a profiler's timeline names the library's calls; without a tool
// attached a push/pop is a call to an empty function.
struct Range {
    explicit Range(const char *name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
    Range(const Range &) = delete;
    Range &operator=(const Range &) = delete;
};

}  // namespace moe
