// What the files of extern "C" entry points share: the NVTX range of a call
// and the alignment check of its pointers.
#pragma once

#include <nvtx3/nvToolsExt.h>
#include <stdint.h>

namespace gdn {

// An NVTX range over the enclosing scope.
struct Range {
    explicit Range(const char *name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
    Range(const Range &) = delete;
    Range &operator=(const Range &) = delete;
};

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace gdn
