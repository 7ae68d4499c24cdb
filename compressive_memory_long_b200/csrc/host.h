// Host-side helpers shared by the library's translation units.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace infini {

// One traced launch: events around the kernel while tracing is enabled (nothing otherwise).
class TraceScope {
public:
    TraceScope(const char *name, cudaStream_t st);
    ~TraceScope();
    TraceScope(const TraceScope &) = delete;
    TraceScope &operator=(const TraceScope &) = delete;

private:
    void *rec_ = nullptr;
};

// Reads the current device's records of the paged entries: a bounded wait that gave up, and page
// numbers or rows outside a cache.  Clears the first, and the second unless a wait is to be reported
// before it (`waits` on entry: one of another unit).  INFINI_OK, or INFINI_ERR_CUDA if a copy failed.
int take_paged_status(bool &waits, bool &pages);

// The bound of the paged entries' device waits, in SM cycles.
int set_paged_wait_limit(long long cycles);

// Whether the eviction's fold withholds its first loader warp's stages (a test hook).
int set_paged_withhold(int on);

}  // namespace infini
