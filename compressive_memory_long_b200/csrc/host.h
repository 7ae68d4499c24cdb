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

// Reads and clears the current device's record of bad page numbers: 0 none, 1 some, -1 if
// the copy failed.
int take_page_status();

}  // namespace infini
