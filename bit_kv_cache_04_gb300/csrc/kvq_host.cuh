// Host helpers shared by the C ABI's translation units (defined in
// kvq_api.cu): error reporting, configuration checks and the derived layout.
#pragma once

#include <stddef.h>

#include "kvq_internal.cuh"

namespace kvq {

// Sets the thread's error message and returns `st`.
kvq_status fail(kvq_status st, const char* fmt, ...);
// Clears the thread's error message.
kvq_status ok();
kvq_status cuda_fail(cudaError_t e, const char* what);

kvq_status check_config(const kvq_config* c, bool allow16);
Layout make_layout(const kvq_config* c);
kvq_status cache_ptrs(const kvq_config* c, const kvq_cache* cache, CachePtrs* cp);
// Streaming multiprocessors of the current device (a GB300's count without one).
int sm_count();
size_t align_up(size_t x);
// Polls of the failure-detection test mode (kvq_test_force_stall), 0 = off.
int stall_polls();

}  // namespace kvq
