// host.h -- what the files that implement the C ABI share: the thread's last
// error, argument checks, stream-capture state, the launch counter, and a launch
// that reads a resident RoPE table.  Defined in tf_ulysses.cpp.
#pragma once

#include <cstddef>
#include <cstdint>
#include <functional>

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "tf_ulysses.h"

namespace tfu {
namespace host {

// A named NVTX range around each C-ABI call, so that a profiler's timeline shows
// which library call issued which launches (header-only NVTX; a few nanoseconds
// when no profiler is attached).
struct CallRange {
    explicit CallRange(const char* name) { nvtxRangePushA(name); }
    ~CallRange() { nvtxRangePop(); }
    CallRange(const CallRange&) = delete;
    CallRange& operator=(const CallRange&) = delete;
};

// Set the calling thread's last error and return `s`.
tf_status fail(tf_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
tf_status cuda_fail(cudaError_t e, const char* what);

tf_status capture_state(cudaStream_t s, bool* capturing);
tf_status current_device(int* dev);

int elem_size(tf_dtype d);  // bytes; 0 for an unknown type
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// P pointers that are not NULL and 16-byte aligned
tf_status check_ptrs(const char* what, const void* const* a, int P);
// strides of a [nb, nt, nh, D] view; a stride of an extent-1 dimension is never used
tf_status check_strides(const char* what, const tf_strides& s, int esize, int64_t nb, int64_t nt, int64_t nh);

// P pointers under a name
struct Named {
    const char* name;
    const void* const* at;
};
// Refuses written tensors that start where one that is read, or another written one, does.  in_place: written tensor x may be
// tensor x of those read, group by group.
tf_status check_starts(const Named* written, int n_written, const Named* read, int n_read, int P, bool in_place);

// scale and cap of attention scores
tf_status check_scores(float scale, float softcap);

void count_launches(int n);
uint64_t launch_count();
const char* last_error();

// Calls `launch` with the resident RoPE table of (theta, S rows, D), built on
// `stream` first if there is none, and marks the table's use in stream order.
tf_status with_rope_table(float theta, int S, int D, cudaStream_t stream,
                          const std::function<cudaError_t(const float*)>& launch);

}  // namespace host
}  // namespace tfu
