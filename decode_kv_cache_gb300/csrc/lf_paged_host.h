// Checks of arguments that the paged entry points share (host side; lf_paged.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "lf_paged.h"
#include "longflow.h"

namespace lf {

// Set the thread's last error; both return the code that the entry point returns.
int fail(int code, const char* fmt, ...);
int cuda_fail(cudaError_t e, const char* what);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline int elem_bytes(const lf_pages* p) { return p->dtype == LF_BF16 ? 2 : 4; }

// The pools, the page table and the lengths of a call, checked, as the kernels take them.
int take_pool(const lf_pages* p, int batch, const int32_t* table, int max_pages, const int32_t* lens,
              PagedPool* out);
// Query heads of a KV head.
int take_heads(const lf_pages* p, int q_heads, int* group);
// Streaming multiprocessors of the current device.
int sm_count(int* sms);

}  // namespace lf
