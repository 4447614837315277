// Host-side helpers of the C ABI, shared by the files that implement it:
// error texts, argument checks and the calling thread's device (ep_api.hip).
#pragma once

#include "ep_internal.hpp"

namespace ep {

// Stores the message for ep_last_error() and returns `code`.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int hip_fail(hipError_t e, const char* what);

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The calling thread's device, checked to be a gfx950, with the compute units
// that `stream` may use, the budget and the slab setting.
int current_device(Budget* b, void* stream);

// T and k, and T * k against EP_MAX_ENTRIES.
int check_common(int T, int k, int H_or_E, const char* what);
// H in whole 16-byte bf16 vectors, recv_rows, and both row counts in slabs.
int check_rows(int H, int64_t recv_rows, int T, const char* what);

}  // namespace ep
