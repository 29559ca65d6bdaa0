// fs_host.hpp -- host-side error handling shared by the entry points' translation
// units (defined in fs_api.hip, which also holds the thread's last message).
// Not installed; not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/flashsample.h"

namespace fs {

// Records the formatted message for fs_last_error() and returns `s`.
fs_status fail(fs_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
fs_status hip_fail(hipError_t e, const char* what);

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A launch holds fewer than 2^32 threads along a dimension of its grid.  The entry
// points refuse what would take more before anything runs.
inline bool grid_fits(int64_t blocks, int64_t threads) { return blocks <= 0xFFFFFFFFll / threads; }

// Testing hook for failure handling: with FS_FAULT_INJECT=launch in the
// environment, every entry point that would launch device work returns
// FS_ERR_HIP once its arguments have passed the checks, before its first
// launch, with the reason in fs_last_error(): the path a failed launch
// takes, without a device and without launching anything.
fs_status injected_failure(const char* who);

// Called by every launching entry point once its arguments have passed the
// checks, just before its first HIP call; true when a failure is to be
// injected (and then no HIP call is made).  HIP keeps one pending error per
// host thread: any failed runtime call sets it, and the next hipGetLastError()
// returns and clears it.  The launchers read it right after each launch, so an
// error left pending by an earlier call (the caller's, or one of this
// library's that has already returned its own status) is discarded here
// rather than reported again against this call's launches.
bool start_launches();

}  // namespace fs
