// spec_host.cuh -- what the host side of every entry point shares: the error
// text of a call, and where an array lives.
#pragma once

#include <cuda_runtime.h>

#include "../../include/spec_verify.h"

namespace spec {

// records the thread's error text and returns `s`
spec_status fail(spec_status s, const char* fmt, ...);
spec_status cuda_fail(cudaError_t e, const char* where);

// Where an array lives.  Device (and managed) memory is used as it is;
// pinned host memory is read and written in place through its mapping into
// the device's address space (on a Grace host, over the NVLink-C2C link);
// pageable host memory cannot be reached by the kernels and is refused.
template <class T>
spec_status map_ptr(const char* who, const char* name, T*& p) {
    if (!p) return SPEC_OK;
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        cudaGetLastError();
        return fail(SPEC_INVALID_ARG, "%s: %s is not memory the device can reach", who, name);
    }
    if (a.type == cudaMemoryTypeDevice || a.type == cudaMemoryTypeManaged) return SPEC_OK;
    if (a.type == cudaMemoryTypeHost && a.devicePointer) {
        p = static_cast<T*>(a.devicePointer);
        return SPEC_OK;
    }
    return fail(SPEC_INVALID_ARG, "%s: %s is pageable host memory (pass device memory or pinned host memory)", who,
                name);
}
#define SPEC_MAP(x)                                              \
    do {                                                         \
        const spec_status map_s_ = ::spec::map_ptr(who, #x, x); \
        if (map_s_ != SPEC_OK) return map_s_;                    \
    } while (0)

// The workspace holds the kernels' queues, flags and partial results: it must
// be device memory.
inline spec_status ws_on_device(const char* who, const void* ws) {
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, ws) != cudaSuccess || a.type != cudaMemoryTypeDevice) {
        cudaGetLastError();
        return fail(SPEC_INVALID_ARG, "%s: the workspace must be device memory", who);
    }
    return SPEC_OK;
}
#define SPEC_WS_DEVICE(w)                                        \
    do {                                                         \
        const spec_status ws_s_ = ::spec::ws_on_device(who, w); \
        if (ws_s_ != SPEC_OK) return ws_s_;                      \
    } while (0)

}  // namespace spec
