// api_checks.h -- argument checks and error reporting shared by the C entry points
// outside moe_api.cu.
#pragma once

#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdio>

#include "../../include/moe.h"
#include "common.h"

namespace moe {

inline moe_status refuse(moe_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    set_error_detail(buf);
    return s;
}

inline moe_status launched(cudaError_t e, const char* where) {
    if (e == cudaSuccess) return MOE_OK;
    return refuse(MOE_ERR_CUDA, "%s: %s (%s)", where, cudaGetErrorName(e), cudaGetErrorString(e));
}

inline bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

#define NEED(p)                                                                            \
    do {                                                                                   \
        if ((p) == nullptr) return refuse(MOE_ERR_INVALID_ARG, "%s is NULL", #p);          \
        if (misaligned(p)) return refuse(MOE_ERR_INVALID_ARG, "%s not 16-byte aligned", #p); \
    } while (0)

#define MAY(p)                                                                             \
    do {                                                                                   \
        if ((p) != nullptr && misaligned(p))                                               \
            return refuse(MOE_ERR_INVALID_ARG, "%s not 16-byte aligned", #p);              \
    } while (0)

#define NEED_WS(bytes)                                                                     \
    do {                                                                                   \
        NEED(ws);                                                                          \
        const size_t need_ = (bytes);                                                      \
        if (ws_bytes < need_)                                                              \
            return refuse(MOE_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws_bytes, need_); \
    } while (0)

inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace moe
