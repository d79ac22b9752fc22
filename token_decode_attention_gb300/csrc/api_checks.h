// api_checks.h -- what the C entry points share: messages of a failure, and checks of
// pointers, strides and overlaps before anything is launched.
#pragma once

#include "dattn.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <exception>

#include "dattn_internal.h"

namespace {

inline int fail(int status, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return dattn::set_last_error(status, buf);
}

inline int fail_cuda(cudaError_t e, const char *what) {
    return fail(DATTN_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

// No C++ exception leaves a C entry point (host memory may run out).
template <typename F>
int guarded(F f) noexcept {
    try {
        return f();
    } catch (const std::exception &e) {
        try {
            return fail(DATTN_ERR_CUDA, "on the host: %s", e.what());
        } catch (const std::exception &) {  // the message's own memory
            return DATTN_ERR_CUDA;
        }
    }
}

inline int check_tensor(const void *p, const char *name) {
    if (p == nullptr) return fail(DATTN_ERR_INVALID_ARG, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) & 15u)
        return fail(DATTN_ERR_MISALIGNED, "%s is not 16-byte aligned", name);
    return DATTN_OK;
}

inline int check_words(const void *p, const char *name) {
    if (p == nullptr) return fail(DATTN_ERR_INVALID_ARG, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) & 3u)
        return fail(DATTN_ERR_MISALIGNED, "%s is not 4-byte aligned", name);
    return DATTN_OK;
}

// Elements from token to token: whole 16-byte vectors, rows that do not overlap.
inline int check_stride(long long stride, long long row, int elem_bytes, const char *name) {
    if (stride < row)
        return fail(DATTN_ERR_INVALID_ARG, "%s=%lld is below the %lld elements of a token", name,
                    stride, row);
    if (stride > (1LL << 40)) return fail(DATTN_ERR_INVALID_ARG, "%s=%lld is too large", name, stride);
    if (stride * elem_bytes % 16 != 0)
        return fail(DATTN_ERR_MISALIGNED, "%s=%lld: a token must start on a 16-byte boundary", name,
                    stride);
    return DATTN_OK;
}

// Two arrays of `tokens` rows of `row` bytes, xs and ys apart, that are either the same
// rows or share no byte (slices of one projection lie in each other's gaps).
inline int check_overlap(const void *x, const void *y, long long tokens, long long row, long long xs,
                  long long ys, const char *names) {
    if (tokens > (1LL << 60) / std::max(xs, ys))
        return fail(DATTN_ERR_INVALID_ARG, "%s: the strides are too large", names);
    const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
    if (a == b && (xs == ys || tokens == 1)) return DATTN_OK;
    const uintptr_t ax = static_cast<uintptr_t>((tokens - 1) * xs + row);
    const uintptr_t by = static_cast<uintptr_t>((tokens - 1) * ys + row);
    if (a + ax <= b || b + by <= a) return DATTN_OK;
    const uintptr_t step = static_cast<uintptr_t>(xs), width = static_cast<uintptr_t>(row);
    const uintptr_t r = (a > b ? a - b : b - a) % step;
    if (xs == ys && r >= width && step - r >= width) return DATTN_OK;
    return fail(DATTN_ERR_INVALID_ARG, "%s overlap without being the same tensor", names);
}

}  // namespace
