// Argument checks shared by the host sides of the entry points.
#pragma once

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "kda_internal.cuh"

namespace kda {
namespace {

kda_status_t fail(kda_status_t st, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return set_error(st, buf);
}
kda_status_t ok() { return set_error(KDA_OK, ""); }
kda_status_t cuda_status(cudaError_t e, const char *what) {
    return e == cudaSuccess ? ok() : fail(KDA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}
bool aligned(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

#define KDA_CHECK(x)                                   \
    do {                                               \
        const kda_status_t st_ = (x);                  \
        if (st_ != KDA_OK) return st_;                 \
    } while (0)

kda_status_t need(const void *p, const char *name, uintptr_t align = 16) {
    if (!p) return fail(KDA_ERR_INVALID_ARG, "%s must not be NULL", name);
    if (!aligned(p, align)) return fail(KDA_ERR_INVALID_ARG, "%s must be %d-byte aligned", name, (int)align);
    return KDA_OK;
}
kda_status_t maybe(const void *p, const char *name, uintptr_t align = 16) {
    return p ? need(p, name, align) : KDA_OK;
}

// The distance between two tokens of a tensor in elements: 0 stands for the
// contiguous H * d; rows must start on 16 bytes and must not overlap.
kda_status_t stride(int64_t &s, int H, int d, kda_dtype_t dt, const char *name) {
    if (s == 0) s = (int64_t)H * d;
    const int per = dt == KDA_BF16 ? 8 : 4;
    if (s < (int64_t)H * d || s % per)
        return fail(KDA_ERR_INVALID_ARG, "%s must be 0 or at least H * d and a multiple of 16 bytes (got %lld)", name,
                    (long long)s);
    return KDA_OK;
}

// a * b * c <= INT32_MAX, for factors >= 0 whose product may not fit in 64 bits
bool fits(int64_t a, int64_t b, int64_t c = 1) {
    if (a == 0 || b == 0 || c == 0) return true;
    return a <= INT32_MAX && b <= INT32_MAX / a && c <= INT32_MAX / (a * b);
}

kda_status_t workspace_ok(const void *ws, size_t have, size_t want) {
    if (!want) return KDA_OK;
    if (!ws || have < want) return fail(KDA_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", want, have);
    if (!aligned(ws, 256)) return fail(KDA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    return KDA_OK;
}

}  // namespace
}  // namespace kda
