// ts_hc_checks.h -- argument checks that the entry points of the decoding step
// and of the prompt operators share. Internal to the library.
#pragma once

#include "hc_kernels.h"
#include "ts_hc_internal.h"

#define TS_TRY(expr)                      \
    do {                                  \
        const ts_status st_ = (expr);     \
        if (st_ != TS_OK)                 \
            return st_;                   \
    } while (0)

namespace tshc {

constexpr int kMaxHeads = 1024;
constexpr int kMaxBatch = 65535;

inline ts_status check_count(int v, const char *name, int lo, int hi)
{
    if (v < lo || v > hi)
        return api_error(TS_ERR_INVALID_ARG, "%s = %d must be in [%d, %d]", name, v, lo, hi);
    return TS_OK;
}

inline ts_status check_stride(long stride, const char *name, long least, long multiple)
{
    if (stride < least || stride % multiple != 0)
        return api_error(TS_ERR_INVALID_ARG, "%s = %ld must be a multiple of %ld and >= %ld", name, stride, multiple, least);
    return TS_OK;
}

inline ts_status device(LaunchCfg *cfg, unsigned **status)
{
    cfg->pdl = true;
    return device_api(&cfg->sm_count, status);
}

inline ts_status launched(cudaError_t e, const char *what) { return e == cudaSuccess ? TS_OK : cuda_error(e, what); }

// Whether [a, a + na) and [b, b + nb) (bytes) share one.
inline bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// Whether n rows of wa 16-bit elements at a + i*sa and n rows of wb at b + i*sb
// share one. Exact for equal strides (slices of one projection's output are
// disjoint), by the address ranges otherwise.
inline bool rows_overlap(const void *a, long sa, long wa, const void *b, long sb, long wb, int n)
{
    if (!overlap(a, 2 * ((size_t)(n - 1) * sa + wa), b, 2 * ((size_t)(n - 1) * sb + wb)))
        return false;
    const intptr_t bytes = reinterpret_cast<intptr_t>(b) - reinterpret_cast<intptr_t>(a);
    if (sa != sb || bytes % 2 != 0)
        return true;
    const long m = ((long)(bytes / 2) % sa + sa) % sa;
    return !(m >= wa && m + wb <= sa);
}

}  // namespace tshc
