// hc_kv.cuh -- the paged cache's addressing and number formats, shared by the
// kernels that write, read, move and attend over it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "hc_spec.h"
#include "ptx.cuh"

namespace tshc {

constexpr int kKvBf16 = 0, kKvFp8 = 1, kKvInt4 = 2;  // ts_kvtype
constexpr unsigned kStatusBadArg = 1u;               // TS_ERR_INVALID_ARG of ts_hc.h

// Page of position pos of sequence b, or -1 (out of the table, or not a page). Only the page table is loaded
// as read-only data: no kernel of the library writes it, and one that does launches no dependent before it ends.
// (Ordinary loads are not moved ahead of the waits: 4 x 64 rows over 65536 FP8 keys 108 us, 119 with them.)
__device__ __forceinline__ long kv_page(const KvView &c, int b, long pos)
{
    const long i = pos >> c.page_shift;
    if (pos < 0 || i >= c.max_pages)
        return -1;
    const int id = __ldg(c.pages + (size_t)b * c.max_pages + i);
    return id >= 0 && id < c.n_pages ? id : -1;
}

// Row index (of rows of all pages) of position pos in page `page`, head h. The
// pool may hold more than 2^31 elements: 64-bit throughout.
__device__ __forceinline__ size_t kv_row(const KvView &c, long page, int h, long pos)
{
    return (((size_t)page * c.heads + h) << c.page_shift) + (size_t)(pos & ((1l << c.page_shift) - 1));
}

// A row that held an infinity or a NaN (FP8).
constexpr int kFp8BadRow = 255;

// The byte of the largest scale, 2^120, whose code 256 would be 2^128, more than a bf16 holds: elements
// that would round to it are held back to 240 2^120, the bf16 with these bits (off by 2^-4 of themselves
// at most, as e4m3 is elsewhere).
constexpr int kFp8TopRow = 247;
constexpr uint32_t kFp8TopBits = 0x7F70u;

// The scale byte of a row with finite maximum amax: the smallest e >= -117 with
// amax <= 448 * 2^e, plus 127. From the bits: 448 = 1.75 * 2^8. At e >= -117 the
// smallest code, 2^-9 * 2^e, is a normal bf16, so that rows read back exactly.
__device__ __forceinline__ int fp8_scale_byte(float amax)
{
    const uint32_t u = __float_as_uint(amax);
    const int k = (int)(u >> 23) - 127;  // amax = m * 2^k, 1 <= m < 2 (a denormal's k is low enough to be clamped)
    const int e = k - ((u & 0x7FFFFFu) <= 0x600000u ? 8 : 7);
    return max(e, -117) + 127;
}

// 2^(byte - 127) for byte in [1, 254]; NaN for a bad row.
__device__ __forceinline__ float fp8_scale(int byte) { return __uint_as_float(byte == kFp8BadRow ? 0x7FC00000u : (uint32_t)byte << 23); }

__device__ __forceinline__ bool finite_f32(float x) { return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u; }

}  // namespace tshc
