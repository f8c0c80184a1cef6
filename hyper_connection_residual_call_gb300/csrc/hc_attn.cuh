// hc_attn.cuh -- what the tree attention's kernels share: how the work is cut
// over the CTAs, where partial results lie, and which nodes a row sees.
//
// An item is one (sequence, key head, block of rows): its keys in tiles, all
// with the same softmax rows. The items' tiles form one line of N, in the order
// sequence, head, row block, tile, which is cut into one run for each of G CTAs: the
// first N mod G of them take N / G + 1 tiles and the others N / G (Cut::first is where
// CTA c's run begins, Cut::cta_of whose run holds a tile). So every CTA has the same
// number of tiles, to one, whatever the sequences' lengths are, and a long context is
// split over as many CTAs as it takes. An item that lies within one CTA is written to the
// output by it; the segments of the others go to the workspace, at most two
// for a CTA (its first and its last item), and a second kernel joins them in
// CTA order, so the result does not depend on timing.
#pragma once

#include "hc_kv.cuh"

namespace tshc {

constexpr int kAttnMaxGrid = 4 * 152;  // CTAs that can write partials (a launch takes at most this many)
constexpr int kAttnWideGrid = 160;     // the same for the wide kernel, one CTA an SM
constexpr int kAttnThreads = 128;

// Tiles of sequence b's items and its keys. A length that does not fit the page
// table is cut to it (and recorded by the caller).
struct SeqLen {
    int ctx, keys, tiles;
    bool bad;
};

// kFromL2: not from L1, for the join, which reads the lengths before its wait.
template <bool kFromL2 = false>
__device__ __forceinline__ SeqLen attn_seq(const AttnParams &p, int b, int tile)
{
    SeqLen s;
    const long cap = (long)p.c.max_pages << p.c.page_shift;
    const int raw = kFromL2 ? __ldcg(p.ctx_len + b) : p.ctx_len[b];
    s.ctx = (int)max(0l, min((long)raw, cap));
    const long keys = min((long)s.ctx + p.T, cap);
    s.bad = raw < 0 || (long)raw + p.T > cap;
    s.keys = (int)keys;
    s.tiles = (int)((keys + tile - 1) / tile);
    return s;
}

constexpr int kAttnMaxWarps = 16;

struct LineScratch {
    long warp_sum[kAttnMaxWarps];
    long base;
    int b;
};

// The line, scanned by all threads of a block (kAttnThreads at least, whose first
// kAttnThreads each take a run of sequences [b0, b1)): `total` tiles.
template <bool kFromL2 = false>
struct Line {
    long total, base, sum, per;
    int b0, b1;

    __device__ __forceinline__ Line(const AttnParams &p, int tile, LineScratch &sc)
    {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        const int chunk = (p.B + kAttnThreads - 1) / kAttnThreads;
        per = (long)p.c.heads * p.row_blocks;
        b0 = min(p.B, tid * chunk);
        b1 = min(p.B, b0 + chunk);
        sum = 0;
#pragma unroll 1
        for (int b = b0; b < b1; ++b)
            sum += attn_seq<kFromL2>(p, b, tile).tiles * per;
        long incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o)
                incl += v;
        }
        if (lane == 31)
            sc.warp_sum[warp] = incl;
        __syncthreads();
        long before = 0;
        total = 0;
#pragma unroll
        for (int w = 0; w < kAttnThreads / 32; ++w) {  // further warps have no sequences
            if (w < warp)
                before += sc.warp_sum[w];
            total += sc.warp_sum[w];
        }
        base = before + incl - sum;
    }

    // The sequence whose tiles hold x (x < total), in sc.b, and the line's index
    // of its first tile, in sc.base.
    __device__ __forceinline__ void find(const AttnParams &p, int tile, long x, LineScratch &sc) const
    {
        if (x >= base && x < base + sum) {  // one thread
            long at = base;
            int b = b0;
#pragma unroll 1
            for (; b + 1 < b1; ++b) {
                const long n = attn_seq<kFromL2>(p, b, tile).tiles * per;
                if (x < at + n)
                    break;
                at += n;
            }
            sc.base = at;
            sc.b = b;
        }
        __syncthreads();
    }
};

// a / b for a >= 0, b > 0, in 32 bits where they fit: the call's start is a chain of such steps.
__device__ __forceinline__ long attn_div(long a, long b) { return (a | b) <= 0x7FFFFFFF ? (long)((unsigned)a / (unsigned)b) : a / b; }

// CTAs that take part: none has fewer than `least` tiles but the only one.
__device__ __forceinline__ int attn_ctas(long n, int grid, int least)
{
    return (int)max(1l, min((long)grid, attn_div(n, least)));
}

// How the line is cut: the first `more` CTAs have share + 1 tiles, the others share.
struct Cut {
    long share, more;
    __device__ __forceinline__ Cut(long n, int ctas) : share(attn_div(n, ctas)), more(n - share * ctas) {}
    __device__ __forceinline__ long first(int c) const { return c * share + min((long)c, more); }
    // The CTA whose range holds tile x.
    __device__ __forceinline__ int cta_of(long x) const
    {
        const long big = more * (share + 1);
        return x < big ? (int)attn_div(x, share + 1) : (int)(more + attn_div(x - big, share));
    }
};

// A CTA's items in turn: the tiles [t0, t1) of one item each.
struct Items {
    long at, end, first, base;
    long from;                // the line's index of this segment's first tile
    int b, head, block, t0, t1;
    SeqLen seq;

    // (Inlined in each role: 4 x 64 rows over 32768 bf16 keys take 80 us, and 87 with a function that is called.)
    __device__ __forceinline__ bool next(const AttnParams &p, int tile)
    {
        while (at < end) {
            seq = attn_seq(p, b, tile);
            const long span = (long)seq.tiles * p.c.heads * p.row_blocks;
            if (at >= base + span) {
                base += span;
                ++b;
                continue;
            }
            const long in = at - base;
            const int item = span <= 0x7FFFFFFF ? (int)in / seq.tiles : (int)(in / seq.tiles);
            t0 = (int)(in - (long)item * seq.tiles);
            head = item / p.row_blocks;
            block = item - head * p.row_blocks;
            t1 = (int)min((long)seq.tiles, t0 + (end - at));
            from = at;
            at += t1 - t0;
            return true;
        }
        return false;
    }
    // Whether the segment is all of its item, and if not, which of the CTA's two slots it takes.
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == seq.tiles; }
    __device__ __forceinline__ int slot() const { return from > first ? 1 : 0; }
};

// How far below a row's maximum the reference of its weights is kept (log2), where they are held in fp16: at
// 2^6 of themselves and more, weights of 2^-20 of the largest and up are normal numbers, and smaller ones are off by
// 2^-31 of it at most. (With the maximum as the reference those below 2^-25 were nothing in the products.) The
// reference moves when the maximum has grown by 2^8 more, so that a weight is at most 2^14, and an infinity in fp16
// only where scores are so large (2^25) that fp32 holds them to no better than a factor of 2 or so.
constexpr float kFp16Lift = 6.f;

// A partial slot: unnormalised sums [rows][D] (the wide kernel's [D / 4][rows][4]), then
// the rows' maxima (in units of log2) and sums.
__host__ __device__ __forceinline__ size_t attn_slot_floats(int rows, int D) { return (size_t)rows * (D + 2); }

// Whether node row t sees position ctx + i (i >= 0). (From L2: an ordinary load here, where it hardly ever
// runs, changes what the compiler makes of the few-row kernel's loop, 94 us to 96 for 2 x 12 rows over 131072 INT4 keys.)
__device__ __forceinline__ bool attn_sees(const AttnParams &p, const uint32_t *mask_row, int t, int i)
{
    if (i >= p.T)
        return false;
    return p.mask ? ((__ldcg(mask_row + (i >> 5)) >> (i & 31)) & 1u) != 0 : i <= t;
}

__device__ __forceinline__ const uint32_t *attn_mask_row(const AttnParams &p, int b, int t)
{
    return p.mask ? p.mask + (size_t)b * p.mask_stride + (size_t)t * p.mask_words : nullptr;
}

// One element of a stored value, as it would be read back (rare paths only).
__device__ __forceinline__ float kv_value_at(const KvView &c, size_t row, int d)
{
    if (c.type == kKvBf16)
        return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(c.v)[row * c.D + d] << 16);
    if (c.type == kKvFp8) {
        const __half_raw h = __nv_cvt_fp8_to_halfraw(c.v[row * c.D + d], __NV_E4M3);
        return __half2float(__half(h)) * fp8_scale(c.vs[row]);
    }
    const size_t g = row * (size_t)(c.D / c.group) + d / c.group;
    const int code = (c.v[row * (c.D / 2) + d / 2] >> (4 * (d & 1))) & 15;
    return fmaf((float)code, __half2float(reinterpret_cast<const __half *>(c.vs)[g]), __half2float(reinterpret_cast<const __half *>(c.vb)[g]));
}

// The sum of the infinities and NaNs among element d of the nodes' values that
// row t sees, for the nodes at positions [from, to) (0 where there are none).
// The kernels put zeros in the place of such values of nodes -- in a product, a
// zero weight would not keep them from the rows that do not see them -- and add
// this where one was found.
static __device__ __forceinline__ float attn_wild_values(const AttnParams &p, int b, int head, int t, int d, int ctx, int from, int to)
{
    const uint32_t *mask = attn_mask_row(p, b, t);
    float sum = 0.f;
    for (int pos = max(from, ctx); pos < to; ++pos) {
        if (!attn_sees(p, mask, t, pos - ctx))
            continue;
        const long page = kv_page(p.c, b, pos);
        if (page < 0)
            continue;
        const float v = kv_value_at(p.c, kv_row(p.c, page, head, pos), d);
        if (!finite_f32(v))
            sum += v;
    }
    return sum;
}

// Which of the 32 positions ctx + n0 .. ctx + n0 + 31 node row t sees (n0 may be
// negative: the context), bit i for ctx + n0 + i. The mask may have been written while this kernel was
// already launched and waiting, so its words are not loaded as read-only data. (Past L1 the softmax
// waits longer for them: 32 x 160 rows over 300 keys of 64, 45 us and 47.)
static __device__ __forceinline__ uint32_t attn_sees32(const AttnParams &p, const uint32_t *mask_row, int t, int n0, const SeqLen &seq)
{
    const auto low = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; };
    const uint32_t present = low(seq.keys - seq.ctx - n0);
    if (!p.mask)
        return low(t + 1 - n0) & present;
    const int w = n0 >> 5;
    const auto word = [&](int i) { return i < 0 ? 0xFFFFFFFFu : i < p.mask_words ? mask_row[i] & low(p.T - 32 * i) : 0u; };
    return __funnelshift_r(word(w), word(w + 1), n0 & 31) & present;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return reinterpret_cast<const uint32_t &>(v);
}

__device__ __forceinline__ uint32_t pack2_f16(float lo, float hi)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return reinterpret_cast<const uint32_t &>(v);
}

// INT4 codes of an 8-code word at bits 4 i and 16 + 4 i -> 16 + q, bf16x2 (exact): the
// code goes to mantissa bits 3-6 of 16.
template <int i>
__device__ __forceinline__ uint32_t int4_bf16x2(uint32_t w)
{
    constexpr int kShift = 3 - 4 * i;
    const uint32_t at = kShift > 0 ? w << (kShift > 0 ? kShift : 0) : w >> (kShift > 0 ? 0 : -kShift);
    return (at & 0x00780078u) | 0x41804180u;
}

// INT4 codes in bits 0-3 (kHigh: 4-7) of the two halves of w -> q * scale + bias, fp16x2.
template <bool kHigh>
__device__ __forceinline__ uint32_t int4_f16x2(uint32_t w, __half2 scale, __half2 bias)
{
    const uint32_t bits = (w & (kHigh ? 0x00F000F0u : 0x000F000Fu)) | 0x64006400u;  // 1024 + q, or 1024 + 16 q
    const __half2 at = reinterpret_cast<const __half2 &>(bits);
    const __half2 q = kHigh ? __hfma2(at, __half2half2(__ushort_as_half(0x2C00)), __half2half2(__ushort_as_half(0xD400)))  // / 16 - 64, exact
                            : __hsub2(at, __half2half2(__ushort_as_half(0x6400)));
    const __half2 v = __hfma2(q, scale, bias);
    return reinterpret_cast<const uint32_t &>(v);
}

// Once per kernel and device: raises the dynamic shared-memory limit to `smem` and finds how many CTAs of
// `threads` an SM holds. A failure is not remembered. (The largest carveout, which the other kernels of the
// library ask for, makes nothing faster here, and 4 x 512 rows over 16384 bf16 keys 0.7% slower: their shared
// memory leaves no room for another kernel's CTAs either way.)
cudaError_t attn_ready(const void *kernel, int threads, int smem, int *per_sm);
// The wide kernel's rows of a block (0: the few-row kernel serves) and its launcher.
int attn_wide_rows(const KvView &c, long rows);
cudaError_t launch_attn_wide(const AttnParams &p, const LaunchCfg &cfg, cudaStream_t stream);
// Joins the segments that either kernel left: blocks of `rows` rows, tiles of `tile` keys.
cudaError_t launch_attn_join(const AttnParams &p, int rows, int tile, int grid, int least, bool by_columns, cudaStream_t stream);

}  // namespace tshc
