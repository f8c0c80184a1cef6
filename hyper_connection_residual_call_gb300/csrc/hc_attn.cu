// hc_attn.cu -- attention of a few drafted tokens (a chain or a tree) over the
// paged cache: blocks of 16 or 32 rows (ts_hc_tree_attention in include/ts_hc.h).
//
//   row (t, h) sees the committed keys and the nodes of its mask row;
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(x_j - m),  x_j = scale log2(e) q . k_j
//
// With T nodes and G query heads a key head an item has T*G rows that share one
// pass over the keys: 4 T G D flops for each key's row bytes, so that up to some
// 32 rows the operator is bound by the cache's bytes. The layout follows from
// that: each warp streams 16-key chunks of its own (every fourth of the line)
// through a ring of its own in shared memory (cp.async; nothing but __syncwarp
// between a chunk's arrival and its use), with its own running maximum and sum, and
// the four warps' results are joined once per item. The products are m16n8k16
// tensor-core products with the rows as M: rows are few, and their S and P stay
// in the registers in which one product leaves them and the next wants them.
//
// FP8 and INT4 codes go to shared memory as they are, so that the ring holds more
// keys, and become operands in registers: e4m3 to bf16 by moving the bits and one
// exact multiplication, the rows' scales applied to the scores and to P. (FP8 keys as
// fp16 by the conversion instruction, with a query scaled to fp16: no faster.) An INT4
// key's codes go into the product as they are (16 + q, exact in bf16, by one shift and
// one logical operation), one product sum a group, and its scale and bias enter in fp32:
//   q . k = sum_groups scale (sum Q (q + 16)) + (bias - 16 scale) sum Q
// An INT4 value becomes q * scale + bias in fp16.
//
// What it measures (GPU times of a call, the join included, replayed back to back in a CUDA
// graph): 32 chains of 8 tokens x 4 heads over up to 6000 bf16 keys of 8 heads,
// 110 us for 0.6 GB, 0.80 of the measured copy rate (some 100 of them this kernel at 75% of
// DRAM's peak, the rest the join); 4 x 16 rows of 256 elements over up to 32768 keys 133 us for
// 0.8 GB. 2 x 12 rows over 131072 keys of 8 heads: INT4 94 us for
// 0.23 GB, bound by its instructions, some 490 for a warp's 16 keys at 61% of the issue
// slots (of them 110 that turn codes into operands, 32 products); FP8 98 us for 0.41 GB,
// likewise (65% of the issue slots). One token of 20 heads over 1000 keys: 10 to 11 us, two
// launches and some six dependent loads.
#include <algorithm>
#include <map>
#include <mutex>
#include <type_traits>
#include <utility>

#include "hc_attn.cuh"

namespace tshc {

namespace {

constexpr int kWarps = kAttnThreads / 32;
constexpr int kChunk = 16;               // keys a warp takes at a time
constexpr int kTile = kChunk * kWarps;   // keys of a tile
constexpr float kRescale = 8.f;          // the reference maximum moves when it is exceeded by this much (log2)

template <int kType, int D>
struct Format {
    static constexpr int kRow = kType == kKvBf16 ? 2 * D : kType == kKvFp8 ? D : D / 2;  // bytes of a row's codes
    static constexpr int kCodes = kChunk * kRow;
    static constexpr int kMaxGroups = D / 32;
    // one scale array's bytes of a chunk (INT4: room for groups of 32)
    static constexpr int kScale = kType == kKvBf16 ? 0 : kType == kKvFp8 ? 16 : kChunk * kMaxGroups * 2;
    static constexpr int kStage = 2 * kCodes + (kType == kKvInt4 ? 4 : 2) * kScale;
    // some 8 to 24 KB a warp in flight
    static constexpr int kStages = kType == kKvBf16 ? (D == 64 ? 6 : D == 128 ? 3 : 2) : kType == kKvFp8 ? (D == 64 ? 6 : 3)
                                                                                     : (D == 64 ? 8 : 4);
    // CTAs an SM: converting codes is a chain of short dependent steps, which more warps hide
    template <int MT>
    static constexpr int blocks() { return kType == kKvBf16 || D * MT > 128 || (D == 64 && MT == 2) ? 2 : 4; }
};

template <int kType, int D, int MT>
struct Smem {
    using F = Format<kType, D>;
    static constexpr int kRing = kWarps * F::kStages * F::kStage;
    static constexpr int kPitch = D + 8;                             // floats: rows 8 banks apart
    static constexpr int kMerge = kWarps * 16 * MT * (kPitch + 2) * 4;  // overlays the ring
    static constexpr int kOver = kRing > kMerge ? kRing : kMerge;
    static constexpr int kSums = kType == kKvInt4 ? 16 * MT * F::kMaxGroups * 4 : 0;
    static constexpr int kTables = kType == kKvInt4 ? F::kMaxGroups * 16 * 12 : 0;  // of a warp
    static constexpr int kTotal = kOver + 16 * MT * D * 2 + kSums + kWarps * kTables + 512;  // and alignment
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid)
{
    const int n = valid ? 16 : 0;  // 0: the 16 bytes are filled with zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

template <bool kHalf>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if (kHalf)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The first product of a sum: d = a b.
__device__ __forceinline__ void mma16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ void mma16816_or_first(bool first, float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if (first)  // known when compiled
        mma16816_first(d, a, b0, b1);
    else
        mma16816<false>(d, a, b0, b1);
}

// e4m3 codes in the high bytes of the two halves of w -> bf16x2. A code's 4
// exponent and 3 mantissa bits, moved under bf16's sign, read as the value times
// 2^-120 (denormals included); the multiplication by 2^120 is exact.
__device__ __forceinline__ uint32_t e4m3_hi_bf16x2(uint32_t w)
{
    const uint32_t r = ((w >> 4) & 0x07F007F0u) | (w & 0x80008000u);
    uint32_t y;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(r), "r"(0x7B807B80u));
    return y;
}

__device__ __forceinline__ uint32_t e4m3_lo_bf16x2(uint32_t w) { return e4m3_hi_bf16x2(w << 8); }

// Two rows' scale bytes -> their scales 2^(byte - 127), bf16x2 (255: NaN).
__device__ __forceinline__ uint32_t fp8_scales_bf16x2(uint32_t bytes)
{
    const uint32_t e = __byte_perm(bytes, 0, 0x4140);
    return e << 7 | ((e + 0x00010001u) >> 2 & 0x00400040u);
}

__device__ __forceinline__ uint32_t mul2_bf16(uint32_t a, uint32_t b)
{
    uint32_t y;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}

__device__ __forceinline__ uint32_t lds32(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

// N consecutive 32-bit words (N = 1, 2 or 4).
template <int N>
__device__ __forceinline__ void lds_words(uint32_t *w, uint32_t a)
{
    if (N == 1)
        w[0] = lds32(a);
    else if (N == 2)
        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a) : "memory");
    else
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a) : "memory");
}

__device__ __forceinline__ uint32_t lds_u8(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t lds_u16(uint32_t a)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
    return v;
}

// 16-byte pieces of a row's codes are permuted so that the reads below meet no
// bank twice (for rows of 128 bytes and more): piece `unit` of row `row` lies at
// unit ^ swizzle(row). The permutation is linear over XOR in the bits that matter, so
// that a lane's address for another row or piece is its first one with constants
// added and XORed.
template <int kType, int D, bool kValue>
__host__ __device__ constexpr int swizzle(int row)
{
    constexpr int kRow = Format<kType, D>::kRow, kUnits = kRow / 16;
    if (kType == kKvBf16)
        return row & 7;  // ldmatrix: 8 rows at one unit
    if (kType == kKvInt4 && !kValue)
        return (row * kRow / 128) & (kUnits - 1) & 7;  // 8 rows at one unit, a word a lane
    if (kUnits >= 8)
        return kValue ? (row & 6) : ((row & 1) << 2);  // keys: rows 2i, 2i+1 at 4 units; values: rows 0, 2, 4, 6 at 2 units
    return kValue ? (row >> 1) & (kUnits - 1) : (row * kRow / 128) & (kUnits - 1);
}

template <int kType, int D, bool kValue>
__device__ __forceinline__ int piece_at(int row, int unit)
{
    return row * Format<kType, D>::kRow + ((unit ^ swizzle<kType, D, kValue>(row)) << 4);
}

// Element d of value column n-tile j for lane group g.
template <int kType, int D>
__device__ __forceinline__ int value_element(int j, int g)
{
    if (kType == kKvBf16)
        return j * 8 + g;
    constexpr int kPiece = kType == kKvFp8 ? (D >= 128 ? 16 : 8) : (D == 256 ? 32 : D / 8);  // elements a lane reads at once
    return (j / kPiece) * (8 * kPiece) + g * kPiece + j % kPiece;
}

// kGroup: an INT4 group's elements. It is known when compiled, so that a group's sum begins
// without zeros and ends without a branch (2 x 12 rows over 131072 keys: 98 us when it was
// taken, with a variable 111).
template <int kType, int D, int MT, int kGroup>
struct Walk {
    using F = Format<kType, D>;
    static constexpr int kGroups = kType == kKvInt4 ? D / kGroup : 1;   // of a row
    static constexpr int kSpans = kType == kKvInt4 ? kGroup / 32 : 1;   // 32-element spans of a group
    static_assert(kType != kKvBf16 || F::kStage % 512 == 0, "constants are XORed into a bf16 stage's addresses");
    static constexpr bool kHalf = kType == kKvInt4;  // P and the values in fp16
    static constexpr float kLift = kHalf ? kFp16Lift : 0.f;
    static constexpr int kSteps = D / 16;
    static constexpr int kCols = D / 8;

    static constexpr int kUnits = F::kRow / 16;

    const AttnParams &p;
    uint32_t ring;            // this warp's ring (shared address)
    uint32_t qs;              // the block's query fragments (shared address)
    uint32_t qsum;            // INT4: the sums of the query's groups [group][row tile][8] of (row g, row g + 8)
    uint32_t tables;          // INT4: this warp's (scale, bias) of a chunk, by group and key
    int lane, g, c, warp;
    int fetch_k, fetch_v;     // where this lane's first piece of a chunk goes
    int read_k, read_v;       // where its first reads of the keys and values lie
    const uint8_t *scales;    // INT4: the array that this lane fetches from
    float sc;                 // |scale| * log2(e), not 0 (its sign went into the query)
    float o[MT][kCols][4];
    float m[MT][2], l[MT][2]; // the reference of each row's weights (times sc), their sum
    float rounded[MT][2];     // bf16 weights: the sum of what the products take of them

    __device__ __forceinline__ Walk(const AttnParams &params) : p(params) {}

    __device__ __forceinline__ void start(int tid)
    {
        lane = tid & 31;
        warp = tid >> 5;
        g = lane >> 2;
        c = lane & 3;
        sc = fmaxf(fabsf(p.scale_log2), 1e-38f);
        fetch_k = piece_at<kType, D, false>(lane / kUnits, lane % kUnits);
        fetch_v = piece_at<kType, D, true>(lane / kUnits, lane % kUnits);
        if (kType == kKvBf16) {
            read_k = piece_at<kType, D, false>((lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1);
            read_v = piece_at<kType, D, true>(lane & 15, lane >> 4);
        } else {
            constexpr int kBytes = kType == kKvFp8 ? (D >= 128 ? 16 : 8) : D / 16;  // of a value's row that a lane reads at once
            read_k = kType == kKvFp8 ? piece_at<kType, D, false>(g, c) : piece_at<kType, D, false>(g, 0) + c * 4;
            read_v = piece_at<kType, D, true>(2 * c, g * kBytes / 16) + g * kBytes % 16;
        }
        if (kType == kKvInt4)
            scales = lane < 8 ? p.c.ks : lane < 16 ? p.c.kb : lane < 24 ? p.c.vs : p.c.vb;
    }

    // Starts the copies of chunk `pos` (its first key) of page `page` into stage s.
    __device__ __forceinline__ void fetch(int s, int page, int head, int pos)
    {
        const bool ok = page >= 0;
        const size_t row = kv_row(p.c, ok ? page : 0, head, pos);
        const uint32_t dst = ring + s * F::kStage;
        const size_t at = row * F::kRow + lane * 16;
        const uint8_t *k = p.c.k + at, *v = p.c.v + at;
        constexpr int kStep = 32 / kUnits;  // rows that the warp's 32 pieces are
        static_assert(kChunk * kUnits >= 32, "a chunk is at least a piece for each lane");
#pragma unroll
        for (int i = 0; i < kChunk * kUnits / 32; ++i) {
            cp_async16(dst + (fetch_k ^ (swizzle<kType, D, false>(kStep * i) << 4)) + i * 512, k + i * 512, ok);
            cp_async16(dst + F::kCodes + (fetch_v ^ (swizzle<kType, D, true>(kStep * i) << 4)) + i * 512, v + i * 512, ok);
        }
        if (kType == kKvFp8 && lane < 2)
            cp_async16(dst + 2 * F::kCodes + lane * F::kScale, (lane ? p.c.vs : p.c.ks) + row, ok);
        if (kType == kKvInt4) {  // 16 * kGroups * 2 bytes of each of the four arrays, eight lanes an array
            const uint8_t *src = scales + row * (2 * kGroups) + (lane & 7) * 16;
            const uint32_t to = dst + 2 * F::kCodes + (lane >> 3) * F::kScale + (lane & 7) * 16;
            constexpr int kParts = 2 * kGroups;  // of 16 bytes
            if ((lane & 7) < kParts)
                cp_async16(to, src, ok);
            if (kParts > 8)
                cp_async16(to + 128, src + 128, ok);
        }
    }

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int j = 0; j < kCols; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[i][j][e] = 0.f;
            m[i][0] = m[i][1] = -INFINITY;
            l[i][0] = l[i][1] = rounded[i][0] = rounded[i][1] = 0.f;
        }
    }

    // Zeros in the place of what must not meet a zero weight: values past the
    // last key (whatever lies there) and infinities and NaNs of the nodes' values.
    // Returns whether a node held any. Warp-wide, only on chunks that reach past the context.
    __device__ __forceinline__ bool tame(int s, int pos, int ctx, int keys)
    {
        const uint32_t v = ring + s * F::kStage + F::kCodes;
        bool wild = false;
        if (kType == kKvBf16) {
            for (int u = lane; u < kChunk * F::kRow / 16; u += 32) {
                const int r = u / (F::kRow / 16);
                if (pos + r < ctx)
                    continue;
                const uint32_t a = v + u * 16;  // the permutation stays inside a row
                uint32_t w[4];
                lds_words<4>(w, a);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool lo = (w[i] & 0x7F80u) == 0x7F80u, hi = (w[i] & 0x7F800000u) == 0x7F800000u;
                    if (pos + r >= keys)
                        w[i] = 0;
                    else if (lo || hi) {
                        wild = true;
                        w[i] &= (lo ? 0xFFFF0000u : 0xFFFFFFFFu) & (hi ? 0x0000FFFFu : 0xFFFFFFFFu);
                    }
                }
                asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
            }
        } else if (kType == kKvFp8) {
            const uint32_t a = ring + s * F::kStage + 2 * F::kCodes + F::kScale + lane;
            if (lane < kChunk && pos + lane >= ctx) {
                const bool past = pos + lane >= keys;
                if (past || lds_u8(a) == kFp8BadRow) {
                    wild = !past;
                    asm volatile("st.shared.u8 [%0], %1;" ::"r"(a), "r"(1) : "memory");
                }
            }
        } else {
            const uint32_t a = ring + s * F::kStage + 2 * F::kCodes + 2 * F::kScale;
            for (int u = lane; u < kChunk * kGroups; u += 32) {
                const int r = u / kGroups;
                if (pos + r < ctx)
                    continue;
                const bool past = pos + r >= keys;
                const uint32_t sc = lds_u16(a + 2 * u), bi = lds_u16(a + F::kScale + 2 * u);
                const bool bad = (sc & 0x7C00u) == 0x7C00u || (bi & 0x7C00u) == 0x7C00u;
                if (past || bad) {
                    wild |= !past;
                    asm volatile("st.shared.u16 [%0], %1;" ::"r"(a + 2 * u), "h"((uint16_t)0) : "memory");
                    asm volatile("st.shared.u16 [%0], %1;" ::"r"(a + F::kScale + 2 * u), "h"((uint16_t)0) : "memory");
                }
            }
        }
        return __any_sync(0xFFFFFFFFu, wild);
    }

    // INT4: a chunk's scales and biases, which lie by key and group, as the products take them:
    // for the keys (scale, bias - 16 scale) in fp32 by group and key, for the values the fp16 scales,
    // then the biases, by group and key. Read with one load each below.
    __device__ __forceinline__ void lay_out_scales(uint32_t stage)
    {
        const int t = lane & 15;
#pragma unroll
        for (int grp = lane >> 4; grp < kGroups; grp += 2) {
            const uint32_t a = stage + 2 * F::kCodes + 2 * (t * kGroups + grp);
            const float s = __half2float(__ushort_as_half((unsigned short)lds_u16(a)));
            const float bias = fmaf(-16.f, s, __half2float(__ushort_as_half((unsigned short)lds_u16(a + F::kScale))));
            asm volatile("st.shared.v2.f32 [%0], {%1,%2};" ::"r"(tables + (grp * 16 + t) * 8), "f"(s), "f"(bias) : "memory");
            const uint32_t vt = tables + F::kMaxGroups * 128 + (grp * 16 + t) * 2;
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(vt), "h"((uint16_t)lds_u16(a + 2 * F::kScale)) : "memory");
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(vt + F::kMaxGroups * 32), "h"((uint16_t)lds_u16(a + 3 * F::kScale)) : "memory");
        }
        __syncwarp();
    }

    // One chunk: scores, softmax update, weighted values. `tail`: it reaches past
    // the context, so the mask is looked at.
    __device__ __forceinline__ void chunk(int s, int pos, bool tail, int b, int row0, const SeqLen &seq)
    {
        const uint32_t stage = ring + s * F::kStage;
        // bf16 stages are multiples of 512 bytes, so that a constant can be XORed into the whole address
        const uint32_t vbase = stage + F::kCodes + read_v;
        const auto key_at = [&](int x) { return kType == kKvBf16 ? (stage + read_k) ^ x : stage + (read_k ^ x); };
        float x[MT][2][4];
        if (kType == kKvInt4)
            lay_out_scales(stage);

        // scores
        if (kType == kKvBf16) {
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                uint32_t kb[4];
                ldmatrix4(kb, key_at(k << 5));
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    uint32_t qa[4];
                    lds_words<4>(qa, qs + ((i * kSteps + k) * 32 + lane) * 16);
                    mma16816_or_first(k == 0, x[i][0], qa, kb[0], kb[1]);
                    mma16816_or_first(k == 0, x[i][1], qa, kb[2], kb[3]);
                }
            }
        } else if (kType == kKvFp8) {
            constexpr int kPieces = F::kRow / 64;  // of 16 bytes, for each lane of a row's four
#pragma unroll
            for (int y = 0; y < kPieces; ++y) {
                uint32_t w[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
                    lds_words<4>(w[n], key_at(y << 6) + n * 8 * F::kRow);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t k00 = e4m3_lo_bf16x2(w[0][k]), k01 = e4m3_hi_bf16x2(w[0][k]);
                    const uint32_t k10 = e4m3_lo_bf16x2(w[1][k]), k11 = e4m3_hi_bf16x2(w[1][k]);
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        uint32_t qa[4];
                        lds_words<4>(qa, qs + ((i * kSteps + y * 4 + k) * 32 + lane) * 16);
                        mma16816_or_first(y + k == 0, x[i][0], qa, k00, k01);
                        mma16816_or_first(y + k == 0, x[i][1], qa, k10, k11);
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float ks = fp8_scale(lds_u8(stage + 2 * F::kCodes + n * 8 + 2 * c + e));
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            x[i][n][2 * h + e] *= ks;
                }
        } else {
            float z[MT][2][4];
#pragma unroll
            for (int y = 0; y < D / 32; ++y) {  // 32 elements of every key, all in one group
                const int grp = y / kSpans;
                const uint32_t w0 = lds32(key_at(y << 4)), w1 = lds32(key_at(y << 4) + 8 * F::kRow);
                const uint32_t k0[4] = {int4_bf16x2<0>(w0), int4_bf16x2<1>(w0), int4_bf16x2<2>(w0), int4_bf16x2<3>(w0)};
                const uint32_t k1[4] = {int4_bf16x2<0>(w1), int4_bf16x2<1>(w1), int4_bf16x2<2>(w1), int4_bf16x2<3>(w1)};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const bool first = y % kSpans + k == 0;
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        uint32_t qa[4];
                        lds_words<4>(qa, qs + ((i * kSteps + 2 * y + k) * 32 + lane) * 16);
                        mma16816_or_first(first, z[i][0], qa, k0[2 * k], k0[2 * k + 1]);
                        mma16816_or_first(first, z[i][1], qa, k1[2 * k], k1[2 * k + 1]);
                    }
                }
                if ((y + 1) % kSpans == 0) {
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        uint32_t q[2];
                        lds_words<2>(q, qsum + (grp * MT + i) * 64 + g * 8);
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            uint32_t t[4];  // (scale, bias) of keys 8n + 2c and 8n + 2c + 1
                            lds_words<4>(t, tables + grp * 128 + c * 16 + n * 64);
#pragma unroll
                            for (int e = 0; e < 2; ++e)
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    float &v = x[i][n][2 * h + e];
                                    const float bias = __uint_as_float(t[2 * e + 1]), sum = __uint_as_float(q[h]);
                                    v = fmaf(__uint_as_float(t[2 * e]), z[i][n][2 * h + e], grp == 0 ? bias * sum : fmaf(bias, sum, v));
                                }
                        }
                    }
                }
            }
        }

        // softmax: this lane has keys 8n + 2c and 8n + 2c + 1 of rows g and g + 8
        if (tail) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int t = (row0 + i * 16 + h * 8 + g) / p.G;
                    const uint32_t see = t < p.T ? attn_sees32(p, attn_mask_row(p, b, t), t, pos - seq.ctx, seq) : 0u;
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (!((see >> (n * 8 + 2 * c + e)) & 1u))
                                x[i][n][2 * h + e] = -INFINITY;
                }
        }
        bool move = false;
        float mx[MT][2];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float top = fmaxf(fmaxf(x[i][0][2 * h], x[i][0][2 * h + 1]), fmaxf(x[i][1][2 * h], x[i][1][2 * h + 1]));
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                mx[i][h] = top * sc;
                move |= mx[i][h] > m[i][h] + (kRescale + kLift);  // also the first that is not -infinity
            }
        if (__any_sync(0xFFFFFFFFu, move)) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float to = fmaxf(m[i][h], mx[i][h] - kLift);
                    const float by = to == -INFINITY ? 1.f : ex2(m[i][h] - to);
                    m[i][h] = to;
                    l[i][h] *= by;
                    rounded[i][h] *= by;
#pragma unroll
                    for (int j = 0; j < kCols; ++j) {
                        o[i][j][2 * h] *= by;
                        o[i][j][2 * h + 1] *= by;
                    }
                }
        }
        uint32_t vs[2];  // the scales of the values of keys 8n + 2c and 8n + 2c + 1, bf16x2
        if (kType == kKvFp8) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
                vs[n] = fp8_scales_bf16x2(lds_u16(stage + 2 * F::kCodes + F::kScale + n * 8 + 2 * c));
        }
        uint32_t pa[MT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float ref = m[i][h] == -INFINITY ? 0.f : m[i][h];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float a = ex2(fmaf(x[i][n][2 * h], sc, -ref)), z = ex2(fmaf(x[i][n][2 * h + 1], sc, -ref));
                    l[i][h] += a + z;
                    // P to 16 bits. In bf16 its rounding is as large as the result's own: dividing by the sum of
                    // the rounded P (the logarithm is of the other) makes the weights sum to one, so that a row that
                    // one key dominates gets that key's value.
                    if (kHalf) {
                        pa[i][2 * n + h] = pack2_f16(a, z);
                    } else {
                        const uint32_t w = pack2_bf16(a, z);
                        rounded[i][h] += bf16_lo(w) + bf16_hi(w);
                        pa[i][2 * n + h] = kType == kKvFp8 ? mul2_bf16(w, vs[n]) : w;
                    }
                }
            }

        // weighted values
        if (kType == kKvBf16) {
#pragma unroll
            for (int j = 0; j < kCols; j += 2) {
                uint32_t vb[4];
                ldmatrix4_trans(vb, vbase ^ (j << 4));
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    mma16816<false>(o[i][j], pa[i], vb[0], vb[1]);
                    mma16816<false>(o[i][j + 1], pa[i], vb[2], vb[3]);
                }
            }
        } else {
            constexpr int kPiece = kType == kKvFp8 ? (D >= 128 ? 16 : 8) : D / 8;  // elements
            constexpr int kBytes = kType == kKvFp8 ? kPiece : kPiece / 2;
            constexpr int kWords = kBytes / 4;
            constexpr int kPer = kType == kKvFp8 ? 4 : 8;                          // elements of a word
            constexpr int kPieces = D / (8 * kPiece);
            uint32_t vsc[2] = {0, 0}, vbi[2] = {0, 0};  // INT4: of keys (2c, 2c + 1) and (2c + 8, 2c + 9)
            if (kType == kKvInt4) {
                const int grp = g * kPiece / kGroup;  // a piece lies in one group
                const uint32_t a = tables + F::kMaxGroups * 128 + grp * 32 + c * 4;
                vsc[0] = lds32(a);
                vsc[1] = lds32(a + 16);
                vbi[0] = lds32(a + F::kMaxGroups * 32);
                vbi[1] = lds32(a + F::kMaxGroups * 32 + 16);
            }
#pragma unroll
            for (int y = 0; y < kPieces; ++y) {
                uint32_t w[4][4];  // keys 2c, 2c+1, 2c+8, 2c+9
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    lds_words<kWords>(w[t], vbase + ((t & 1) + (t >> 1) * 8) * F::kRow + y * 128);
#pragma unroll
                for (int k = 0; k < kWords; ++k) {
                    uint32_t lo[2], hi[2];
#pragma unroll
                    for (int t = 0; t < 2; ++t) {  // the two keys' low and high 16 bits side by side
                        lo[t] = __byte_perm(w[2 * t][k], w[2 * t + 1][k], 0x5410);
                        hi[t] = __byte_perm(w[2 * t][k], w[2 * t + 1][k], 0x7632);
                    }
#pragma unroll
                    for (int e = 0; e < kPer; ++e) {
                        uint32_t vb[2];
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (kType == kKvFp8) {
                                const uint32_t z = e < 2 ? lo[t] : hi[t];
                                vb[t] = (e & 1) ? e4m3_hi_bf16x2(z) : e4m3_lo_bf16x2(z);
                            } else {
                                const uint32_t z = (e < 4 ? lo[t] : hi[t]) >> (8 * ((e >> 1) & 1));
                                const __half2 &sc2 = reinterpret_cast<const __half2 &>(vsc[t]), &bi2 = reinterpret_cast<const __half2 &>(vbi[t]);
                                vb[t] = (e & 1) ? int4_f16x2<true>(z, sc2, bi2) : int4_f16x2<false>(z, sc2, bi2);
                            }
                        }
                        const int j = y * kPiece + k * kPer + e;
#pragma unroll
                        for (int i = 0; i < MT; ++i)
                            mma16816<kHalf>(o[i][j], pa[i], vb[0], vb[1]);
                    }
                }
            }
        }
    }
};

// Element (row, d) of a block's rows, which the query was permuted from.
__device__ __forceinline__ const uint16_t *query_row(const AttnParams &p, int b, int head, int row)
{
    const int t = row / p.G, h = head * p.G + row % p.G;
    return p.q + ((size_t)b * p.T + t) * p.q_stride + (size_t)h * p.c.D;
}

// MT * 16 rows a block; grid: any number of CTAs up to kAttnMaxGrid.
template <int kType, int D, int MT, int kGroup>
__global__ void __launch_bounds__(kAttnThreads, (Format<kType, D>::template blocks<MT>())) hc_attn_few_kernel(const __grid_constant__ AttnParams p, const int least)
{
    using W = Walk<kType, D, MT, kGroup>;
    using F = Format<kType, D>;
    using S = Smem<kType, D, MT>;
    constexpr int kRows = 16 * MT;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ LineScratch scratch;
    __shared__ int wild_any;
    pdl_wait();
    pdl_launch_dependents();  // after the wait: the join reads the lengths before its own
    const int tid = threadIdx.x;
    const Line<> line(p, kTile, scratch);
    const int ctas = attn_ctas(line.total, gridDim.x, least);
    if ((int)blockIdx.x >= ctas || line.total == 0)
        return;
    const Cut cut(line.total, ctas);
    Items it;
    it.at = it.first = cut.first(blockIdx.x);
    it.end = cut.first(blockIdx.x + 1);
    line.find(p, kTile, it.at, scratch);
    it.b = scratch.b;
    it.base = scratch.base;

    uint8_t *ring = smem + ((512u - (smem_addr(smem) & 511u)) & 511u);
    uint8_t *qsm = ring + S::kOver;
    W w(p);
    w.start(tid);
    w.ring = smem_addr(ring) + w.warp * F::kStages * F::kStage;
    w.qs = smem_addr(qsm);
    float *qsum = reinterpret_cast<float *>(qsm + 16 * MT * D * 2);
    w.qsum = smem_addr(qsum);
    w.tables = w.qsum + S::kSums + w.warp * S::kTables;
    float *merge = reinterpret_cast<float *>(ring);  // [warp][row][D], then maxima and sums [warp][row]
    float *merge_m = merge + kWarps * kRows * S::kPitch, *merge_l = merge_m + kWarps * kRows;

    while (it.next(p, kTile)) {
        const SeqLen seq = it.seq;
        const int b = it.b, head = it.head, row0 = it.block * kRows, t0 = it.t0, t1 = it.t1;
        if (seq.bad && tid == 0 && p.status)
            atomicExch(p.status, kStatusBadArg);

        w.clear();
        // pages of the next 32 tiles' chunks, one a lane
        int pages = -1, pages_next = -1;
        const auto page_of = [&](int t) {
            const long pos = (long)t * kTile + w.warp * kChunk;
            return t < t1 && pos < seq.keys ? (int)kv_page(p.c, b, pos) : -1;
        };
        pages = page_of(t0 + w.lane);
        pages_next = page_of(t0 + 32 + w.lane);
        int fetched = t0, into = 0;
        const auto fetch_next = [&]() {
            if (fetched < t1) {
                const int i = (fetched - t0) & 31;
                if (i == 0 && fetched > t0) {
                    pages = pages_next;
                    pages_next = page_of(fetched + 32 + w.lane);
                }
                const int page = __shfl_sync(0xFFFFFFFFu, pages, i);
                const int pos = fetched * kTile + w.warp * kChunk;
                if (pos < seq.keys) {
                    if (page < 0 && w.lane == 0 && p.status)
                        atomicExch(p.status, kStatusBadArg);
                    w.fetch(into, page, head, pos);
                }
            }
            ++fetched;
            into = into + 1 == F::kStages ? 0 : into + 1;
            cp_commit();
        };
#pragma unroll 1
        for (int s = 0; s < F::kStages - 1; ++s)  // on their way while the query is laid out
            fetch_next();

        // The query, as the fragments that the products take. A thread reads 16 bytes of a row, four
        // pairs, each of which is one register of one lane's fragment.
        {
            constexpr int kPieces = D / 8, kStep = kAttnThreads / kPieces, kPasses = kRows / kStep;
            const int x8 = tid % kPieces;
            uint4 v[kPasses];
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int row = row0 + tid / kPieces + i * kStep;
                v[i] = row < p.rows ? *reinterpret_cast<const uint4 *>(query_row(p, b, head, row) + x8 * 8) : make_uint4(0, 0, 0, 0);
            }
            const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int r = tid / kPieces + i * kStep, rr = r & 15;
                const uint4 q = make_uint4(v[i].x ^ flip, v[i].y ^ flip, v[i].z ^ flip, v[i].w ^ flip);
                uint32_t *frag = reinterpret_cast<uint32_t *>(qsm) + (r >> 4) * W::kSteps * 128 + (rr & 7) * 16 + (rr >> 3);
                if (kType == kKvBf16) {  // pair w: lane quarter w, register 0 or 2
                    uint32_t *at = frag + (x8 >> 1) * 128 + (x8 & 1) * 2;
                    at[0] = q.x;
                    at[4] = q.y;
                    at[8] = q.z;
                    at[12] = q.w;
                } else if (kType == kKvFp8) {  // a lane quarter's 16 elements are four steps: pairs (0, 2) and (1, 3) of each four
                    uint32_t *at = frag + ((x8 >> 3) * 4 + (x8 & 1) * 2) * 128 + ((x8 >> 1) & 3) * 4;
                    at[0] = __byte_perm(q.x, q.y, 0x5410);
                    at[2] = __byte_perm(q.x, q.y, 0x7632);
                    at[128] = __byte_perm(q.z, q.w, 0x5410);
                    at[130] = __byte_perm(q.z, q.w, 0x7632);
                } else {  // a lane quarter's 8 elements are two steps: pairs (0, 4), (1, 5) and (2, 6), (3, 7)
                    uint32_t *at = frag + (x8 >> 2) * 256 + (x8 & 3) * 4;
                    at[0] = __byte_perm(q.x, q.z, 0x5410);
                    at[2] = __byte_perm(q.x, q.z, 0x7632);
                    at[128] = __byte_perm(q.y, q.w, 0x5410);
                    at[130] = __byte_perm(q.y, q.w, 0x7632);
                    float sum = ((bf16_lo(q.x) + bf16_hi(q.x)) + (bf16_lo(q.y) + bf16_hi(q.y))) +
                                ((bf16_lo(q.z) + bf16_hi(q.z)) + (bf16_lo(q.w) + bf16_hi(q.w)));
                    constexpr int lanes = kGroup / 8;  // 4, 8 or 16 lanes hold a group
                    for (int o = lanes / 2; o > 0; o >>= 1)
                        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                    if (x8 % lanes == 0)
                        qsum[((x8 / lanes * MT + (r >> 4)) * 8 + (rr & 7)) * 2 + (rr >> 3)] = sum;
                }
            }
        }
        if (tid == 0)
            wild_any = 0;
        __syncthreads();

        bool wild = false;
        int stage = 0;
        for (int t = t0; t < t1; ++t) {
            cp_wait<F::kStages - 2>();
            __syncwarp();
            fetch_next();
            const int pos = t * kTile + w.warp * kChunk;
            if (pos < seq.keys) {
                const bool tail = pos + kChunk > seq.ctx;
                if (tail) {
                    wild |= w.tame(stage, pos, seq.ctx, seq.keys);
                    __syncwarp();
                }
                w.chunk(stage, pos, tail, b, row0, seq);
            }
            stage = stage + 1 == F::kStages ? 0 : stage + 1;
        }
        cp_wait<0>();
        if (wild && w.lane == 0)
            wild_any = 1;
        __syncthreads();

        // join the warps
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float sum = w.l[i][h];
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
                if (!W::kHalf) {
                    float rounded = w.rounded[i][h];
                    rounded += __shfl_xor_sync(0xFFFFFFFFu, rounded, 1);
                    rounded += __shfl_xor_sync(0xFFFFFFFFu, rounded, 2);
                    const float by = rounded == 0.f ? 1.f : sum / rounded;
#pragma unroll
                    for (int j = 0; j < W::kCols; ++j) {
                        w.o[i][j][2 * h] *= by;
                        w.o[i][j][2 * h + 1] *= by;
                    }
                }
                const int r = i * 16 + h * 8 + w.g;
                if (w.c == 0) {
                    merge_m[w.warp * kRows + r] = w.m[i][h];
                    merge_l[w.warp * kRows + r] = sum;
                }
                float *row = merge + (w.warp * kRows + r) * S::kPitch;
                if (kType == kKvBf16) {  // lane quarter c holds columns 2c, 2c + 1 of n-tile j
#pragma unroll
                    for (int j = 0; j < W::kCols; ++j)
                        *reinterpret_cast<float2 *>(row + j * 8 + 2 * w.c) = make_float2(w.o[i][j][2 * h], w.o[i][j][2 * h + 1]);
                } else {  // n-tiles j .. j + 3 are four elements side by side, of the pieces 2c and 2c + 1
#pragma unroll
                    for (int j = 0; j < W::kCols; j += 4)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            *reinterpret_cast<float4 *>(row + value_element<kType, D>(j, 2 * w.c + e)) =
                                make_float4(w.o[i][j][2 * h + e], w.o[i][j + 1][2 * h + e], w.o[i][j + 2][2 * h + e], w.o[i][j + 3][2 * h + e]);
                }
            }
        __syncthreads();
        const bool whole = it.whole();
        float *slot = p.part + (size_t)(2 * blockIdx.x + it.slot()) * attn_slot_floats(kRows, D);
        for (int i = tid; i < kRows * (D / 4); i += kAttnThreads) {
            const int r = i / (D / 4), d = (i % (D / 4)) * 4, row = row0 + r;
            if (row >= p.rows)
                continue;
            float top = merge_m[r];
#pragma unroll
            for (int v = 1; v < kWarps; ++v)
                top = fmaxf(top, merge_m[v * kRows + r]);
            const float ref = top == -INFINITY ? 0.f : top;
            float sum = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int v = 0; v < kWarps; ++v) {
                const float f = ex2(merge_m[v * kRows + r] - ref);
                sum += f * merge_l[v * kRows + r];
                const float4 x = *reinterpret_cast<const float4 *>(merge + (v * kRows + r) * S::kPitch + d);
                acc.x += f * x.x;
                acc.y += f * x.y;
                acc.z += f * x.z;
                acc.w += f * x.w;
            }
            const int t = row / p.G, h = head * p.G + row % p.G;
            if (wild_any) {
                const int from = t0 * kTile, to = min(seq.keys, t1 * kTile);
                acc.x += attn_wild_values(p, b, head, t, d, seq.ctx, from, to);
                acc.y += attn_wild_values(p, b, head, t, d + 1, seq.ctx, from, to);
                acc.z += attn_wild_values(p, b, head, t, d + 2, seq.ctx, from, to);
                acc.w += attn_wild_values(p, b, head, t, d + 3, seq.ctx, from, to);
            }
            if (whole) {
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                const size_t n = ((size_t)b * p.T + t) * p.q_heads + h;
                *reinterpret_cast<uint2 *>(p.out + n * D + d) =
                    make_uint2(pack2_bf16(acc.x * inv, acc.y * inv), pack2_bf16(acc.z * inv, acc.w * inv));
                if (d == 0 && p.lse)
                    p.lse[n] = top == -INFINITY ? (sum == 0.f ? -INFINITY : sum) : (top + log2f(sum)) * 0.6931471805599453f;
            } else {
                *reinterpret_cast<float4 *>(slot + (size_t)r * D + d) = acc;
                if (d == 0) {
                    slot[(size_t)kRows * D + r] = top;
                    slot[(size_t)kRows * (D + 1) + r] = sum;
                }
            }
        }
        __syncthreads();
    }
}

constexpr int kJoinLoads = 4;  // segments whose rows a lane has in flight

// The CTAs c0 .. c1 whose segments make up blockIdx.x's item (sequence, head, row block);
// c0 = c1 where there is nothing to join.
struct Segments {
    int b, item, c0 = 0, c1 = 0, skew = 0;

    __device__ __forceinline__ Segments(const AttnParams &p, int rows, int tile, int grid, int least, LineScratch &scratch)
    {
        const Line<true> line(p, tile, scratch);
        const int ctas = attn_ctas(line.total, grid, least);
        const int blocks = p.c.heads * p.row_blocks;
        b = blockIdx.x / blocks;
        item = blockIdx.x % blocks;
        if (line.total == 0)
            return;
        const SeqLen seq = attn_seq<true>(p, b, tile);
        // the line's index of sequence b: the thread that has it in its run
        if (b >= line.b0 && b < line.b1) {
            long at = line.base;
            for (int i = line.b0; i < b; ++i)
                at += attn_seq<true>(p, i, tile).tiles * line.per;
            scratch.base = at;
        }
        __syncthreads();
        const long from = scratch.base + (long)item * seq.tiles;
        const Cut cut(line.total, ctas);
        c0 = cut.cta_of(from);
        c1 = cut.cta_of(from + seq.tiles - 1);
        skew = cut.first(c0) < from ? 1 : 0;
    }

    // A CTA's segment of this item is its first, unless it is CTA c0 and began before the item.
    __device__ __forceinline__ float *slot(const AttnParams &p, int c, int rows, int D) const
    {
        return p.part + (size_t)(2 * c + (c == c0 ? skew : 0)) * attn_slot_floats(rows, D);
    }
};

// Joins the segments of the items that more than one CTA worked on: a warp a row (or,
// kWarpsARow = 4, a block a row, its warps with every fourth segment, for few rows in
// many segments), lane i with the maximum and the sum of segment i (of up to 32 at a
// time), and the segments' rows added in their order. What the kernel costs is its chain
// of dependent loads -- lengths, then maxima and the first rows together, then further
// rows, some 0.7 us each -- and how many warps wait at a time. 12 rows in 76 segments:
// 9 us a warp a row with eight loads in flight, 16 with four, 8 with a block a row. The
// lengths are read while the attention kernel ends, which is 1 to 2 us of it.
template <int D, int kWarpsARow>
__global__ void __launch_bounds__(kAttnThreads, D == 256 ? 8 : 10) hc_attn_join_kernel(const __grid_constant__ AttnParams p, const int rows, const int tile,
                                                                                       const int grid, const int least)
{
    __shared__ float across[kWarpsARow > 1 ? kWarps : 1][D + 2];
    __shared__ LineScratch scratch;
    pdl_launch_dependents();
    // the lengths only, which nothing changes from the attention kernel's start on
    const Segments of(p, rows, tile, grid, least, scratch);
    pdl_wait();
    const int b = of.b, item = of.item, c0 = of.c0, c1 = of.c1;
    if (c0 == c1)
        return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = kWarpsARow > 1 ? blockIdx.y : blockIdx.y * kWarps + warp, row = (item % p.row_blocks) * rows + r;
    if (r >= rows || row >= p.rows)
        return;
    const auto slot = [&](int c) { return of.slot(p, c, rows, D); };
    constexpr int kVec = D / 32 >= 4 ? 4 : 2;  // floats of a load
    constexpr int kLoads = D / (32 * kVec);    // loads of a lane: 1, or 2 for D = 256
    using Vec = typename std::conditional<kVec == 4, float4, float2>::type;
    float acc[kLoads * kVec];
#pragma unroll
    for (int i = 0; i < kLoads * kVec; ++i)
        acc[i] = 0.f;
    float sum = 0.f, top = -INFINITY;
    const int first = kWarpsARow > 1 ? warp : 0;  // this warp's segments: first, first + kWarpsARow, ...
    const int segs = (c1 - c0 - first) / kWarpsARow + (c1 - c0 >= first ? 1 : 0);
#pragma unroll 1
    for (int base = 0; base < segs; base += 32) {
        const int n = min(32, segs - base);
        const auto seg = [&](int i) { return slot(c0 + first + (base + i) * kWarpsARow); };
        Vec v[kJoinLoads][kLoads];
        const auto load = [&](int i0) {
#pragma unroll
            for (int i = 0; i < kJoinLoads; ++i)
                if (i0 + i < n) {
                    const Vec *x = reinterpret_cast<const Vec *>(seg(i0 + i) + (size_t)r * D);
#pragma unroll
                    for (int k = 0; k < kLoads; ++k)
                        v[i][k] = __ldcg(x + lane + 32 * k);
                }
        };
        float m = -INFINITY, l = 0.f;
        if (lane < n) {
            const float *s = seg(lane) + (size_t)rows * D + r;
            m = __ldcg(s);
            l = __ldcg(s + rows);
        }
        load(0);
        float now = m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            now = fmaxf(now, __shfl_xor_sync(0xFFFFFFFFu, now, o));
        const float to = fmaxf(top, now), ref = to == -INFINITY ? 0.f : to;
        const float by = ex2(top - ref);  // 0 at the first
        const float f = ex2(m - ref);
        top = to;
        float part = f * l;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            part += __shfl_xor_sync(0xFFFFFFFFu, part, o);
        sum = sum * by + part;
#pragma unroll
        for (int i = 0; i < kLoads * kVec; ++i)
            acc[i] *= by;
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += kJoinLoads) {
            if (i0 > 0)
                load(i0);
#pragma unroll
            for (int i = 0; i < kJoinLoads; ++i)
                if (i0 + i < n) {
                    const float g = __shfl_sync(0xFFFFFFFFu, f, i0 + i);
#pragma unroll
                    for (int k = 0; k < kLoads; ++k)
#pragma unroll
                        for (int e = 0; e < kVec; ++e)
                            acc[k * kVec + e] += g * reinterpret_cast<const float *>(&v[i][k])[e];
                }
        }
    }
    if (kWarpsARow > 1) {  // the warps' sums, in their order
        float *mine = across[warp];
#pragma unroll
        for (int k = 0; k < kLoads; ++k)
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                mine[(lane + 32 * k) * kVec + e] = acc[k * kVec + e];
        if (lane == 0) {
            mine[D] = top;
            mine[D + 1] = sum;
        }
        __syncthreads();
        if (warp > 0)
            return;
        top = fmaxf(fmaxf(across[0][D], across[kWarpsARow > 1 ? 1 : 0][D]), fmaxf(across[kWarpsARow > 1 ? 2 : 0][D], across[kWarpsARow > 1 ? 3 : 0][D]));
        const float ref = top == -INFINITY ? 0.f : top;
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < kLoads * kVec; ++i)
            acc[i] = 0.f;
#pragma unroll
        for (int w = 0; w < (kWarpsARow > 1 ? kWarps : 1); ++w) {
            const float f = ex2(across[w][D] - ref);
            sum += f * across[w][D + 1];
#pragma unroll
            for (int k = 0; k < kLoads; ++k)
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    acc[k * kVec + e] += f * across[w][(lane + 32 * k) * kVec + e];
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int t = row / p.G, h = (item / p.row_blocks) * p.G + row % p.G;
    const size_t n = ((size_t)b * p.T + t) * p.q_heads + h;
    uint32_t *out = reinterpret_cast<uint32_t *>(p.out + n * D);
#pragma unroll
    for (int k = 0; k < kLoads; ++k)
#pragma unroll
        for (int e = 0; e < kVec / 2; ++e)
            out[(lane + 32 * k) * (kVec / 2) + e] = pack2_bf16(acc[k * kVec + 2 * e] * inv, acc[k * kVec + 2 * e + 1] * inv);
    if (lane == 0 && p.lse)
        p.lse[n] = top == -INFINITY ? (sum == 0.f ? -INFINITY : sum) : (top + log2f(sum)) * 0.6931471805599453f;
}

// The same for the wide kernel's slots, whose sums lie by four columns: a block has eight
// rows, whose pieces fill a line, and a thread adds up its row's pieces, of up to four
// segments at a time, with its own factors. 64 items of 256 rows in 3 to 4 segments,
// 28 MB: 12 us (17 a warp a row from sums that lay by rows, whose stores took the
// attention kernel 10 us more).
template <int D>
__global__ void __launch_bounds__(kAttnThreads, 8) hc_attn_join_wide_kernel(const __grid_constant__ AttnParams p, const int rows, const int tile,
                                                                            const int grid, const int least)
{
    constexpr int kLoads = D / 64;  // pieces of a thread: a row has D / 4, 16 threads a row
    __shared__ LineScratch scratch;
    pdl_launch_dependents();
    // the lengths only, which nothing changes from the attention kernel's start on
    const Segments of(p, rows, tile, grid, least, scratch);
    pdl_wait();
    if (of.c0 == of.c1)
        return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = blockIdx.y * 8 + (lane & 7), row = (of.item % p.row_blocks) * rows + r;
    const int piece = warp * (D / 16) + (lane >> 3);  // and every fourth from there
    float acc[kLoads][4] = {}, sum = 0.f, top = -INFINITY;
#pragma unroll 1
    for (int c = of.c0; c <= of.c1; c += kJoinLoads) {
        float m[kJoinLoads], l[kJoinLoads];
        float4 v[kJoinLoads][kLoads];
#pragma unroll
        for (int i = 0; i < kJoinLoads; ++i) {
            m[i] = -INFINITY;
            if (c + i <= of.c1) {
                const float *s = of.slot(p, c + i, rows, D);
                m[i] = __ldcg(s + (size_t)rows * D + r);
                l[i] = __ldcg(s + (size_t)rows * (D + 1) + r);
#pragma unroll
                for (int k = 0; k < kLoads; ++k)
                    v[i][k] = __ldcg(reinterpret_cast<const float4 *>(s) + (size_t)(piece + 4 * k) * rows + r);
            }
        }
        const float to = fmaxf(fmaxf(fmaxf(top, m[0]), m[1]), fmaxf(m[2], m[3])), ref = to == -INFINITY ? 0.f : to;
        const float by = ex2(top - ref);  // 0 at the first
        top = to;
        sum *= by;
#pragma unroll
        for (int k = 0; k < kLoads; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[k][e] *= by;
#pragma unroll
        for (int i = 0; i < kJoinLoads; ++i)
            if (c + i <= of.c1) {
                const float f = ex2(m[i] - ref);
                sum += f * l[i];
#pragma unroll
                for (int k = 0; k < kLoads; ++k) {
                    acc[k][0] += f * v[i][k].x;
                    acc[k][1] += f * v[i][k].y;
                    acc[k][2] += f * v[i][k].z;
                    acc[k][3] += f * v[i][k].w;
                }
            }
    }
    if (row >= p.rows)
        return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int t = row / p.G, h = (of.item / p.row_blocks) * p.G + row % p.G;
    const size_t n = ((size_t)of.b * p.T + t) * p.q_heads + h;
    uint2 *out = reinterpret_cast<uint2 *>(p.out + n * D);
#pragma unroll
    for (int k = 0; k < kLoads; ++k)
        out[piece + 4 * k] = make_uint2(pack2_bf16(acc[k][0] * inv, acc[k][1] * inv), pack2_bf16(acc[k][2] * inv, acc[k][3] * inv));
    if (piece == 0 && p.lse)
        p.lse[n] = top == -INFINITY ? (sum == 0.f ? -INFINITY : sum) : (top + log2f(sum)) * 0.6931471805599453f;
}

constexpr int kLeastTiles = 2;  // tiles a CTA has at least, where there is a choice

template <int kType, int D, int MT, int kGroup>
cudaError_t launch_few(AttnParams p, const LaunchCfg &cfg, cudaStream_t stream)
{
    constexpr int kRows = 16 * MT;
    constexpr int kSmem = Smem<kType, D, MT>::kTotal;
    p.row_blocks = (p.rows + kRows - 1) / kRows;
    auto *kernel = hc_attn_few_kernel<kType, D, MT, kGroup>;
    int per_sm = 1;
    cudaError_t e = attn_ready(reinterpret_cast<const void *>(kernel), kAttnThreads, kSmem, &per_sm);
    if (e != cudaSuccess)
        return e;
    const int grid = std::min(per_sm * cfg.sm_count, kAttnMaxGrid);
    cudaLaunchConfig_t lc{};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = at;
    lc.numAttrs = 1;
    lc.stream = stream;
    lc.blockDim = dim3(kAttnThreads);
    lc.gridDim = dim3(grid);
    lc.dynamicSmemBytes = kSmem;
    e = cudaLaunchKernelEx(&lc, kernel, p, kLeastTiles);
    if (e != cudaSuccess)
        return e;
    return launch_attn_join(p, kRows, kTile, grid, kLeastTiles, false, stream);
}

// kGroup: of INT4; the others have none (32 stands for it).
template <int kType, int kGroup = 32>
cudaError_t launch_type(const AttnParams &p, const LaunchCfg &cfg, cudaStream_t stream)
{
    if (p.c.D == 64) {
        if constexpr (kGroup <= 64)
            return p.rows <= 16 ? launch_few<kType, 64, 1, kGroup>(p, cfg, stream) : launch_few<kType, 64, 2, kGroup>(p, cfg, stream);
        else
            return cudaErrorInvalidValue;
    }
    if (p.c.D == 128)
        return p.rows <= 16 ? launch_few<kType, 128, 1, kGroup>(p, cfg, stream) : launch_few<kType, 128, 2, kGroup>(p, cfg, stream);
    return launch_few<kType, 256, 1, kGroup>(p, cfg, stream);
}

}  // namespace

cudaError_t attn_ready(const void *kernel, int threads, int smem, int *per_sm)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    static std::mutex mu;
    static std::map<std::pair<const void *, int>, int> done;
    std::lock_guard<std::mutex> lock(mu);
    const auto key = std::make_pair(kernel, dev);
    const auto at = done.find(key);
    if (at != done.end()) {
        *per_sm = at->second;
        return cudaSuccess;
    }
    int n = 0;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem);
    if (e == cudaSuccess)
        done[key] = *per_sm = std::max(n, 1);
    return e;
}

cudaError_t launch_attn_join(const AttnParams &p, int rows, int tile, int grid, int least, bool by_columns, cudaStream_t stream)
{
    cudaLaunchConfig_t lc{};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = at;
    lc.numAttrs = 1;
    lc.stream = stream;
    lc.blockDim = dim3(kAttnThreads);
    const int used = std::min(rows, p.rows);
    const long items = (long)p.B * p.c.heads * p.row_blocks;
    // few rows: each has many segments, or there is little to do either way
    const bool few = items * used <= 2 * grid;
    const int a_block = by_columns ? 8 : few ? 1 : kWarps;  // rows
    lc.gridDim = dim3((unsigned)items, (unsigned)((used + a_block - 1) / a_block));
    void (*kernel)(AttnParams, int, int, int, int) = nullptr;
    if (by_columns)
        kernel = p.c.D == 64 ? hc_attn_join_wide_kernel<64> : hc_attn_join_wide_kernel<128>;
    else switch (p.c.D) {
    case 64: kernel = few ? hc_attn_join_kernel<64, kWarps> : hc_attn_join_kernel<64, 1>; break;
    case 128: kernel = few ? hc_attn_join_kernel<128, kWarps> : hc_attn_join_kernel<128, 1>; break;
    default: kernel = few ? hc_attn_join_kernel<256, kWarps> : hc_attn_join_kernel<256, 1>; break;
    }
    return cudaLaunchKernelEx(&lc, kernel, p, rows, tile, grid, least);
}

size_t attn_part_bytes(int, int T, int q_heads, const KvView &c)
{
    const long rows = (long)T * (q_heads / c.heads);
    const int wide = attn_wide_rows(c, rows);
    if (wide)
        return sizeof(float) * 2 * kAttnWideGrid * attn_slot_floats(wide, c.D);
    return sizeof(float) * 2 * kAttnMaxGrid * attn_slot_floats(rows <= 16 || c.D == 256 ? 16 : 32, c.D);
}

cudaError_t launch_tree_attention(AttnParams p, const LaunchCfg &cfg, cudaStream_t stream)
{
    if (attn_wide_rows(p.c, p.rows))
        return launch_attn_wide(p, cfg, stream);
    switch (p.c.type) {
    case kKvBf16: return launch_type<kKvBf16>(p, cfg, stream);
    case kKvFp8: return launch_type<kKvFp8>(p, cfg, stream);
    default:
        return p.c.group == 32 ? launch_type<kKvInt4, 32>(p, cfg, stream)
               : p.c.group == 64 ? launch_type<kKvInt4, 64>(p, cfg, stream) : launch_type<kKvInt4, 128>(p, cfg, stream);
    }
}

}  // namespace tshc
