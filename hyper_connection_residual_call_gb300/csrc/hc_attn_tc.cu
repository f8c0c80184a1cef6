// hc_attn_tc.cu -- attention of many rows (a wide tree of drafted tokens, many
// query heads a key head) over the paged cache, on the tensor cores with TMEM
// accumulators: blocks of 128 or 256 rows (ts_hc_tree_attention in include/ts_hc.h).
//
// From some 40 rows on, the products S = Q K^T and O += P V (4 D flops a row and
// key) are more than register-operand products can do in the time that the
// cache's bytes take. Here a tile of 128 keys meets 128 rows in one 128 x 128 x D
// product each way:
//   - Q lies in shared memory (K-major), a tile's keys and values too, as they
//     come from the cache: a value tile [key][d] is a B operand in MN-major order,
//     so nothing is transposed.
//   - S and O are in TMEM, 128 lanes = 128 rows. A softmax thread owns one row: it
//     needs no shuffles, and writes P (bf16) over its S, from where the second
//     product takes it as its A operand.
//   - Two streams keep the tensor cores busy while the other's softmax runs: with
//     256 rows the two halves of the rows, with 128 the even and the odd tiles,
//     which have maxima, sums and accumulators of their own and meet at the end.
//   - O is rescaled only when a row's maximum grows by more than 2^8 over the one
//     it is kept relative to.
// Roles: warps 0-3 and 4-7 softmax of the two streams; warps 8-11, 14 and 15 put
// what has to be converted into shared memory (the query; FP8 tiles; the values of
// a tile that reaches past the context, where what lies behind the last key, and
// infinities and NaNs of nodes, are taken out); warp 12 issues the products, warp 13
// the copies: TMA boxes for bf16 tiles, bulk copies of FP8 codes to a ring of their
// own. FP8 tiles of 64 rows or fewer (kNarrow) are bound by their conversion, so that
// warps 2, 3, 6 and 7, which own no row there, take part in it. A warp runs on scheduler
// (its number mod 4): the softmax is then on schedulers 0 and 1 and most of the conversion
// on 2 and 3.
// Every wait is bounded; the first that runs out records TS_ERR_TIMEOUT and ends
// the others.
#include <algorithm>

#include "hc_attn.cuh"
#include "hc_tc.h"
#include "umma.cuh"

namespace tshc {

namespace {

constexpr int kKeys = 128;               // keys of a tile
constexpr int kThreads = 512;            // 16 warps: the most that leaves 128 registers a thread
constexpr int kMmaWarp = 12, kLoadWarp = 13;
constexpr float kGrow = 8.f;             // log2: how far a row's maximum may grow over its reference
constexpr uint32_t kTmemCols = 512;      // S of two streams, O of two streams

// kNarrow: 64 rows or fewer, so that half of the softmax warps have none and convert too.
template <int kType, int D, int NT, bool kNarrow>
struct Plan {
    static constexpr int kSoftThreads = kNarrow ? 128 : 256, kConvThreads = kThreads - 64 - kSoftThreads;
    static constexpr int kTileBytes = kKeys * D * 2;              // a tile's keys or values as bf16
    static constexpr int kHalf = kKeys * 128;                     // 64 columns of it
    static constexpr int kQBytes = NT * kTileBytes;
    static constexpr int kRawCodes = kKeys * D;                   // FP8
    static constexpr int kRawBytes = kType == kKvFp8 ? kRawCodes + 256 : 0;  // and its rows' scales
    static constexpr int kBudget = (NT == 1 ? 223 : 225) * 1024 - kQBytes;  // beside the barriers (and NT = 1's maxima and sums)
    static constexpr int kSlots = kType == kKvFp8 ? 3 : std::min(8, kBudget / kTileBytes);
    static constexpr int kRaw = kType == kKvFp8 ? std::min(8, (kBudget - kSlots * kTileBytes) / kRawBytes) : 1;
    static constexpr int kQ = kSlots * kTileBytes, kRing = kQ + kQBytes;
    static constexpr int kTotal = kRing + kRaw * kRawBytes + 1024;  // and alignment
};

template <int NT>
struct Shared {
    // Each barrier has one role that waits on it, or waiters whose own arrivals its next phase needs: a
    // parity tells a phase from the next only, so that nobody may fall a phase behind.
    uint64_t full[8], empty[8];          // a tile slot
    uint64_t go[8];                      // bf16: an empty slot is the conversion warps' to fill
    uint64_t raw_full[8], raw_empty[8];  // an FP8 code slot
    uint64_t q_full, q_empty;
    uint64_t s_ready[2], p_ready[2], o_done[2];
    uint32_t tmem;
    int dead;                            // a wait ran out
    int wild[4];                         // by item: a node's value held an infinity or a NaN
    uint32_t raw_valid[8];               // which 16-key chunks of a code slot lie in a page
    float m[2][NT == 1 ? 128 : 1], l[2][NT == 1 ? 128 : 1];  // of the two streams
    LineScratch line;
};

// Waits for the phase; false when it (or another wait of the block) ran out. The
// warp's lanes leave together with one answer. (One lane looking for all of them
// was slower: 165 us against 132 for 4 x 64 nodes over 16384 bf16 keys.)
template <int NT>
__device__ __forceinline__ bool wait_or_dead(uint64_t *bar, uint32_t parity, Shared<NT> &sh, unsigned *status)
{
    bool there = mbar_try_wait(bar, parity);
    if (!there) {
        const uint64_t t0 = global_timer_ns();
        for (;;) {
#pragma unroll 1
            for (int i = 0; i < 16 && !there; ++i)
                there = mbar_try_wait(bar, parity);
            if (there || *reinterpret_cast<volatile int *>(&sh.dead))
                break;
            if (global_timer_ns() - t0 > kWaitLimitNs) {
                *reinterpret_cast<volatile int *>(&sh.dead) = 1;
                if (status)
                    atomicExch(status, kStatusTimeout);
                break;
            }
        }
    }
    return __all_sync(0xFFFFFFFFu, there);
}

__device__ __forceinline__ void named_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

// The order in which a segment of n tiles' keys and values are first used, and so
// loaded: two products ahead of the values. NT = 2 (each tile serves both
// streams): K0 V0 K1 V1 ...; NT = 1 (tiles alternate): K0 K1 V0 K2 V1 ...
template <int NT>
__device__ __forceinline__ int key_index(int j)
{
    return NT == 2 ? 2 * j : j == 0 ? 0 : 2 * j - 1;
}

template <int NT>
__device__ __forceinline__ int value_index(int j, int n)
{
    return NT == 2 ? 2 * j + 1 : j + 1 < n ? 2 * j + 2 : 2 * j + 1;
}

// The e-th of them.
template <int NT>
__device__ __forceinline__ void load_at(int e, int n, int &tile, bool &value)
{
    if (NT == 2) {
        tile = e >> 1;
        value = e & 1;
    } else {
        value = e == 2 * n - 1 || (e > 0 && !(e & 1));
        tile = e == 2 * n - 1 ? n - 1 : e == 0 ? 0 : (e & 1) ? (e + 1) >> 1 : (e >> 1) - 1;
    }
}

// FP8 columns: the conversion leaves elements (0, 2, 1, 3) of each four, in keys,
// values and query alike; the results are put back when they are written.
template <int kType>
__device__ __forceinline__ constexpr int column_of(int d)
{
    return kType == kKvFp8 ? (d & ~3) | ((d & 1) << 1) | ((d >> 1) & 1) : d;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t y;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}

// 8 e4m3 codes -> 8 bf16 (columns permuted as above), times 2^-120 of the bf16 with
// the bits `factor`: a code's bits moved under bf16's sign read as its value times
// 2^-120. For a row's scale 2^e the factor is 2^(120 + e). (The conversion instruction to
// fp16, two to fp32 and one to bf16, and the scale: the same time, 160 us for 159.)
__device__ __forceinline__ uint4 fp8_to_bf16(uint32_t w0, uint32_t w1, uint32_t factor)
{
    const uint32_t f = factor * 0x10001u;
    const uint32_t a = w0 << 8, b = w0, c = w1 << 8, d = w1;
    return make_uint4(mul_bf16x2(((a >> 4) & 0x07F007F0u) | (a & 0x80008000u), f), mul_bf16x2(((b >> 4) & 0x07F007F0u) | (b & 0x80008000u), f),
                      mul_bf16x2(((c >> 4) & 0x07F007F0u) | (c & 0x80008000u), f), mul_bf16x2(((d >> 4) & 0x07F007F0u) | (d & 0x80008000u), f));
}

__device__ __forceinline__ void sts128(uint32_t a, uint4 v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}


// Address of 16-byte piece x (8 columns) of row r in a 128-row tile of D columns.
__device__ __forceinline__ uint32_t tile_piece(uint32_t tile, int r, int x)
{
    return tile + (uint32_t)(x >> 3) * (kKeys * 128) + (uint32_t)r * 128 + (uint32_t)(((x & 7) ^ (r & 7)) << 4);
}

// Scores that a row does not see become -infinity.
__device__ __forceinline__ void hide(uint32_t (&x)[32], uint32_t see)
{
#pragma unroll
    for (int c = 0; c < 32; ++c)
        if (!((see >> c) & 1u))
            x[c] = 0xFF800000u;
}

template <int kType, int D, int NT, bool kNarrow>
__global__ void __launch_bounds__(kThreads, 1)
hc_attn_wide_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const int least)
{
    using P = Plan<kType, D, NT, kNarrow>;
    constexpr int kSoftThreads = P::kSoftThreads, kConvThreads = P::kConvThreads;
    constexpr int kRows = 128 * NT;
    constexpr int kPieces = D / 8;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Shared<NT> sh;
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;

    const Line line(p, kKeys, sh.line);
    const int ctas = attn_ctas(line.total, gridDim.x, least);
    if ((int)blockIdx.x >= ctas || line.total == 0)
        return;
    const Cut cut(line.total, ctas);
    Items it;
    it.at = it.first = cut.first(blockIdx.x);
    it.end = cut.first(blockIdx.x + 1);
    line.find(p, kKeys, it.at, sh.line);
    it.b = sh.line.b;
    it.base = sh.line.base;

    if (tid == 0) {
        for (int i = 0; i < 8; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1);
            mbar_init(&sh.go[i], 1);
            mbar_init(&sh.raw_full[i], 1);
            mbar_init(&sh.raw_empty[i], 1);
        }
        mbar_init(&sh.q_full, 1);
        mbar_init(&sh.q_empty, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh.s_ready[s], 1);
            mbar_init(&sh.p_ready[s], kSoftThreads / 2);
            mbar_init(&sh.o_done[s], 1);
        }
        sh.dead = 0;
        mbar_fence_init();
        fence_async_shared();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&sh.tmem, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    unsigned *status = p.status;

    if (warp < 8 && !(kNarrow && (warp & 2))) {
        // ---------------------------------------------------------- softmax
        const int s = warp >> 2, row_in = tid & 127;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lane_base + s * kKeys, to = tmem + lane_base + 256 + s * 128;
        const float sc = fmaxf(fabsf(p.scale_log2), 1e-38f);  // its sign went into the query; not 0, for masked scores' sake
        uint32_t s_phase = 0, o_phase = 0;
        bool ok = true;
        for (int item = 0; ok && it.next(p, kKeys); ++item) {
            const SeqLen seq = it.seq;
            const int it_b = it.b, it_head = it.head, it_t0 = it.t0, it_t1 = it.t1, it_block = it.block;  // (the walk itself lives in memory)
            if (seq.bad && tid == 0 && status)
                atomicExch(status, kStatusBadArg);
            const int n = it_t1 - it_t0, row0 = it_block * kRows;
            const int row = row0 + (NT == 2 ? s * 128 : 0) + row_in;
            const bool valid = row < p.rows;
            const int t = valid ? row / p.G : 0;
            const uint32_t *mask = attn_mask_row(p, it_b, t);
            // a warp of rows past the last has nothing to do (rows do not meet)
            const bool idle = row0 + (NT == 2 ? s * 128 : 0) + (warp & 3) * 32 >= p.rows;
            float m = -INFINITY, mc = 0.f, l = 0.f;  // the reference (raw units), the same times sc (0 for none), the sum
            int units = 0;
            for (int j = NT == 2 ? 0 : s; j < n; j += 3 - NT, ++units) {
                ok = wait_or_dead(&sh.s_ready[s], s_phase, sh, status);
                if (!ok)
                    break;
                s_phase ^= 1;
                tc_fence_after();
                if (!idle) {
                    const int pos = (it_t0 + j) * kKeys;
                    const bool tail = pos + kKeys > seq.ctx;
                    const auto see = [&](int i) { return attn_sees32(p, mask, t, pos + 32 * i - seq.ctx, seq); };
                    uint32_t x[32], y[32];
                    // the row's maximum: two loads in flight, four chains
                    float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                    for (int i = 0; i < 4; i += 2) {
                        tmem_ld32_async(ts + 32 * i, x);
                        tmem_ld32_async(ts + 32 * i + 32, y);
                        tmem_wait_ld32(x);
                        tmem_wait_ld32(y);
                        if (tail) {
                            hide(x, see(i));
                            hide(y, see(i + 1));
                        }
#pragma unroll
                        for (int c = 0; c < 32; c += 4)
#pragma unroll
                            for (int v = 0; v < 4; ++v)
                                tops[v] = fmaxf(tops[v], fmaxf(__uint_as_float(x[c + v]), __uint_as_float(y[c + v])));
                    }
                    const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                    const bool grow = top * sc > mc + kGrow || (m == -INFINITY && top > -INFINITY);
                    if (__any_sync(0xFFFFFFFFu, grow)) {
                        const float to_m = fmaxf(m, top);
                        const float to_mc = to_m == -INFINITY ? 0.f : to_m * sc;
                        const float by = m == -INFINITY ? 0.f : ex2(mc - to_mc);
                        m = to_m;
                        mc = to_mc;
                        l *= by;
                        if (units > 0) {  // before the first, the accumulator holds nothing
#pragma unroll 1
                            for (int i = 0; i < D / 32; ++i) {
                                tmem_ld32(to + 32 * i, x);
#pragma unroll
                                for (int c = 0; c < 32; ++c)
                                    x[c] = __float_as_uint(__uint_as_float(x[c]) * by);
                                tmem_st32_async(to + 32 * i, x);
                            }
                        }
                    }
                    const uint64_t sc2 = f32x2(sc, sc), off2 = f32x2(-mc, -mc);
                    uint64_t sums[4] = {0, 0, 0, 0};
                    const auto weigh = [&](const uint32_t(&v)[32], int i) {
                        uint32_t w[16];
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            float a, z;
                            f32x2_unpack(ffma2(f32x2(__uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1])), sc2, off2), a, z);
                            a = ex2(a);
                            z = ex2(z);
                            sums[c & 3] = fadd2(sums[c & 3], f32x2(a, z));
                            w[c] = pack2_bf16(a, z);
                        }
                        tmem_st16_async(ts + 16 * i, w);
                    };
                    // P: the next load runs while this one's columns are worked on; each store goes over
                    // columns that this row has read
                    tmem_ld32_async(ts, x);
#pragma unroll 1
                    for (int i = 0; i < 4; i += 2) {
                        tmem_wait_ld32(x);
                        tmem_ld32_async(ts + 32 * (i + 1), y);
                        if (tail)
                            hide(x, see(i));
                        weigh(x, i);
                        tmem_wait_ld32(y);
                        if (i == 0)
                            tmem_ld32_async(ts + 64, x);
                        if (tail)
                            hide(y, see(i + 1));
                        weigh(y, i + 1);
                    }
                    float a, z;
                    f32x2_unpack(fadd2(fadd2(sums[0], sums[1]), fadd2(sums[2], sums[3])), a, z);
                    l += a + z;
                    tmem_wait_st();
                }
                tc_fence_before();
                mbar_arrive(&sh.p_ready[s]);
            }
            if (ok && units > 0) {
                ok = wait_or_dead(&sh.o_done[s], o_phase, sh, status);
                o_phase ^= 1;
                tc_fence_after();
            }
            // results: with NT = 1 both streams hold sums of every row
            if (NT == 1) {
                sh.m[s][row_in] = m == -INFINITY ? -INFINITY : mc;
                sh.l[s][row_in] = l;
                named_sync(2, kSoftThreads);
            }
            if (ok && !idle) {
                float w0 = 1.f, w1 = 0.f, sum = l, top = m == -INFINITY ? -INFINITY : mc;
                bool two = false;
                if (NT == 1) {
                    const float a = sh.m[0][row_in], z = sh.m[1][row_in];
                    top = fmaxf(a, z);
                    const float ref = top == -INFINITY ? 0.f : top;
                    w0 = ex2(a - ref);
                    w1 = ex2(z - ref);
                    two = n > 1;  // the odd tiles' accumulator holds something
                    sum = w0 * sh.l[0][row_in] + (two ? w1 * sh.l[1][row_in] : 0.f);
                }
                const bool whole = it_t0 == 0 && it_t1 == seq.tiles;
                const float scale = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
                const int h = it_head * p.G + (valid ? row % p.G : 0);
                const size_t at = ((size_t)it_b * p.T + t) * p.q_heads + h;
                const int r = (NT == 2 ? s * 128 : 0) + row_in;
                float *slot = p.part + (size_t)(2 * blockIdx.x + it.slot()) * attn_slot_floats(kRows, D);
                const int wild = *reinterpret_cast<volatile int *>(&sh.wild[item & 3]);
                const int from = it_t0 * kKeys, upto = min(seq.keys, it_t1 * kKeys);
                const uint32_t o0 = tmem + lane_base + 256 + (NT == 2 ? s * 128 : 0), o1 = o0 + 128;
                // NT = 1: each stream's threads write half of the columns
                const int i0 = NT == 1 ? s * (D / 64) : 0, i1 = NT == 1 ? i0 + D / 64 : D / 32;
#pragma unroll 1
                for (int i = i0; i < i1; ++i) {
                    uint32_t x[32];
                    __syncwarp();
                    tmem_ld32(o0 + 32 * i, x);
                    if (NT == 1 && two) {
                        uint32_t y[32];
                        tmem_ld32(o1 + 32 * i, y);
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            x[c] = __float_as_uint(w0 * __uint_as_float(x[c]) + w1 * __uint_as_float(y[c]));
                    }
                    if (!valid)
                        continue;
                    if (whole) {
                        uint4 *out = reinterpret_cast<uint4 *>(p.out + at * D + 32 * i);
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            uint32_t w[4];
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                w[c] = pack2_bf16(__uint_as_float(x[column_of<kType>(8 * v + 2 * c)]) * scale,
                                                  __uint_as_float(x[column_of<kType>(8 * v + 2 * c + 1)]) * scale);
                            out[v] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    } else {
                        float4 *out = reinterpret_cast<float4 *>(slot + (size_t)r * D + 32 * i);
#pragma unroll
                        for (int v = 0; v < 8; ++v)
                            out[v] = make_float4(__uint_as_float(x[column_of<kType>(4 * v)]), __uint_as_float(x[column_of<kType>(4 * v + 1)]),
                                                 __uint_as_float(x[column_of<kType>(4 * v + 2)]), __uint_as_float(x[column_of<kType>(4 * v + 3)]));
                    }
                }
                if (wild && valid) {  // infinities and NaNs of values that the row sees: they are the element's sum
                    for (int d = 32 * i0; d < 32 * i1; ++d) {
                        const float v = attn_wild_values(p, it_b, it_head, t, d, seq.ctx, from, upto);
                        if (finite_f32(v))
                            continue;
                        if (whole)
                            p.out[at * D + d] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
                        else
                            slot[(size_t)r * D + d] = v;
                    }
                }
                if (valid && (NT == 2 || s == 0)) {
                    if (!whole) {
                        slot[(size_t)kRows * D + r] = top;
                        slot[(size_t)kRows * (D + 1) + r] = sum;
                    } else if (p.lse) {
                        p.lse[at] = top == -INFINITY ? (sum == 0.f ? -INFINITY : sum) : (top + log2f(sum)) * 0.6931471805599453f;
                    }
                }
            }
            if (NT == 1)
                named_sync(2, kSoftThreads);  // the accumulators may be used again
            tc_fence_before();
        }
    } else if (warp < kMmaWarp || warp > kLoadWarp) {
        // ---------------------------------------------------------- conversion
        // 8-11, 14, 15 in turn, then the softmax warps without rows (2, 3, 6, 7)
        const int ct = (warp >= 8 ? warp - 8 - (warp > kLoadWarp ? 2 : 0) : 6 + (warp & 1) + (warp >> 2) * 2) * 32 + lane;
        int index = 0;                    // tile slots used so far
        int raw = 0;                      // code slots used so far
        uint32_t go_phase = 0;            // bit s: of go[s]
        uint32_t q_phase = 1;
        bool ok = true;
        for (int item = 0; ok && it.next(p, kKeys); ++item) {
            const SeqLen seq = it.seq;
            const int it_b = it.b, it_head = it.head, it_t0 = it.t0, it_t1 = it.t1, it_block = it.block;  // (the walk itself lives in memory)
            const int n = it_t1 - it_t0, row0 = it_block * kRows;
            if (ct == 0)
                *reinterpret_cast<volatile int *>(&sh.wild[item & 3]) = 0;
            named_sync(1, kConvThreads);
            // the query
            ok = wait_or_dead(&sh.q_empty, q_phase, sh, status);
            q_phase ^= 1;
            if (ok) {
                const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
                // a thread keeps its 16-byte piece of a row and goes down the rows, eight loads in flight
                constexpr int kStep = kConvThreads / kPieces;
                const int x = ct % kPieces;
                int row = row0 + ct / kPieces, t = row / p.G, g = row - t * p.G;
                const uint16_t *q = p.q + (size_t)it_b * p.T * p.q_stride + (size_t)it_head * p.G * D + x * 8;
                for (int r0 = ct / kPieces; r0 < kRows; r0 += 8 * kStep) {
                    uint4 v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        v[i] = row < p.rows ? *reinterpret_cast<const uint4 *>(q + (size_t)t * p.q_stride + g * D) : make_uint4(0, 0, 0, 0);
                        row += kStep;
                        g += kStep;
                        while (g >= p.G) {
                            g -= p.G;
                            ++t;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = r0 + i * kStep;
                        if (r >= kRows)
                            break;
                        uint4 w = make_uint4(v[i].x ^ flip, v[i].y ^ flip, v[i].z ^ flip, v[i].w ^ flip);
                        if (kType == kKvFp8)  // elements (0, 2, 1, 3) of each four
                            w = make_uint4(__byte_perm(w.x, w.y, 0x5410), __byte_perm(w.x, w.y, 0x7632), __byte_perm(w.z, w.w, 0x5410),
                                           __byte_perm(w.z, w.w, 0x7632));
                        sts128(tile_piece(base + P::kQ + (r >> 7) * P::kTileBytes, r & 127, x), w);
                    }
                }
                fence_async_shared();
                named_sync(1, kConvThreads);
                if (ct == 0)
                    mbar_arrive(&sh.q_full);
            }
            // tiles
#pragma unroll 1
            for (int e = 0; ok && e < 2 * n; ++e) {
                int j;
                bool value;
                load_at<NT>(e, n, j, value);
                const int slot = (index + e) % P::kSlots, use = (index + e) / P::kSlots;
                const int pos = (it_t0 + j) * kKeys;
                const bool tail = pos + kKeys > seq.ctx;
                if (kType == kKvBf16) {
                    if (!(value && tail))
                        continue;  // the copy warp's
                    ok = wait_or_dead(&sh.go[slot], (go_phase >> slot) & 1, sh, status);
                    go_phase ^= 1u << slot;
                } else {
                    ok = wait_or_dead(&sh.empty[slot], (use & 1) ^ 1, sh, status);
                }
                if (!ok)
                    break;
                const uint32_t tile = base + slot * P::kTileBytes;
                const int rs = kType == kKvFp8 ? raw % P::kRaw : 0;
                bool wild = false;
                if (kType == kKvFp8) {
                    ok = wait_or_dead(&sh.raw_full[rs], (raw / P::kRaw) & 1, sh, status);
                    if (!ok)
                        break;
                    const uint32_t codes = base + P::kRing + rs * P::kRawBytes;
                    const uint32_t valid = *reinterpret_cast<volatile uint32_t *>(&sh.raw_valid[rs]);
                    // The rows are shared out over kShares warps' worth of threads; warps 8 and 9, whose schedulers
                    // have the narrow softmax and no other conversion, take two shares each. A thread keeps its 16
                    // columns and goes down the rows by kStep, a multiple of 8: every address is its first one plus
                    // a constant.
                    constexpr int kWarps = kConvThreads / 32, kShares = kNarrow ? kWarps + 2 : kWarps;
                    constexpr int kUnits = D / 16, kStep = kShares * 32 / kUnits, kPasses = (kKeys + kStep - 1) / kStep;
                    static_assert(kStep % 8 == 0, "the permutation of a row's pieces");
                    const uint8_t *src = smem_raw + (codes - smem_addr(smem_raw));
#pragma unroll 1
                    for (int share = ct; share < kShares * 32; share += kConvThreads) {
                        const int r0 = share / kUnits, x = share % kUnits;
                        // half of the lanes convert and store their second 8 columns first, so that a store's lanes meet
                        // no bank twice
                        const bool swap = (x >> 2) & 1;
                        const uint32_t a = tile_piece(tile, r0, 2 * x + swap), b = tile_piece(tile, r0, 2 * x + !swap);
                        const bool last = r0 + kStep * (kPasses - 1) < kKeys;  // the same for a warp
                        const uint8_t *at = src + r0 * D + x * 16;
                        uint4 in[kPasses];
                        int byte[kPasses], most = 0;
#pragma unroll
                        for (int i = 0; i < kPasses; ++i)
                            if (i + 1 < kPasses || last) {
                                in[i] = *reinterpret_cast<const uint4 *>(at + kStep * i * D);
                                byte[i] = src[P::kRawCodes + r0 + kStep * i];
                                most = max(most, byte[i]);
                            }
                        // Whole tiles of the context whose rows' factors are bf16 go straight through; branches
                        // inside this loop cost more than its arithmetic (2020 cycles a tile against 3300 unrolled
                        // with them, 16 warps of four kinds of code sharing the instruction caches).
                        const bool plain = !(tail && value) && valid == 0xFFu && most <= 134;
                        if (__all_sync(0xFFFFFFFFu, plain)) {
#pragma unroll
                            for (int i = 0; i < kPasses; ++i)
                                if (i + 1 < kPasses || last) {
                                    const uint32_t f = (uint32_t)(120 + byte[i]) << 7;
                                    sts128(a + kStep * i * 128, fp8_to_bf16(swap ? in[i].z : in[i].x, swap ? in[i].w : in[i].y, f));
                                    sts128(b + kStep * i * 128, fp8_to_bf16(swap ? in[i].x : in[i].z, swap ? in[i].y : in[i].w, f));
                                }
                        } else {
#pragma unroll 1
                            for (int i = 0; i < kPasses; ++i) {
                                const int r = r0 + kStep * i;
                                if (r >= kKeys)
                                    break;
                                const int by = src[P::kRawCodes + r];
                                uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
                                bool use_it = (valid >> (r >> 4)) & 1u;
                                if (tail && value && pos + r >= seq.ctx) {
                                    if (pos + r >= seq.keys) {
                                        use_it = false;
                                    } else if (by == kFp8BadRow) {
                                        wild |= use_it;
                                        use_it = false;
                                    }
                                }
                                if (use_it) {
                                    const uint4 v = *reinterpret_cast<const uint4 *>(at + kStep * i * D);
                                    const bool big = by > 134 && by != kFp8BadRow;  // its factor is not a bf16: two steps
                                    const uint32_t f = by == kFp8BadRow ? 0x7FC0u : big ? 0x7B80u : (uint32_t)(120 + by) << 7;
                                    lo = fp8_to_bf16(v.x, v.y, f);
                                    hi = fp8_to_bf16(v.z, v.w, f);
                                    if (big) {
                                        const uint32_t g = (uint32_t)by << 7 | (uint32_t)by << 23;
                                        lo = make_uint4(mul_bf16x2(lo.x, g), mul_bf16x2(lo.y, g), mul_bf16x2(lo.z, g), mul_bf16x2(lo.w, g));
                                        hi = make_uint4(mul_bf16x2(hi.x, g), mul_bf16x2(hi.y, g), mul_bf16x2(hi.z, g), mul_bf16x2(hi.w, g));
                                    }
                                }
                                sts128(a + kStep * i * 128, swap ? hi : lo);
                                sts128(b + kStep * i * 128, swap ? lo : hi);
                            }
                        }
                    }
                } else {  // bf16 values that reach past the context
#pragma unroll 4
                    for (int u = ct; u < kKeys * kPieces; u += kConvThreads) {
                        const int r = u / kPieces, x = u % kPieces, at = pos + r;
                        uint4 v = make_uint4(0, 0, 0, 0);
                        const long page = at < seq.keys ? kv_page(p.c, it_b, at) : -1;
                        if (page >= 0) {
                            v = *reinterpret_cast<const uint4 *>(p.c.v + (kv_row(p.c, page, it_head, at) * D + x * 8) * 2);
                            if (at >= seq.ctx) {
                                uint32_t *w = &v.x;
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const bool lo = (w[i] & 0x7F80u) == 0x7F80u, hi = (w[i] & 0x7F800000u) == 0x7F800000u;
                                    if (lo || hi) {
                                        wild = true;
                                        w[i] &= (lo ? 0xFFFF0000u : ~0u) & (hi ? 0x0000FFFFu : ~0u);
                                    }
                                }
                            }
                        }
                        sts128(tile_piece(tile, r, x), v);
                    }
                }
                if (wild)
                    *reinterpret_cast<volatile int *>(&sh.wild[item & 3]) = 1;
                fence_async_shared();
                named_sync(1, kConvThreads);
                if (ct == 0) {
                    mbar_arrive(&sh.full[slot]);
                    if (kType == kKvFp8)
                        mbar_arrive(&sh.raw_empty[rs]);
                }
                ++raw;
            }
            index += 2 * n;
        }
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------- products
        constexpr uint32_t kIdescS = umma_idesc_bf16(128, kKeys), kIdescO = umma_idesc_bf16(128, D) | kIdescBMnMajor;
        int index = 0;
        uint32_t q_phase = 0, p_phase[2] = {0, 0};
        bool ok = true;
        while (ok && it.next(p, kKeys)) {
            const int n = it.t1 - it.t0, units = NT == 2 ? 2 * n : n;
            ok = wait_or_dead(&sh.q_full, q_phase, sh, status);
            q_phase ^= 1;
            if (!ok)
                break;
            const auto scores = [&](int u) {
                const int s = u & 1, j = NT == 2 ? u >> 1 : u, e = index + key_index<NT>(j);
                const int slot = e % P::kSlots;
                if (!wait_or_dead(&sh.full[slot], (e / P::kSlots) & 1, sh, status))
                    return false;
                tc_fence_after();
                const uint32_t q = desc_lo(base + P::kQ + (NT == 2 ? s * P::kTileBytes : 0), 16);
                const uint32_t k = desc_lo(base + slot * P::kTileBytes, 16);
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const uint32_t at = ((i >> 2) * P::kHalf + (i & 3) * 32) >> 4;
                        umma_bf16_lo(tmem + s * kKeys, q + at, k + at, kIdescS, i > 0);
                    }
                    umma_commit(&sh.s_ready[s]);
                    if (NT == 1 || s == 1)
                        umma_commit(&sh.empty[slot]);
                    if (u == units - 1)
                        umma_commit(&sh.q_empty);
                }
                __syncwarp();
                return true;
            };
#pragma unroll 1
            for (int u = -2; ok && u < units; ++u) {
                if (u < 0) {  // two score products ahead
                    if (u + 2 < units)
                        ok = scores(u + 2);
                    continue;
                }
                const int s = u & 1, j = NT == 2 ? u >> 1 : u, e = index + value_index<NT>(j, n);
                const int slot = e % P::kSlots;
                ok = wait_or_dead(&sh.full[slot], (e / P::kSlots) & 1, sh, status) &&
                     wait_or_dead(&sh.p_ready[s], p_phase[s], sh, status);
                if (!ok)
                    break;
                p_phase[s] ^= 1;
                tc_fence_after();
                const uint32_t v = desc_lo(base + slot * P::kTileBytes, P::kHalf);
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < kKeys / 16; ++i)
                        umma_bf16_ts_lo(tmem + 256 + s * 128, tmem + s * kKeys + i * 8, v + i * (2048 >> 4), kIdescO, i > 0 || u >= 2);
                    if (NT == 1 || s == 1)
                        umma_commit(&sh.empty[slot]);
                    if (u + 2 >= units)
                        umma_commit(&sh.o_done[s]);
                }
                __syncwarp();
                if (u + 2 < units)
                    ok = scores(u + 2);
            }
            index += 2 * n;
        }
    } else {
        // ---------------------------------------------------------- copies
        const int per_page = min(kKeys, 1 << p.c.page_shift);  // keys of a chunk that lies in one page
        const int chunks = kKeys / per_page;                   // at most 8
        const long total_rows = (p.c.n_pages * p.c.heads) << p.c.page_shift;
        int index = 0, raw = 0;
        bool ok = true;
        if (kType == kKvBf16 && lane == 0) {
            tma_prefetch_map(&map_k);
            tma_prefetch_map(&map_v);
        }
        while (ok && it.next(p, kKeys)) {
            const SeqLen seq = it.seq;
            const int it_b = it.b, it_head = it.head, it_t0 = it.t0, it_t1 = it.t1;  // (the walk itself lives in memory)
            const int n = it_t1 - it_t0;
            // pages: lane 8 i + c holds chunk c of tile 4 g + i, for the group g being loaded and its neighbours
            const auto pages_of = [&](int g) {
                const int j = 4 * g + (lane >> 3), c = lane & 7;
                const long pos = (long)(it_t0 + j) * kKeys + c * per_page;
                return j < n && c < chunks && pos < seq.keys ? (int)kv_page(p.c, it_b, pos) : -1;
            };
            int before = -1, now = pages_of(0), after = pages_of(1), group = 0;
#pragma unroll 1
            for (int e = 0; ok && e < 2 * n; ++e) {
                int j;
                bool value;
                load_at<NT>(e, n, j, value);
                if (!value && (j >> 2) != group) {
                    before = now;
                    now = after;
                    group = j >> 2;
                    after = pages_of(group + 1);
                }
                const int page = __shfl_sync(0xFFFFFFFFu, (j >> 2) == group ? now : before, (j & 3) * 8 + (lane & 7));
                const int pos = (it_t0 + j) * kKeys, mine = pos + lane * per_page;
                const bool chunk = lane < chunks, there = chunk && page >= 0;
                if (chunk && page < 0 && mine < seq.keys && status)
                    atomicExch(status, kStatusBadArg);
                const long row = there ? (long)kv_row(p.c, page, it_head, mine) : total_rows;
                if (kType == kKvBf16) {
                    const int slot = (index + e) % P::kSlots;
                    ok = wait_or_dead(&sh.empty[slot], (((index + e) / P::kSlots) & 1) ^ 1, sh, status);
                    if (!ok)
                        break;
                    if (value && pos + kKeys > seq.ctx) {  // the conversion warps' to fill
                        if (lane == 0)
                            mbar_arrive(&sh.go[slot]);
                        continue;
                    }
                    if (lane == 0)
                        mbar_arrive_expect_tx(&sh.full[slot], P::kTileBytes);
                    __syncwarp();
                    if (chunk) {  // a chunk without a page is read past the last row: zeros
                        uint8_t *dst = smem_raw + (base - smem_addr(smem_raw)) + slot * P::kTileBytes + lane * per_page * 128;
#pragma unroll
                        for (int h = 0; h < D / 64; ++h)
                            tma_load_2d(dst + h * P::kHalf, value ? &map_v : &map_k, h * 64, (int)row, &sh.full[slot]);
                    }
                    __syncwarp();
                } else {
                    const int rs = raw % P::kRaw;
                    ok = wait_or_dead(&sh.raw_empty[rs], ((raw / P::kRaw) & 1) ^ 1, sh, status);
                    if (!ok)
                        break;
                    const unsigned have = __ballot_sync(0xFFFFFFFFu, there);
                    if (lane == 0) {
                        uint32_t bits = 0;
                        for (int c = 0; c < chunks; ++c)
                            if ((have >> c) & 1u)
                                bits |= ((1u << (per_page / 16)) - 1u) << (c * (per_page / 16));
                        *reinterpret_cast<volatile uint32_t *>(&sh.raw_valid[rs]) = bits;
                        mbar_arrive_expect_tx(&sh.raw_full[rs], __popc(have) * per_page * (D + 1));
                    }
                    __syncwarp();
                    if (there) {
                        uint8_t *dst = smem_raw + (base - smem_addr(smem_raw)) + P::kRing + rs * P::kRawBytes;
                        bulk_copy_g2s(dst + lane * per_page * D, (value ? p.c.v : p.c.k) + row * D, per_page * D, &sh.raw_full[rs]);
                        bulk_copy_g2s(dst + P::kRawCodes + lane * per_page, (value ? p.c.vs : p.c.ks) + row, per_page, &sh.raw_full[rs]);
                    }
                    __syncwarp();
                    ++raw;
                }
            }
            index += 2 * n;
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*reinterpret_cast<volatile int *>(&sh.dead)) {
        // a wait ran out: copies and products may still be in flight; give them time before the memory goes
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 50000000ull) {}
        __syncthreads();
    }
    if (warp == kMmaWarp)
        tmem_dealloc(tmem, kTmemCols);
}

constexpr int kLeastWide = 2;  // tiles a CTA has at least, where there is a choice

template <int kType, int D, int NT, bool kNarrow = false>
cudaError_t launch_wide(AttnParams p, const LaunchCfg &cfg, cudaStream_t stream)
{
    using Pl = Plan<kType, D, NT, kNarrow>;
    auto *kernel = hc_attn_wide_kernel<kType, D, NT, kNarrow>;
    static_assert(Pl::kTotal + sizeof(Shared<NT>) <= 227 * 1024, "shared memory");
    static const cudaError_t set = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Pl::kTotal);
    if (set != cudaSuccess)
        return set;
    p.row_blocks = (p.rows + 128 * NT - 1) / (128 * NT);
    CUtensorMap map_k{}, map_v{};
    if (kType == kKvBf16) {
        const uint64_t rows = (uint64_t)p.c.n_pages * p.c.heads << p.c.page_shift;
        const uint32_t box = (uint32_t)std::min(kKeys, 1 << p.c.page_shift);
        if (!tc_make_map_2d(&map_k, p.c.k, rows, D, 64, box) || !tc_make_map_2d(&map_v, p.c.v, rows, D, 64, box))
            return cudaErrorInvalidValue;
    }
    cudaLaunchConfig_t lc{};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = at;
    lc.numAttrs = 1;
    lc.stream = stream;
    lc.blockDim = dim3(kThreads);
    const int grid = std::min(cfg.sm_count, kAttnWideGrid);
    lc.gridDim = dim3(grid);
    lc.dynamicSmemBytes = Pl::kTotal;
    cudaError_t e = cudaLaunchKernelEx(&lc, kernel, p, map_k, map_v, kLeastWide);
    if (e != cudaSuccess)
        return e;
    return launch_attn_join(p, 128 * NT, kKeys, grid, kLeastWide, stream);
}

}  // namespace

// Rows of a block of the wide kernel, or 0 where it does not serve: more than 32
// rows; head_dim 64 or 128 (two accumulators and two score tiles fill TMEM); bf16
// and FP8 rows (an INT4 key's exact value does not fit a bf16); fewer rows in the
// pool than a tensor map's coordinates reach.
int attn_wide_rows(const KvView &c, long rows)
{
    if (rows <= 32 || c.D == 256 || c.type == kKvInt4)
        return 0;
    if (((c.n_pages * c.heads) << c.page_shift) >= (1l << 31) - kKeys)
        return 0;
    return rows <= 128 ? 128 : 256;
}

cudaError_t launch_attn_wide(const AttnParams &p, const LaunchCfg &cfg, cudaStream_t stream)
{
    const bool two = attn_wide_rows(p.c, p.rows) == 256;
    if (p.c.type == kKvBf16) {
        if (p.c.D == 64)
            return two ? launch_wide<kKvBf16, 64, 2>(p, cfg, stream) : launch_wide<kKvBf16, 64, 1>(p, cfg, stream);
        return two ? launch_wide<kKvBf16, 128, 2>(p, cfg, stream) : launch_wide<kKvBf16, 128, 1>(p, cfg, stream);
    }
    const bool narrow = p.rows <= 64;
    if (p.c.D == 64)
        return two ? launch_wide<kKvFp8, 64, 2>(p, cfg, stream)
                   : narrow ? launch_wide<kKvFp8, 64, 1, true>(p, cfg, stream) : launch_wide<kKvFp8, 64, 1>(p, cfg, stream);
    return two ? launch_wide<kKvFp8, 128, 2>(p, cfg, stream)
               : narrow ? launch_wide<kKvFp8, 128, 1, true>(p, cfg, stream) : launch_wide<kKvFp8, 128, 1>(p, cfg, stream);
}

}  // namespace tshc
