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
// Roles: warps 0-7 softmax, four a stream; warps 8-11, 14 and 15 put
// what has to be converted into shared memory (the query; FP8 tiles; the values of
// a tile that reaches past the context, where what lies behind the last key, and
// infinities and NaNs of nodes, are taken out; INT4 tiles: a key as the sum of two bf16, a
// value in fp16); warp 12 issues the products, warp 13 the copies: TMA boxes for bf16
// tiles, bulk copies of codes to a ring of their own.
//
// Blocks of 64 rows or fewer (kNarrow) have the query's rows twice in a tile, on lanes
// 0-63 and 64-127, and each stream works on a copy of its own: a row's softmax is two
// threads' work, each with half of the columns, which stay in registers from the maximum
// to the weights, and the two streams' warps are spread over all four schedulers. FP8
// keys then go into the product as the codes that they are: the query is split into two
// e4m3 parts, whose products with the codes are exact, and the keys' scales go to the
// scores. 4 x 64 rows over 65536 FP8 keys: converted keys 165 us, codes 156, two threads
// a row 130, scores in registers 111. (For more rows there is no lane left for a copy, and
// the conversion is hidden as well: some 160 us for 96 rows either way.)
//
// As in hc_attn.cu, a row's sums are divided by the sum of the weights as they were
// rounded, which costs some 2% (119.6 -> 123 us, 110 -> 112, when it was taken) and takes the results'
// mean error against 64 bits from 1.3 times a plain fp32 form's to 1.15 (the root of its mean
// square, over |out|'s, is 0.0020 to 0.0022, the plain form's, which is the result's own rounding,
// 0.0017).
//
// What bounds it (GPU times of a call, the join included, replayed back to back in a CUDA
// graph): 4 x 512 rows over 16384 bf16 keys take 119 us, 55 of them tensor-core
// time: a stream's chain of product, softmax and product, of some 3500 cycles a tile
// against 2048 of products. 4 x 64 rows over 32768 bf16 keys, 81 us for 60 of bytes: five
// tiles in shared memory are what is in flight. 64 FP8 rows, 109 us for 60 of bytes: the
// softmax's chain, the conversion of the values and the copy warp's instructions, each
// some 2000 of the 2400 cycles a tile.
//
// Every wait is bounded; the first that runs out records TS_ERR_TIMEOUT and ends
// the others.
#include <algorithm>

#include "hc_attn.cuh"
#include "hc_tc.h"
#include "umma.cuh"

namespace tshc {

namespace {

constexpr int kKeys = 128;               // keys of a tile
constexpr int kSoftThreads = 256, kConvThreads = 192;
constexpr int kThreads = kSoftThreads + kConvThreads + 64;  // 16 warps: the most that leaves 128 registers a thread
constexpr int kMmaWarp = 12, kLoadWarp = 13;
constexpr float kGrow = 8.f;             // log2: how far a row's maximum may grow over its reference
constexpr uint32_t kTmemCols = 512;      // S of two streams, O of two streams

// kNarrow: 64 rows or fewer.
template <int kType, int D, int NT, bool kNarrow>
struct Plan {
    static constexpr int kTileBytes = kKeys * D * 2;              // a tile's keys or values as bf16
    static constexpr int kHalf = kKeys * 128;                     // 64 columns of it
    static constexpr int kQBytes = NT * kTileBytes;
    static constexpr bool kCoded = kType != kKvBf16;
    static constexpr int kRawRow = kType == kKvFp8 ? D : D / 2;   // bytes of a row's codes
    static constexpr int kRawCodes = kKeys * kRawRow;             // a tile's, with its rows' scales (INT4: scales, then biases)
    static constexpr int kRawScales = kType == kKvFp8 ? 256 : kKeys * (D / 32) * 2;
    static constexpr int kRawBytes = !kCoded ? 0 : kType == kKvFp8 ? kRawCodes + kRawScales : kRawCodes + 2 * kRawScales;
    static constexpr int kExchange = kNarrow ? 2 * 64 * 36 * 4 : 0;  // 32 columns of 64 rows, twice, rows 36 floats apart
    static constexpr int kBudget = (NT == 1 ? 220 : 222) * 1024 - kQBytes - kExchange;  // beside the barriers and tables
    // Narrow blocks' FP8 keys go into the products as they lie in the cache, so that only values are converted.
    static constexpr bool kRawKeys = kNarrow && kType == kKvFp8 && D == 128;  // a row is one 128-byte line of an operand
    // An INT4 key's value is kept as the sum of two bf16 tiles (16 bits of significand), one behind the other.
    static constexpr int kKeyBytes = kRawKeys ? kKeys * D : kType == kKvInt4 ? 2 * kTileBytes : kTileBytes;
    // Key tiles are needed two products ahead, value tiles (and, FP8, their codes) a little later. 256 FP8 rows have
    // room for three converted tiles: one of keys, which both products are through with early, and two of values
    // (4 x 512 rows over 16384 keys: 125 us; when it was taken 139, two of keys and one of values 156).
    static constexpr int kKeySlots = kRawKeys ? 3 : D == 64 ? 4 : kType == kKvInt4 || (kType == kKvFp8 && NT == 2) ? 1 : 2;
    static constexpr int kSlots = kCoded ? 2 : std::min(8, (kBudget - kKeySlots * kKeyBytes) / kTileBytes);
    static constexpr int kRaw = kCoded ? std::min(8, (kBudget - kSlots * kTileBytes - kKeySlots * kKeyBytes) / kRawBytes) : 1;
    static constexpr int kQ = kSlots * kTileBytes, kKeyRing = kQ + kQBytes, kRing = kKeyRing + kKeySlots * kKeyBytes;
    static constexpr int kTrade = kRing + kRaw * kRawBytes, kTotal = kTrade + kExchange + 1024;  // and alignment
    static_assert(!kCoded || kRaw >= 2, "codes of a tile's keys and values");
};

constexpr int kScaleSlots = 8;  // of the keys' scales: they are read until a tile's softmax is through, two units after its product

template <int NT, bool kRawKeys, bool kNarrow>
struct Shared {
    // Each barrier has one role that waits on it, or waiters whose own arrivals its next phase needs: a
    // parity tells a phase from the next only, so that nobody may fall a phase behind.
    uint64_t full[8], empty[8];          // a value slot
    uint64_t go[8];                      // bf16: an empty value slot is the conversion warps' to fill
    uint64_t raw_full[8], raw_empty[8];  // an FP8 code slot
    uint64_t k_full[4], k_empty[4];      // a key slot
    uint64_t q_full, q_empty;
    uint64_t s_ready[2], p_half[2], p_ready[2], o_done[2];
    uint32_t tmem;
    int dead;                            // a wait ran out
    int wild[4];                         // by item: a node's value held an infinity or a NaN
    uint32_t raw_valid[8];               // which 16-key chunks of a code slot lie in a page
    float m[2][NT == 1 ? 128 : 1], l[2][NT == 1 ? 128 : 1], lr[2][NT == 1 ? 128 : 1];  // of the two streams
    alignas(16) uint8_t key_scale[kRawKeys ? kScaleSlots : 1][128];
    alignas(16) float factor[2][2][kRawKeys ? 128 : 4];      // of a stream's tile, by turns: its keys' scales times log2(e) scale
    float q_scale[2][kRawKeys ? 64 : 1];                     // of the query's rows, by items in turn
    float top[2][2][2][kNarrow ? 64 : 1];                   // of a stream's tile, by turns: each column half's maxima
    LineScratch line;
};

// Waits for the phase; false when it (or another wait of the block) ran out. The
// warp's lanes leave together with one answer. (One lane looking for all of them
// was slower: 165 us against 132 for 4 x 64 nodes over 16384 bf16 keys.)
template <typename S>
__device__ __forceinline__ bool wait_or_dead(uint64_t *bar, uint32_t parity, S &sh, unsigned *status)
{
    bool there = mbar_try_wait(bar, parity);
    if (!there) {
        const uint64_t t0 = global_timer_ns();
        for (;;) {
            if (*reinterpret_cast<volatile int *>(&sh.dead))
                break;
#pragma unroll 1
            for (int i = 0; i < 16 && !there; ++i)
                there = mbar_try_wait(bar, parity);
            if (there)
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

// The conversion of FP8 leaves elements (0, 2, 1, 3) of each four, that of INT4
// (0, 4, 1, 5, 2, 6, 3, 7) of each eight. The query takes the same order against converted
// keys, and the results are put back when they are written.
template <int kType>
__device__ __forceinline__ constexpr int column_of(int d)
{
    return kType == kKvFp8 ? (d & ~3) | ((d & 1) << 1) | ((d >> 1) & 1) : kType == kKvInt4 ? (d & ~7) | ((d & 3) << 1) | ((d >> 2) & 1) : d;
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


// Eight elements of a query row, 16 lanes a row, as two e4m3 parts: the row is scaled by
// the smallest power of two that brings it to at most 448, the first part is its nearest
// e4m3, the second the rest's. A bf16 has 8 significant bits, each part 4: the sum is
// exact for scaled elements of 2^-2 or more and off by at most 2^-10, half of e4m3's least
// spacing, for smaller ones; the row's largest is more than 224, so that is at most 2^-17.8
// of it. Returns the scale to undo (NaN for a row with an infinity
// or a NaN).
__device__ __forceinline__ float split_e4m3(const uint4 q, uint2 &hi, uint2 &lo)
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        top = __vmaxu2(top, w[i] & 0x7FFF7FFFu);
    const unsigned lanes = 0xFFFFu << (threadIdx.x & 16);  // the row's
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
        top = __vmaxu2(top, __shfl_xor_sync(lanes, top, o));
    top = max(top & 0xFFFFu, top >> 16);
    const bool bad = top >= 0x7F80u;
    const int byte = fp8_scale_byte(__uint_as_float(top << 16));
    const float inv = bad ? 0.f : __uint_as_float((uint32_t)(254 - byte) << 23);
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = make_float2(bf16_lo(w[i]) * inv, bf16_hi(w[i]) * inv);
        h[i] = __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
        const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)h[i], __NV_E4M3)));
        l[i] = __nv_cvt_float2_to_fp8x2(make_float2(v.x - f.x, v.y - f.y), __NV_SATFINITE, __NV_E4M3);
    }
    hi = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
    lo = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
    return bad ? __uint_as_float(0x7FC00000u) : __uint_as_float((uint32_t)byte << 23);
}

// Address of 16-byte piece x (8 columns) of row r in a 128-row tile of D columns.
__device__ __forceinline__ uint32_t tile_piece(uint32_t tile, int r, int x)
{
    return tile + (uint32_t)(x >> 3) * (kKeys * 128) + (uint32_t)r * 128 + (uint32_t)(((x & 7) ^ (r & 7)) << 4);
}

// Scores times their columns' factors (one address for all lanes).
__device__ __forceinline__ void scale_columns(uint32_t (&x)[32], const float *factor)
{
#pragma unroll
    for (int c = 0; c < 32; c += 4) {
        const float4 f = *reinterpret_cast<const float4 *>(factor + c);
        x[c] = __float_as_uint(__uint_as_float(x[c]) * f.x);
        x[c + 1] = __float_as_uint(__uint_as_float(x[c + 1]) * f.y);
        x[c + 2] = __float_as_uint(__uint_as_float(x[c + 2]) * f.z);
        x[c + 3] = __float_as_uint(__uint_as_float(x[c + 3]) * f.w);
    }
}

// sum += both halves of w.
template <bool kHalf>
__device__ __forceinline__ void add_pair(float &sum, uint32_t w)
{
    if (kHalf)
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tadd.f32.f16 %0, lo, %0;\n\tadd.f32.f16 %0, hi, %0;\n\t}" : "+f"(sum) : "r"(w));
    else
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tadd.f32.bf16 %0, lo, %0;\n\tadd.f32.bf16 %0, hi, %0;\n\t}" : "+f"(sum) : "r"(w));
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
    constexpr int kRows = 128 * NT;
    constexpr int kPieces = D / 8;
    extern __shared__ uint8_t smem_raw[];
    constexpr bool kRawKeys = P::kRawKeys, kCoded = P::kCoded;
    constexpr bool kHalf = kType == kKvInt4;  // weights and values in fp16, which holds an INT4 value's 11 bits
    constexpr float kLift = kHalf ? kFp16Lift : 0.f;
    __shared__ Shared<NT, kRawKeys, kNarrow> sh;
    pdl_wait();
    pdl_launch_dependents();  // after the wait: the join reads the lengths before its own
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;

    const Line<> line(p, kKeys, sh.line);
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
        for (int i = 0; i < 4; ++i) {
            mbar_init(&sh.k_full[i], 1);
            mbar_init(&sh.k_empty[i], 1);
        }
        mbar_init(&sh.q_full, 1);
        mbar_init(&sh.q_empty, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh.s_ready[s], 1);
            mbar_init(&sh.p_half[s], kSoftThreads / 2);
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

    if (warp < 8) {
        // ---------------------------------------------------------- softmax
        // A stream's warps: four, one for each 32 rows; narrow, four too, two for each 32 of 64 rows, with half
        // of the columns each: the query's rows lie twice in its tile, and the streams take the copies on
        // different lanes, so that all schedulers have their part of both.
        const int s = kNarrow ? (warp >> 1) & 1 : warp >> 2, half = kNarrow ? warp >> 2 : 0;
        const int row_in = tid & (kNarrow ? 63 : 127);
        constexpr int kCols = kNarrow ? 64 : 128, kChunks = kCols / 32;  // a thread's columns
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lane_base + s * kKeys + half * 64, to = tmem + lane_base + 256 + s * 128 + half * (D / 2);
        const float sc = fmaxf(fabsf(p.scale_log2), 1e-38f);  // its sign went into the query; not 0, for masked scores' sake
        uint32_t s_phase = 0, o_phase = 0;
        int key_tile = 0, turn = 0;       // raw keys: tiles before this item's
        // (A wait that ran out ends nothing here: the warps go on through the same barriers, on whatever lies
        // there, and every further wait returns at once.)
        for (int item = 0; it.next(p, kKeys); ++item) {
            const SeqLen seq = it.seq;
            const int it_b = it.b, it_head = it.head, it_t0 = it.t0, it_t1 = it.t1, it_block = it.block;
            if (seq.bad && tid == 0 && status)
                atomicExch(status, kStatusBadArg);
            const int n = it_t1 - it_t0, row0 = it_block * kRows;
            const int row = row0 + (NT == 2 ? s * 128 : 0) + row_in;
            const bool valid = row < p.rows;
            const int t = valid ? row / p.G : 0;
            const uint32_t *mask = attn_mask_row(p, it_b, t);
            // a warp of rows past the last has nothing to do (rows do not meet)
            const bool idle = !kNarrow && row0 + (NT == 2 ? s * 128 : 0) + (warp & 3) * 32 >= p.rows;
            float m = -INFINITY, l = 0.f, lr = 0.f;  // the reference (in units of log2), the weights' sum, that of the rounded weights
            int units = 0;
            float q_scale = 1.f;
            for (int j = NT == 2 ? 0 : s; j < n; j += 3 - NT, ++units) {
                wait_or_dead(&sh.s_ready[s], s_phase, sh, status);
                s_phase ^= 1;
                tc_fence_after();
                const float *factor = sh.factor[s][turn] + half * 64;
                if (kRawKeys) {  // the tile's factors, one a thread
                    const int i = half * 64 + row_in;
                    sh.factor[s][turn][i] = fp8_scale(sh.key_scale[(key_tile + j) % kScaleSlots][i]) * sc;
                    if (units == 0)
                        q_scale = sh.q_scale[item & 1][row_in];
                    named_sync(3 + s, kSoftThreads / 2);
                }
                turn ^= 1;
                if (!idle) {
                    const int pos = (it_t0 + j) * kKeys;
                    const bool tail = pos + kKeys > seq.ctx;
                    const auto see = [&](int i) { return attn_sees32(p, mask, t, pos + half * 64 + 32 * i - seq.ctx, seq); };
                    uint32_t x[32], y[32];
                    // the row's maximum: two loads in flight, four chains
                    float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                    for (int i = 0; i < kChunks; i += 2) {
                        tmem_ld32_async(ts + 32 * i, x);
                        tmem_ld32_async(ts + 32 * i + 32, y);
                        tmem_wait_ld32(x);
                        tmem_wait_ld32(y);
                        if (kRawKeys) {
                            scale_columns(x, factor + 32 * i);
                            scale_columns(y, factor + 32 * i + 32);
                        }
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
                    // with raw keys the scores have the factor already, and the query row's scale is still to come
                    const float by_row = kRawKeys ? q_scale : sc;
                    float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                    if (kNarrow) {  // the row's other half
                        sh.top[s][turn][half][row_in] = top;
                        named_sync(5 + s, kSoftThreads / 2);
                        top = fmaxf(top, sh.top[s][turn][half ^ 1][row_in]);
                    }
                    top *= by_row;
                    if (__any_sync(0xFFFFFFFFu, top > m + (kGrow + kLift))) {  // also the first that is not -infinity
                        const float to_m = fmaxf(m, top - kLift), by = ex2(m - (to_m == -INFINITY ? 0.f : to_m));
                        m = to_m;
                        l *= by;
                        lr *= by;
                        if (units > 0) {  // before the first, the accumulator holds nothing
                            uint32_t z[16];
#pragma unroll 1
                            for (int i = 0; i < (kNarrow ? D / 32 : D / 16); ++i) {
                                tmem_ld16_async(to + 16 * i, z);
                                tmem_wait_ld(z);
#pragma unroll
                                for (int c = 0; c < 16; ++c)
                                    z[c] = __float_as_uint(__uint_as_float(z[c]) * by);
                                tmem_st16_async(to + 16 * i, z);
                            }
                        }
                    }
                    const float off = m == -INFINITY ? 0.f : -m;
                    const uint64_t sc2 = f32x2(by_row, by_row), off2 = f32x2(off, off);
                    uint64_t sums[4] = {0, 0, 0, 0};
                    float rounded[2] = {0.f, 0.f};
                    const auto weigh = [&](const uint32_t(&v)[32], int i) {
                        uint32_t w[16];
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            float a, z;
                            f32x2_unpack(ffma2(f32x2(__uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1])), sc2, off2), a, z);
                            a = ex2(a);
                            z = ex2(z);
                            sums[c & 3] = fadd2(sums[c & 3], f32x2(a, z));
                            w[c] = kHalf ? pack2_f16(a, z) : pack2_bf16(a, z);
                            add_pair<kHalf>(rounded[c & 1], w[c]);
                        }
                        tmem_st16_async(ts + 16 * i, w);
                    };
                    if (kNarrow) {  // the registers still hold all of the thread's scores
                        weigh(x, 0);
                        weigh(y, 1);
                    } else {
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
                            if (i == 0) {  // the product can begin with the first 64 keys
                                tmem_wait_st();
                                tc_fence_before();
                                mbar_arrive(&sh.p_half[s]);
                            }
                        }
                    }
                    float a, z;
                    f32x2_unpack(fadd2(fadd2(sums[0], sums[1]), fadd2(sums[2], sums[3])), a, z);
                    l += a + z;
                    lr += rounded[0] + rounded[1];
                    tmem_wait_st();
                } else {
                    mbar_arrive(&sh.p_half[s]);
                }
                tc_fence_before();
                mbar_arrive(&sh.p_ready[s]);
            }
            if (units > 0) {
                wait_or_dead(&sh.o_done[s], o_phase, sh, status);
                o_phase ^= 1;
                tc_fence_after();
            }
            // results: with NT = 1 both streams hold sums of every row
            if (NT == 1) {
                if (half == 0)
                    sh.m[s][row_in] = m;
                sh.l[s][half * 64 + row_in] = l;
                sh.lr[s][half * 64 + row_in] = lr;
                named_sync(2, kSoftThreads);
            }
            if (!idle) {
                // the weights' sum over the rounded weights' makes up for the rounding (as in hc_attn.cu)
                const auto made_up = [](float sum, float rounded) { return rounded == 0.f ? 1.f : sum / rounded; };
                float w0 = 1.f, w1 = 0.f, sum = l, top = m;
                bool two = false;
                if (NT == 1) {
                    const float a = sh.m[0][row_in], z = sh.m[1][row_in];
                    top = fmaxf(a, z);
                    const float ref = top == -INFINITY ? 0.f : top;
                    w0 = ex2(a - ref);
                    w1 = ex2(z - ref);
                    two = n > 1;  // the odd tiles' accumulator holds something
                    float l0 = sh.l[0][row_in], l1 = sh.l[1][row_in], r0 = sh.lr[0][row_in], r1 = sh.lr[1][row_in];
                    if (kNarrow) {
                        l0 += sh.l[0][64 + row_in];
                        l1 += sh.l[1][64 + row_in];
                        r0 += sh.lr[0][64 + row_in];
                        r1 += sh.lr[1][64 + row_in];
                    }
                    sum = w0 * l0 + (two ? w1 * l1 : 0.f);
                    w0 *= made_up(l0, r0);
                    w1 *= made_up(l1, r1);
                } else {
                    w0 = made_up(l, lr);
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
                // NT = 1: each stream's threads write half of the columns; narrow, the second stream hands its
                // part of the sums, which lies on other lanes, to the first, which writes
                const int i0 = kNarrow ? D / 64 * half : NT == 1 ? s * (D / 64) : 0, i1 = NT == 1 ? i0 + D / 64 : D / 32;
                float *trade = reinterpret_cast<float *>(smem_raw + (base - smem_addr(smem_raw)) + P::kTrade) + (half * 64 + row_in) * 36;
#pragma unroll 1
                for (int i = i0; i < i1; ++i) {
                    uint32_t x[32];
                    __syncwarp();
                    if (kNarrow) {
                        tmem_ld32(to + 32 * (i - i0), x);
                        if (s == 1)
#pragma unroll
                            for (int c = 0; c < 32; c += 4)
                                *reinterpret_cast<float4 *>(trade + c) =
                                    two ? make_float4(w1 * __uint_as_float(x[c]), w1 * __uint_as_float(x[c + 1]), w1 * __uint_as_float(x[c + 2]),
                                                      w1 * __uint_as_float(x[c + 3]))
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
                        named_sync(2, kSoftThreads);
                        if (s == 0)
#pragma unroll
                            for (int c = 0; c < 32; c += 4) {
                                const float4 y = *reinterpret_cast<const float4 *>(trade + c);
                                x[c] = __float_as_uint(fmaf(w0, __uint_as_float(x[c]), y.x));
                                x[c + 1] = __float_as_uint(fmaf(w0, __uint_as_float(x[c + 1]), y.y));
                                x[c + 2] = __float_as_uint(fmaf(w0, __uint_as_float(x[c + 2]), y.z));
                                x[c + 3] = __float_as_uint(fmaf(w0, __uint_as_float(x[c + 3]), y.w));
                            }
                        named_sync(2, kSoftThreads);
                        if (s == 1)
                            continue;
                    } else {
                        tmem_ld32(o0 + 32 * i, x);
                        if (NT == 1 && two) {
                            uint32_t y[32];
                            tmem_ld32(o1 + 32 * i, y);
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                x[c] = __float_as_uint(w0 * __uint_as_float(x[c]) + w1 * __uint_as_float(y[c]));
                        } else {
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                x[c] = __float_as_uint(w0 * __uint_as_float(x[c]));
                        }
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
                        // by four columns, so that the lanes' stores lie side by side
                        float4 *out = reinterpret_cast<float4 *>(slot) + (size_t)(8 * i) * kRows + r;
#pragma unroll
                        for (int v = 0; v < 8; ++v)
                            out[v * kRows] = make_float4(__uint_as_float(x[column_of<kType>(4 * v)]), __uint_as_float(x[column_of<kType>(4 * v + 1)]),
                                                 __uint_as_float(x[column_of<kType>(4 * v + 2)]), __uint_as_float(x[column_of<kType>(4 * v + 3)]));
                    }
                }
                if (wild && valid && !(kNarrow && s == 1)) {  // infinities and NaNs of values that the row sees: they are the element's sum
                    for (int d = 32 * i0; d < 32 * i1; ++d) {
                        const float v = attn_wild_values(p, it_b, it_head, t, d, seq.ctx, from, upto);
                        if (finite_f32(v))
                            continue;
                        if (whole)
                            p.out[at * D + d] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
                        else
                            slot[((size_t)(d >> 2) * kRows + r) * 4 + (d & 3)] = v;
                    }
                }
                if (valid && (NT == 2 || (s == 0 && half == 0))) {
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
            key_tile += n;
        }
    } else if (warp < kMmaWarp || warp > kLoadWarp) {
        // ---------------------------------------------------------- conversion
        const int ct = warp < kMmaWarp ? tid - kSoftThreads : tid - kSoftThreads - 64;
        int index = 0;                    // tile slots used so far
        int raw = 0;                      // code slots used so far
        uint32_t go_phase = 0;            // bit s: of go[s]
        uint32_t q_phase = 1;
        for (int item = 0; it.next(p, kKeys); ++item) {  // (as above: no wait ends it)
            const SeqLen seq = it.seq;
            const int it_b = it.b, it_head = it.head, it_t0 = it.t0, it_t1 = it.t1, it_block = it.block;
            const int n = it_t1 - it_t0, row0 = it_block * kRows;
            if (ct == 0)
                *reinterpret_cast<volatile int *>(&sh.wild[item & 3]) = 0;
            named_sync(1, kConvThreads);
            // the query
            wait_or_dead(&sh.q_empty, q_phase, sh, status);
            q_phase ^= 1;
            {
                const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
                // a thread keeps its 16-byte piece of a row and goes down the rows, eight loads in flight
                constexpr int kStep = kConvThreads / kPieces;
                const int x = ct % kPieces;
                int row = row0 + ct / kPieces, t = row / p.G, g = row - t * p.G;
                const uint16_t *q = p.q + (size_t)it_b * p.T * p.q_stride + (size_t)it_head * p.G * D + x * 8;
                constexpr int kQRows = kNarrow ? 64 : kRows;
                for (int r0 = ct / kPieces; r0 < kQRows; r0 += 8 * kStep) {
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
                        if (r >= kQRows)  // the same for the lanes of a row
                            break;
                        uint4 w = make_uint4(v[i].x ^ flip, v[i].y ^ flip, v[i].z ^ flip, v[i].w ^ flip);
                        if (kRawKeys) {
                            uint2 hi, lo;
                            const float scale = split_e4m3(w, hi, lo);
                            const uint32_t at = base + P::kQ + r * 128 + ((((uint32_t)x >> 1) ^ (r & 7)) << 4) + (x & 1) * 8;
#pragma unroll
                            for (int copy = 0; copy < 2; ++copy) {
                                asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(at + copy * 64 * 128), "r"(hi.x), "r"(hi.y) : "memory");
                                asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(at + (kKeys + copy * 64) * 128), "r"(lo.x), "r"(lo.y) : "memory");
                            }
                            if (x == 0)
                                sh.q_scale[item & 1][r] = scale;
                            continue;
                        }
                        if (kType == kKvInt4)  // the converted keys' columns are permuted
                            w = make_uint4(__byte_perm(w.x, w.z, 0x5410), __byte_perm(w.x, w.z, 0x7632), __byte_perm(w.y, w.w, 0x5410),
                                           __byte_perm(w.y, w.w, 0x7632));
                        if (kType == kKvFp8)
                            w = make_uint4(__byte_perm(w.x, w.y, 0x5410), __byte_perm(w.x, w.y, 0x7632), __byte_perm(w.z, w.w, 0x5410),
                                           __byte_perm(w.z, w.w, 0x7632));
                        sts128(tile_piece(base + P::kQ + (r >> 7) * P::kTileBytes, r & 127, x), w);
                        if (kNarrow)  // and the copy
                            sts128(tile_piece(base + P::kQ, r + 64, x), w);
                    }
                }
                fence_async_shared();
                named_sync(1, kConvThreads);
                if (ct == 0)
                    mbar_arrive(&sh.q_full);
            }
            // tiles
#pragma unroll 1
            for (int e = 0; e < 2 * n; ++e) {  // keys and values in turn; the keys only where they are converted
                const int j = e >> 1, tile_no = index + j;
                const bool value = e & 1;
                if (!value && (kType == kKvBf16 || kRawKeys))
                    continue;
                const int slot = value ? tile_no % P::kSlots : tile_no % P::kKeySlots;
                const int use = value ? tile_no / P::kSlots : tile_no / P::kKeySlots;
                const int pos = (it_t0 + j) * kKeys;
                const bool tail = value && pos + kKeys > seq.ctx;
                if (kType == kKvBf16) {
                    if (!tail)
                        continue;  // the copy warp's
                    wait_or_dead(&sh.go[slot], (go_phase >> slot) & 1, sh, status);
                    go_phase ^= 1u << slot;
                } else {
                    wait_or_dead(value ? &sh.empty[slot] : &sh.k_empty[slot], (use & 1) ^ 1, sh, status);
                }
                const uint32_t tile = base + (value ? slot * P::kTileBytes : P::kKeyRing + slot * P::kKeyBytes);
                const int rs = kCoded ? raw % P::kRaw : 0;
                bool wild = false;
                if (kType == kKvFp8) {
                    wait_or_dead(&sh.raw_full[rs], (raw / P::kRaw) & 1, sh, status);
                    const uint32_t codes = base + P::kRing + rs * P::kRawBytes;
                    const uint32_t valid = *reinterpret_cast<volatile uint32_t *>(&sh.raw_valid[rs]);
                    // A thread keeps its 16 columns and goes down the rows by kStep, a multiple of 8: every address is
                    // its first one plus a constant.
                    constexpr int kUnits = D / 16, kStep = kConvThreads / kUnits, kPasses = (kKeys + kStep - 1) / kStep;
                    static_assert(kStep % 8 == 0, "the permutation of a row's pieces");
                    const uint8_t *src = smem_raw + (codes - smem_addr(smem_raw));
                    {
                        const int r0 = ct / kUnits, x = ct % kUnits;
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
                        const bool plain = !tail && valid == 0xFFu && most <= 134;
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
                                if (tail && pos + r >= seq.ctx) {
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
                } else if (kType == kKvInt4) {
                    wait_or_dead(&sh.raw_full[rs], (raw / P::kRaw) & 1, sh, status);
                    const uint32_t valid = *reinterpret_cast<volatile uint32_t *>(&sh.raw_valid[rs]);
                    const uint8_t *src = smem_raw + (base + P::kRing + rs * P::kRawBytes - smem_addr(smem_raw));
                    // A thread has 32 columns of a row, which lie in one group: four pieces, each from one word.
                    constexpr int kUnits = D / 32, kStep = kConvThreads / kUnits;
                    static_assert(kStep % 8 == 0, "the permutation of a row's pieces");
                    const int r0 = ct / kUnits, x = ct % kUnits, groups = D / p.c.group, grp = x * 32 / p.c.group;
                    const bool swap = x >> 1;  // half of the lanes store their pieces in another order: no bank twice
#pragma unroll 1
                    for (int r = r0; r < kKeys; r += kStep) {
                        uint4 in = *reinterpret_cast<const uint4 *>(src + r * P::kRawRow + x * 16);
                        const uint16_t *scales = reinterpret_cast<const uint16_t *>(src + P::kRawCodes) + r * groups + grp;
                        uint32_t sb = scales[0], bb = scales[P::kRawScales / 2];
                        bool use_it = (valid >> (r >> 4)) & 1u;
                        if (tail && pos + r >= seq.ctx) {
                            if (pos + r >= seq.keys) {
                                use_it = false;
                            } else if ((sb & 0x7C00u) == 0x7C00u || (bb & 0x7C00u) == 0x7C00u) {
                                wild |= use_it;
                                use_it = false;
                            }
                        }
                        if (!use_it)
                            sb = bb = 0;
                        const __half hs = __ushort_as_half((unsigned short)sb), hb = __ushort_as_half((unsigned short)bb);
                        const float fs = __half2float(hs), fb = fmaf(-16.f, fs, __half2float(hb));
                        const __half2 s2 = __half2half2(hs), b2 = __half2half2(hb);
                        const uint32_t words[4] = {swap ? in.z : in.x, swap ? in.w : in.y, swap ? in.x : in.z, swap ? in.y : in.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t at = tile_piece(tile, r, 4 * x + (j ^ (swap ? 2 : 0))), w = words[j];
                            if (value) {
                                sts128(at, make_uint4(int4_f16x2<false>(w, s2, b2), int4_f16x2<true>(w, s2, b2), int4_f16x2<false>(w >> 8, s2, b2),
                                                      int4_f16x2<true>(w >> 8, s2, b2)));
                            } else {
                                const uint32_t q[4] = {int4_bf16x2<0>(w), int4_bf16x2<1>(w), int4_bf16x2<2>(w), int4_bf16x2<3>(w)};
                                uint32_t hi[4], lo[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const float a = fmaf(bf16_lo(q[i]), fs, fb), z = fmaf(bf16_hi(q[i]), fs, fb);
                                    hi[i] = pack2_bf16(a, z);
                                    lo[i] = pack2_bf16(a - bf16_lo(hi[i]), z - bf16_hi(hi[i]));
                                }
                                sts128(at, make_uint4(hi[0], hi[1], hi[2], hi[3]));
                                sts128(at + P::kTileBytes, make_uint4(lo[0], lo[1], lo[2], lo[3]));
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
                    mbar_arrive(value ? &sh.full[slot] : &sh.k_full[slot]);
                    if (kCoded)
                        mbar_arrive(&sh.raw_empty[rs]);
                }
                ++raw;
            }
            index += n;
        }
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------- products
        constexpr uint32_t kIdescS = kRawKeys ? umma_idesc_e4m3(128, kKeys) : umma_idesc_bf16(128, kKeys), kIdescO = (kHalf ? umma_idesc_f16(128, D) : umma_idesc_bf16(128, D)) | kIdescBMnMajor;
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
                const int s = u & 1, j = NT == 2 ? u >> 1 : u, e = index + j;
                const int slot = e % P::kKeySlots;
                if (!wait_or_dead(&sh.k_full[slot], (e / P::kKeySlots) & 1, sh, status))
                    return false;
                tc_fence_after();
                const uint32_t q = desc_lo(base + P::kQ + (NT == 2 ? s * P::kTileBytes : 0), 16);
                const uint32_t k = desc_lo(base + P::kKeyRing + slot * P::kKeyBytes, 16);
                if (elect_one()) {
                    if (kRawKeys) {  // the query's two parts, each a tile of 128 rows of 128 bytes
#pragma unroll
                        for (int i = 0; i < 2 * (D / 32); ++i)
                            umma_e4m3_lo(tmem + s * kKeys, q + ((i >> 2) * kKeys * 128 + (i & 3) * 32) / 16, k + (i & 3) * 2, kIdescS, i > 0);
                    } else {
#pragma unroll
                        for (int part = 0; part < P::kKeyBytes / P::kTileBytes; ++part)  // INT4: two parts of a key
#pragma unroll
                            for (int i = 0; i < D / 16; ++i) {
                                const uint32_t at = ((i >> 2) * P::kHalf + (i & 3) * 32) >> 4;
                                umma_bf16_lo(tmem + s * kKeys, q + at, k + part * (P::kTileBytes >> 4) + at, kIdescS, part + i > 0);
                            }
                    }
                    umma_commit(&sh.s_ready[s]);
                    if (NT == 1 || s == 1)
                        umma_commit(&sh.k_empty[slot]);
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
                const int s = u & 1, j = NT == 2 ? u >> 1 : u, e = index + j;
                const int slot = e % P::kSlots;
                ok = wait_or_dead(&sh.full[slot], (e / P::kSlots) & 1, sh, status);
                if (!ok)
                    break;
                const uint32_t v = desc_lo(base + slot * P::kTileBytes, P::kHalf);
                const auto weighted = [&](int i) {
                    umma_bf16_ts_lo(tmem + 256 + s * 128, tmem + s * kKeys + (kNarrow && i >= 4 ? 64 + (i - 4) * 8 : i * 8), v + i * (2048 >> 4), kIdescO,
                                    i > 0 || u >= 2);
                };
                constexpr int kEarly = kNarrow ? 0 : 4;  // steps of the first 64 keys
                if (!kNarrow) {
                    ok = wait_or_dead(&sh.p_half[s], p_phase[s], sh, status);
                    if (!ok)
                        break;
                    tc_fence_after();
                    if (elect_one())
#pragma unroll
                        for (int i = 0; i < kEarly; ++i)
                            weighted(i);
                    __syncwarp();
                }
                ok = wait_or_dead(&sh.p_ready[s], p_phase[s], sh, status);
                if (!ok)
                    break;
                p_phase[s] ^= 1;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int i = kEarly; i < kKeys / 16; ++i)
                        weighted(i);
                    if (NT == 1 || s == 1)
                        umma_commit(&sh.empty[slot]);
                    if (u + 2 >= units)
                        umma_commit(&sh.o_done[s]);
                }
                __syncwarp();
                if (u + 2 < units)
                    ok = scores(u + 2);
            }
            index += n;
        }
    } else {
        // ---------------------------------------------------------- copies
        const int per_page = min(kKeys, 1 << p.c.page_shift);  // keys of a chunk that lies in one page
        const int chunks = kKeys / per_page;                   // at most 8
        const long total_rows = (p.c.n_pages * p.c.heads) << p.c.page_shift;
        int index = 0;
        bool ok = true;
        if ((kType == kKvBf16 || kRawKeys) && lane == 0)
            tma_prefetch_map(&map_k);
        if (kType == kKvBf16 && lane == 1)
            tma_prefetch_map(&map_v);
        // One pass a tile, keys and values together: the warp's own instructions were what bound a stream of
        // tiles (1400 cycles for each of the two, of some 130 instructions in turn). Lane 8 i + c copies chunk c:
        //   bf16: the two 64-column halves of the keys (i = 0, 1) and of the values (2, 3);
        //   FP8, INT4: the keys' codes (0) and scales (1; INT4: and biases), the values' codes (2) and scales (3).
        const int part = lane >> 3, c = lane & 7;
        const bool value = part >= 2, chunk = c < chunks;
        uint8_t *const tiles = smem_raw + (base - smem_addr(smem_raw));
        while (ok && it.next(p, kKeys)) {
            const SeqLen seq = it.seq;
            const int it_b = it.b, it_head = it.head, it_t0 = it.t0, it_t1 = it.t1;
            const int n = it_t1 - it_t0;
            // pages: lane 8 i + c holds chunk c of tile 4 g + i, for the group g at hand and the next
            const auto pages_of = [&](int g) {
                const int j = 4 * g + part;
                const long pos = (long)(it_t0 + j) * kKeys + c * per_page;
                return j < n && chunk && pos < seq.keys ? (int)kv_page(p.c, it_b, pos) : -1;
            };
            int now = pages_of(0), after = pages_of(1);
#pragma unroll 1
            for (int j = 0; ok && j < n; ++j) {
                if (j > 0 && (j & 3) == 0) {
                    now = after;
                    after = pages_of((j >> 2) + 1);
                }
                const int page = __shfl_sync(0xFFFFFFFFu, now, (j & 3) * 8 + c);
                const int pos = (it_t0 + j) * kKeys, mine = pos + c * per_page;
                const bool there = chunk && page >= 0, tail = pos + kKeys > seq.ctx;
                if (chunk && page < 0 && mine < seq.keys && status)
                    atomicExch(status, kStatusBadArg);
                const long row = there ? (long)kv_row(p.c, page, it_head, mine) : total_rows;
                const int tile = index + j, ks = tile % P::kKeySlots;
                if (kType == kKvBf16 || kRawKeys) {
                    ok = wait_or_dead(&sh.k_empty[ks], ((tile / P::kKeySlots) & 1) ^ 1, sh, status);
                    if (!ok)
                        break;
                }
                // the keys first: their product runs ahead of the values'
                uint8_t *const key_tile = tiles + P::kKeyRing + ks * P::kKeyBytes;
                if (kType == kKvBf16) {
                    const int vs = tile % P::kSlots, half = part & 1;
                    if (lane == 0)
                        mbar_arrive_expect_tx(&sh.k_full[ks], P::kTileBytes);
                    __syncwarp();
                    // a chunk without a page is read past the last row: zeros
                    if (chunk && !value && half < D / 64)
                        tma_load_2d(key_tile + half * P::kHalf + c * per_page * 128, &map_k, half * 64, (int)row, &sh.k_full[ks]);
                    __syncwarp();
                    ok = wait_or_dead(&sh.empty[vs], ((tile / P::kSlots) & 1) ^ 1, sh, status);
                    if (!ok)
                        break;
                    if (lane == 0) {
                        if (tail)  // the conversion warps' to fill
                            mbar_arrive(&sh.go[vs]);
                        else
                            mbar_arrive_expect_tx(&sh.full[vs], P::kTileBytes);
                    }
                    __syncwarp();
                    if (chunk && value && half < D / 64 && !tail)
                        tma_load_2d(tiles + vs * P::kTileBytes + half * P::kHalf + c * per_page * 128, &map_v, half * 64, (int)row, &sh.full[vs]);
                } else {
                    const unsigned have = __ballot_sync(0xFFFFFFFFu, there && part == 0);
                    const int bytes = __popc(have) * per_page;
                    // which chunks of 16 keys lie in a page: bits of `have`, each per_page / 16 times
                    uint32_t bits = 0xFFu;
                    if (have != (1u << chunks) - 1) {
                        bits = 0;
                        for (int i = 0; i < 8; ++i)
                            bits |= ((have >> (i * 16 / per_page)) & 1u) << i;
                    }
                    // a ring slot of codes and scales for the keys' or the values' lanes
                    const auto codes_to = [&](int raw, bool values) {
                        const int rs = raw % P::kRaw;
                        if (!wait_or_dead(&sh.raw_empty[rs], ((raw / P::kRaw) & 1) ^ 1, sh, status))
                            return false;
                        const int groups = kType == kKvInt4 ? D / p.c.group : 0, of_row = kType == kKvFp8 ? 1 : 2 * groups;  // a row's scales, bytes
                        if (lane == 0) {
                            *reinterpret_cast<volatile uint32_t *>(&sh.raw_valid[rs]) = bits;
                            mbar_arrive_expect_tx(&sh.raw_full[rs], bytes * (P::kRawRow + (kType == kKvInt4 ? 2 : 1) * of_row));
                        }
                        __syncwarp();
                        if (value == values && there) {
                            uint8_t *codes = tiles + P::kRing + rs * P::kRawBytes;
                            const uint8_t *from = values ? p.c.v : p.c.k, *scales = values ? p.c.vs : p.c.ks, *biases = values ? p.c.vb : p.c.kb;
                            const bool code = !(part & 1);
                            uint8_t *to = code ? codes + c * per_page * P::kRawRow : codes + P::kRawCodes + c * per_page * of_row;
                            bulk_copy_g2s(to, code ? from + row * P::kRawRow : scales + row * of_row, per_page * (code ? P::kRawRow : of_row),
                                          &sh.raw_full[rs]);
                            if (kType == kKvInt4 && !code)
                                bulk_copy_g2s(to + P::kRawScales, biases + row * of_row, per_page * of_row, &sh.raw_full[rs]);
                        }
                        __syncwarp();
                        return true;
                    };
                    if (kRawKeys) {
                        uint8_t *scales = sh.key_scale[tile % kScaleSlots];
                        if (part == 1 && chunk && !there)  // codes 0 with a scale of 1
                            for (int i = 0; i < per_page; i += 4)
                                *reinterpret_cast<volatile uint32_t *>(scales + c * per_page + i) = 0x7F7F7F7Fu;
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive_expect_tx(&sh.k_full[ks], P::kKeyBytes + bytes);
                        __syncwarp();
                        if (part == 0 && chunk)  // without a page: past the last row, zeros
                            tma_load_2d(key_tile + c * per_page * D, &map_k, 0, (int)row, &sh.k_full[ks]);
                        if (part == 1 && there)
                            bulk_copy_g2s(scales + c * per_page, p.c.ks + row, per_page, &sh.k_full[ks]);
                        __syncwarp();
                        ok = codes_to(tile, true);
                    } else {
                        ok = codes_to(2 * tile, false) && codes_to(2 * tile + 1, true);
                    }
                    if (!ok)
                        break;
                }
                __syncwarp();
            }
            index += n;
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

template <int kType, int D, int NT, bool kNarrow>
cudaError_t launch_wide(AttnParams p, const LaunchCfg &cfg, cudaStream_t stream)
{
    using Pl = Plan<kType, D, NT, kNarrow>;
    auto *kernel = hc_attn_wide_kernel<kType, D, NT, kNarrow>;
    static_assert(Pl::kTotal + sizeof(Shared<NT, Pl::kRawKeys, kNarrow>) <= 227 * 1024, "shared memory");
    int per_sm = 1;
    cudaError_t e = attn_ready(reinterpret_cast<const void *>(kernel), kThreads, Pl::kTotal, &per_sm);
    if (e != cudaSuccess)
        return e;
    p.row_blocks = (p.rows + 128 * NT - 1) / (128 * NT);
    CUtensorMap map_k{}, map_v{};
    if (kType == kKvBf16) {
        const uint64_t rows = (uint64_t)p.c.n_pages * p.c.heads << p.c.page_shift;
        const uint32_t box = (uint32_t)std::min(kKeys, 1 << p.c.page_shift);
        if (!tc_make_map_2d(&map_k, p.c.k, rows, D, 64, box) || !tc_make_map_2d(&map_v, p.c.v, rows, D, 64, box))
            return cudaErrorInvalidValue;
    }
    if (Pl::kRawKeys) {
        const uint64_t rows = (uint64_t)p.c.n_pages * p.c.heads << p.c.page_shift;
        if (!tc_make_map_2d_u8(&map_k, p.c.k, rows, D, 128, (uint32_t)std::min(kKeys, 1 << p.c.page_shift)))
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
    const int grid = std::min(per_sm * cfg.sm_count, kAttnWideGrid);
    lc.gridDim = dim3(grid);
    lc.dynamicSmemBytes = Pl::kTotal;
    e = cudaLaunchKernelEx(&lc, kernel, p, map_k, map_v, kLeastWide);
    if (e != cudaSuccess)
        return e;
    return launch_attn_join(p, 128 * NT, kKeys, grid, kLeastWide, true, stream);
}

template <int D>
cudaError_t launch_rows(const AttnParams &p, const LaunchCfg &cfg, cudaStream_t stream)
{
    const bool narrow = p.rows <= 64, two = attn_wide_rows(p.c, p.rows) == 256;
    switch (p.c.type) {
    case kKvBf16:
        return two ? launch_wide<kKvBf16, D, 2, false>(p, cfg, stream)
               : narrow ? launch_wide<kKvBf16, D, 1, true>(p, cfg, stream) : launch_wide<kKvBf16, D, 1, false>(p, cfg, stream);
    case kKvFp8:
        return two ? launch_wide<kKvFp8, D, 2, false>(p, cfg, stream)
               : narrow ? launch_wide<kKvFp8, D, 1, true>(p, cfg, stream) : launch_wide<kKvFp8, D, 1, false>(p, cfg, stream);
    default: return two ? launch_wide<kKvInt4, D, 2, false>(p, cfg, stream) : launch_wide<kKvInt4, D, 1, false>(p, cfg, stream);
    }
}

}  // namespace

// Rows of a block of the wide kernel, or 0 where it does not serve: rows of 64 or 128
// elements (two accumulators and two score tiles fill TMEM); fewer rows in the pool than a
// tensor map's coordinates reach; more than 32 rows, of INT4, whose keys are converted to
// two tiles, more than 64. us in blocks of 32 rows and here, over long contexts: 64 rows of
// FP8 x 64 95 and 65, of INT4 x 128 132 and 142, 96 of INT4 x 128 186 and 145, 100 of
// INT4 x 64 174 and 106. Over some hundred keys this kernel's longer start costs 2 us or so;
// the host does not know the lengths.
int attn_wide_rows(const KvView &c, long rows)
{
    if (rows <= (c.type == kKvInt4 ? 64 : 32) || c.D > 128)
        return 0;
    if (((c.n_pages * c.heads) << c.page_shift) >= (1l << 31) - kKeys)
        return 0;
    return rows <= 128 ? 128 : 256;
}

cudaError_t launch_attn_wide(const AttnParams &p, const LaunchCfg &cfg, cudaStream_t stream)
{
    return p.c.D == 64 ? launch_rows<64>(p, cfg, stream) : launch_rows<128>(p, cfg, stream);
}

}  // namespace tshc
