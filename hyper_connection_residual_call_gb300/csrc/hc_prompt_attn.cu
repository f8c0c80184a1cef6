// hc_prompt_attn.cu -- causal attention over packed prompts, on the tensor cores
// with TMEM accumulators (ts_hc_prompt_attention in include/ts_hc.h).
//
//   out_t = sum_{j <= t} p_tj v_j,  p_tj = exp(scale q_t . k_j - lse_t)
//
// for the tokens of one sequence: 4 D flops a pair of a row and a key that it sees,
// which for long prompts is all that counts. Two products of 128 rows with a tile of
// 128 keys, S = Q K^T and O += P V, run on the tensor cores; S and O are in TMEM,
// and a softmax thread owns one row: it takes its 128 scores to registers, needs no
// shuffles, and writes its weights P (bf16) over S, from where the second product
// takes them as its A operand. V tiles [key][d] are B operands in MN-major order, so
// that nothing is transposed.
//
// A block has 256 rows, two streams of 128: while one's softmax runs, the tensor cores
// work for the other. Rows are tokens times the query heads that share a key head, so
// that short prompts fill them and a tile of keys serves all of its heads. O is rescaled
// only where a row's maximum grows by more than 2^8 over the one it is kept relative to.
//
// Which keys a row sees is a matter of the last tiles of a block only. Their scores are
// masked; of their values, infinities and NaNs, whose products with weights of 0 would be
// NaNs, are taken out in shared memory and given back at the end to the rows that see them.
//
// Roles: warps 0-7 softmax, four a stream; warp 8 issues the products, warp 9 the copies,
// warp 10 looks through the last tiles' values, warp 11 finds the next block. Every wait is
// bounded; the first that runs out records TS_ERR_TIMEOUT and ends the others.
//
// Results are divided by the sum of the weights as they were before they were rounded. By the rounded ones' sum, as in the
// attention over the cache, they are off by 2.00e-3 and not by 2.02e-3 (1.61e-3 and not 1.81e-3 where a few keys have the
// weight; the results' rounding is 1.6e-3 of it); the second sum costs the long prompt 46 us, the batch 2.6, the short ones 0.6.
//
// One prompt of 16384 tokens, 32 heads of 128 over 8, takes 1.50 ms, 1.47 PFLOP/s, 0.86 of what a library product holds
// under the power cap (up to 1.59 in plain calls; heads of 64: 1.26): a block's pair of tiles takes some 3280 cycles, 2048 of them products, the rest what the
// exponentials and the products of one stream wait for the other's. Eight prompts of 256 to 2048 tokens take 125 us,
// of which 79 are tiles: the others are the blocks' first tiles, their last products (700 cycles) and the results' way
// out (3700 cycles, 2000 of them the stores, a row a lane). 48 prompts of up to 200 tokens, 16 heads of 64 over 2: 18.9 us.
// Before the last tiles' keys were masked by 32, and those that none of a warp's rows sees left out, it was 1.54 ms and 126
// us, and to that compare: two threads a row, 16 softmax warps, 1.60 and 131; two places for the queries, one less for
// the rest, 1.57 and 125.
#include <algorithm>

#include "hc_attn.cuh"
#include "hc_prompt.h"
#include "hc_prompt_plan.h"
#include "hc_tc.h"
#include "umma.cuh"

namespace tshc {

namespace {

constexpr unsigned kStatusInvalidArg = 1u;   // TS_ERR_INVALID_ARG of ts_hc.h
constexpr int kKeys = 128;                    // of a tile
constexpr int kSoftThreads = 256, kThreads = kSoftThreads + 128;
constexpr int kMmaWarp = 8, kLoadWarp = 9, kCleanWarp = 10;  // and the planning one
constexpr int kSoftRegs = 208, kOtherRegs = 80;  // 256 * 208 + 128 * 80 = 63488 <= 384 * 168, what the launch has
constexpr float kGrow = 8.f;                  // log2: how far a row's maximum may grow over its reference
constexpr uint32_t kTmemCols = 512;           // S of two streams, O of two streams

template <int D>
struct Plan {
    static constexpr int kTile = kKeys * D * 2, kHalf = kKeys * 128;
    static constexpr int kQ = 2 * kTile;
    static constexpr int kSlots = D == 64 ? 8 : 5;               // tiles of keys and of values, in turn
    static constexpr int kTotal = kQ + kSlots * kTile + 1024;    // and alignment
};

struct Item {
    int start, len, token;  // the sequence's first row and length; the block's first token in it
    int head, g0;           // key head, and the first of its query heads
    int tiles0, tiles1;     // of the streams, 0: none
};

struct Shared {
    uint64_t full[8], empty[8], go[8];  // tiles; go: a tile of values that is to be looked through
    uint64_t q_full, q_empty;
    uint64_t s_ready[2], p_half[2], p_ready[2], o_done[2];
    uint64_t item_full[2], item_empty[2], taken;
    alignas(16) uint4 answer;
    Item item[2];
    int last[2];            // no item: the end
    int wild[4];            // by items in turn: a value was an infinity or a NaN
    uint32_t tmem;
    int dead;               // a wait ran out
    int before[65535 / kRound + 2];  // blocks before a round's sequences
};

__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, Shared &sh, unsigned *status)
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

// Blocks of a sequence; 0 for one that is out of range (recorded).
__device__ __forceinline__ int blocks_of(const PromptAttnParams &p, int s)
{
    if (s >= p.S)
        return 0;
    const int n = blocks_of_rows(p.starts[s], p.starts[s + 1], p.N, 2 * p.TB);
    if (n < 0 && p.status)
        atomicExch(p.status, kStatusInvalidArg);
    return max(n, 0);
}

// The planning warp's work: which block is the n-th. Blocks of up to 256 sequences are taken in turn, each
// sequence's last one, which has the most keys, first, so that the blocks at the end are short ones.
struct Rounds {
    int round, blocks[kRound / 32], most;  // the round at hand; the lane's sequences' blocks, and the most of any
    __device__ __forceinline__ void init(const PromptAttnParams &p, Shared &sh)
    {
        const int lane = threadIdx.x & 31;
        round = -1;
        int sum = 0;
        for (int r = 0; r * kRound < p.S; ++r) {
            if (lane == 0)
                sh.before[r] = sum;
            int mine = 0;
#pragma unroll
            for (int i = 0; i < kRound / 32; ++i)
                mine += blocks_of(p, r * kRound + lane * (kRound / 32) + i);
            sum = add_blocks(sum, __reduce_add_sync(0xFFFFFFFFu, mine));
        }
        if (lane == 0)
            sh.before[(p.S + kRound - 1) / kRound] = sum;
        __syncwarp();
    }
    __device__ __forceinline__ int upto(int k) const  // blocks in the first k turns
    {
        int mine = 0;
#pragma unroll
        for (int i = 0; i < kRound / 32; ++i)
            mine += min(blocks[i], k);
        return __reduce_add_sync(0xFFFFFFFFu, mine);
    }
    __device__ __forceinline__ bool find(const PromptAttnParams &p, long n, Shared &sh, Item &it)
    {
        const int lane = threadIdx.x & 31, sub = p.G / p.Gp, heads = p.kv_heads * sub, rounds = (p.S + kRound - 1) / kRound;
        const long block = n / heads;
        if (block >= sh.before[rounds])
            return false;
        int lo = 0, hi = rounds - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (sh.before[mid] <= block)
                lo = mid;
            else
                hi = mid - 1;
        }
        if (lo != round) {
            round = lo;
            most = 0;
#pragma unroll
            for (int i = 0; i < kRound / 32; ++i) {
                blocks[i] = blocks_of(p, round * kRound + lane * (kRound / 32) + i);
                most = max(most, blocks[i]);
            }
            most = __reduce_max_sync(0xFFFFFFFFu, most);
        }
        const int at = (int)(block - sh.before[round]);
        int turn = 0, above = most;  // upto(turn) <= at < upto(above)
        while (above - turn > 1) {
            const int mid = (turn + above) / 2;
            if (upto(mid) <= at)
                turn = mid;
            else
                above = mid;
        }
        int left = at - upto(turn), has = 0;
#pragma unroll
        for (int i = 0; i < kRound / 32; ++i)
            has += blocks[i] > turn;
        int pre = has;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xFFFFFFFFu, pre, o);
            pre += lane >= o ? x : 0;
        }
        pre -= has;
        const int owner = __ffs(__ballot_sync(0xFFFFFFFFu, left >= pre && left < pre + has)) - 1;
        left -= pre;
        int seq = 0, of = 0;
#pragma unroll
        for (int i = 0; i < kRound / 32; ++i)
            if (blocks[i] > turn && left-- == 0) {
                seq = round * kRound + lane * (kRound / 32) + i;
                of = blocks[i];
            }
        seq = __shfl_sync(0xFFFFFFFFu, seq, owner);
        of = __shfl_sync(0xFFFFFFFFu, of, owner);
        const int h = (int)(n - block * heads);
        it.start = p.starts[seq];
        it.len = p.starts[seq + 1] - it.start;
        it.token = (of - 1 - turn) * 2 * p.TB;
        it.head = h / sub;
        it.g0 = (h - it.head * sub) * p.Gp;
        it.tiles0 = (min(it.token + p.TB, it.len) - 1) / kKeys + 1;
        it.tiles1 = it.token + p.TB < it.len ? (min(it.token + 2 * p.TB, it.len) - 1) / kKeys + 1 : 0;
        return true;
    }
};

// A consumer's side of the items.
struct Items {
    uint32_t count = 0;
    __device__ __forceinline__ bool next(Item &it, Shared &sh, unsigned *status)
    {
        const int slot = count & 1;
        if (!wait(&sh.item_full[slot], (count >> 1) & 1, sh, status))
            return false;
        it = sh.item[slot];
        const bool end = sh.last[slot];
        __syncwarp();
        if ((threadIdx.x & 31) == 0)
            mbar_arrive(&sh.item_empty[slot]);
        ++count;
        return !end;
    }
};

// Bits 15 and 31: whether the halves are infinities or NaNs (exponents of ones carry into them).
__device__ __forceinline__ uint32_t odd_bits(uint32_t w) { return (w & 0x7F807F80u) + 0x00800080u; }

// 32 bytes, a whole sector: a lane has a row of its own. By one instruction where the results lie so; they need only lie on
// 16 bytes.
__device__ __forceinline__ void store32(uint16_t *to, const uint32_t *w, bool whole)
{
    if (whole) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                     ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
    } else {
        *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4 *>(to + 8) = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
hc_prompt_attn_kernel(const __grid_constant__ PromptAttnParams p, const __grid_constant__ CUtensorMap map_q,
                      const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v)
{
    using P = Plan<D>;
    constexpr int kSlots = P::kSlots;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Shared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t *const tiles = smem_raw + (base - smem_addr(smem_raw));
    unsigned *const status = p.status;
    if (tid == 0) {
        for (int i = 0; i < 8; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1);
            mbar_init(&sh.go[i], 1);
        }
        mbar_init(&sh.q_full, 1);
        mbar_init(&sh.q_empty, 1);
        mbar_init(&sh.taken, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh.s_ready[s], 1);
            mbar_init(&sh.p_half[s], kSoftThreads / 2);
            mbar_init(&sh.p_ready[s], kSoftThreads / 2);
            mbar_init(&sh.o_done[s], 1);
            mbar_init(&sh.item_full[s], 1);
            mbar_init(&sh.item_empty[s], kSoftThreads / 32 + 3);
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
    pdl_wait();
    pdl_launch_dependents();

    if (warp < kMmaWarp) {
        // ---------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        const int s = warp >> 2, row = tid & 127;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lane_base + s * kKeys, to = tmem + lane_base + 256 + s * 128;
        const float sc = p.scale_log2;
        const bool whole = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
        const int row_t = row / p.Gp, row_g = row - row_t * p.Gp;
        uint32_t s_phase = 0, o_phase = 0;
        Items items;
        Item it;
        for (int turn = 0; items.next(it, sh, status); ++turn) {
            const int n = s == 0 ? it.tiles0 : it.tiles1;
            if (n == 0)
                continue;
            const int first = it.token + s * p.TB, t = first + row_t;  // the stream's first token, the row's
            const bool valid = row_t < p.TB && t < it.len;
            float m = -INFINITY, l = 0.f;  // the reference (in units of log2) and the weights' sum
            // (A wait that ran out ends nothing here: the warps go on through the same barriers, on whatever lies
            // there, and every further wait returns at once.)
#pragma unroll 1
            for (int j = 0; j < n; ++j) {
                wait(&sh.s_ready[s], s_phase, sh, status);
                s_phase ^= 1;
                tc_fence_after();
                uint32_t x[4][32];
                tmem_ld32_async(ts, x[0]);
                tmem_ld32_async(ts + 32, x[1]);
                tmem_ld32_async(ts + 64, x[2]);
                tmem_ld32_async(ts + 96, x[3]);
                tmem_wait_ld32(x[0]);
                tmem_wait_ld32(x[1]);
                tmem_wait_ld32(x[2]);
                tmem_wait_ld32(x[3]);
                const bool cut = j * kKeys + kKeys - 1 > first;  // not every row sees all keys
                const int sees = t - j * kKeys;                  // the last that this one sees
                if (cut)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (!__all_sync(0xFFFFFFFFu, sees >= i * 32 + 31))
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (i * 32 + c > sees)
                                    x[i][c] = 0xFF800000u;
                float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int c = 0; c < 32; c += 2)
                        tops[i] = fmaxf(tops[i], fmaxf(__uint_as_float(x[i][c]), __uint_as_float(x[i][c + 1])));
                const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * sc;
                const bool grows = top > m + kGrow;  // also the first that is not -infinity
                if (__any_sync(0xFFFFFFFFu, grows)) {  // (for its own row's sake only: rows do not depend on one another)
                    const float to_m = grows ? top : m, by = ex2(m - (to_m == -INFINITY ? 0.f : to_m));
                    m = to_m;
                    l *= by;
                    if (j > 0) {  // before the first, the accumulator holds nothing
                        uint32_t z[16];
#pragma unroll 1
                        for (int i = 0; i < D / 16; ++i) {
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
                const uint64_t sc2 = f32x2(sc, sc), off2 = f32x2(off, off);
                uint64_t sums[2] = {0, 0};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t w[16];
                    if (cut && !__any_sync(0xFFFFFFFFu, sees >= i * 32)) {  // nobody sees these
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            w[c] = 0;
                    } else
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        float a, z;
                        f32x2_unpack(ffma2(f32x2(__uint_as_float(x[i][2 * c]), __uint_as_float(x[i][2 * c + 1])), sc2, off2), a, z);
                        a = ex2(a);
                        z = ex2(z);
                        sums[c & 1] = fadd2(sums[c & 1], f32x2(a, z));
                        w[c] = pack2_bf16(a, z);
                    }
                    tmem_st16_async(ts + 16 * i, w);
                    if (i == 1) {  // the product can begin with the first 64 keys (with 32: 1524 us for 1499, with 96: 1510)
                        tmem_wait_st();
                        tc_fence_before();
                        mbar_arrive(&sh.p_half[s]);
                    }
                }
                float a, z;
                f32x2_unpack(fadd2(sums[0], sums[1]), a, z);
                l += a + z;
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&sh.p_ready[s]);
            }
            wait(&sh.o_done[s], o_phase, sh, status);
            o_phase ^= 1;
            tc_fence_after();
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const size_t at = (size_t)(it.start + (valid ? t : 0)) * p.q_heads + it.head * p.G + it.g0 + row_g;
            const int wild = *reinterpret_cast<volatile int *>(&sh.wild[turn & 3]);
#pragma unroll 1
            for (int i = 0; i < D / 32; ++i) {
                uint32_t x[32], w[16];
                __syncwarp();
                tmem_ld32(to + 32 * i, x);
                if (!valid)
                    continue;
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    w[c] = pack2_bf16(__uint_as_float(x[2 * c]) * inv, __uint_as_float(x[2 * c + 1]) * inv);
                uint16_t *const out = p.out + at * D + 32 * i;
                store32(out, w, whole);
                store32(out + 16, w + 8, whole);
            }
            if (wild && valid) {  // infinities and NaNs among the values that were looked through and that the row sees
                const int from = it.token / kKeys * kKeys;
                for (int d = 0; d < D; ++d) {
                    float sum = 0.f;
                    for (int k = from; k <= t; ++k) {
                        const float v = __uint_as_float((uint32_t)p.v[(size_t)(it.start + k) * p.v_stride + it.head * D + d] << 16);
                        if (!(fabsf(v) < INFINITY))
                            sum += v;
                    }
                    if (!(fabsf(sum) < INFINITY)) {
                        uint16_t *o = p.out + at * D + d;
                        *o = (uint16_t)(__float_as_uint(sum + __uint_as_float((uint32_t)*o << 16)) >> 16);
                    }
                }
            }
            if (valid && p.lse)
                p.lse[at] = m == -INFINITY ? (l == 0.f ? -INFINITY : l) : (m + log2f(l)) * 0.6931471805599453f;
            tc_fence_before();
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kMmaWarp) {
            // ---------------------------------------------------------- products
            constexpr uint32_t kIdescS = umma_idesc_bf16(128, kKeys), kIdescO = umma_idesc_bf16(128, D) | kIdescBMnMajor;
            uint32_t tile = 0, q_phase = 0, p_phase[2] = {0, 0};  // tile: keys' and values', in turn
            Items items;
            Item it;
            bool ok = true;
            while (ok && items.next(it, sh, status)) {
                const int n = max(it.tiles0, it.tiles1);
                ok = wait(&sh.q_full, q_phase, sh, status);
                q_phase ^= 1;
                const auto scores = [&](int s, int j) {  // the last stream frees the slot
                    const uint32_t slot = (tile + 2 * j) % kSlots;
                    const uint32_t q = desc_lo(base + s * P::kTile, 16), k = desc_lo(base + P::kQ + slot * P::kTile, 16);
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            const uint32_t at = ((i >> 2) * P::kHalf + (i & 3) * 32) >> 4;
                            umma_bf16_lo(tmem + s * kKeys, q + at, k + at, kIdescS, i > 0);
                        }
                        umma_commit(&sh.s_ready[s]);
                        if (s == (j < it.tiles1)) {
                            umma_commit(&sh.empty[slot]);
                            if (j == n - 1)
                                umma_commit(&sh.q_empty);
                        }
                    }
                    __syncwarp();
                };
                const auto arrived = [&](int e) {
                    const uint32_t i = tile + e;
                    const bool there = wait(&sh.full[i % kSlots], (i / kSlots) & 1, sh, status);
                    tc_fence_after();
                    return there;
                };
                ok = ok && arrived(0);
                if (ok) {
                    if (it.tiles0 > 0)
                        scores(0, 0);
                    if (it.tiles1 > 0)
                        scores(1, 0);
                }
#pragma unroll 1
                for (int j = 0; ok && j < n; ++j) {
                    ok = arrived(2 * j + 1);
#pragma unroll 1
                    for (int s = 0; ok && s < 2; ++s) {
                        const int mine = s == 0 ? it.tiles0 : it.tiles1;
                        if (j >= mine)
                            continue;
                        const uint32_t slot = (tile + 2 * j + 1) % kSlots;
                        const uint32_t v = desc_lo(base + P::kQ + slot * P::kTile, P::kHalf);
                        const auto weighted = [&](int i) {
                            umma_bf16_ts_lo(tmem + 256 + s * 128, tmem + s * kKeys + i * 8, v + i * (2048 >> 4), kIdescO, i > 0 || j > 0);
                        };
                        ok = wait(&sh.p_half[s], p_phase[s], sh, status);
                        if (!ok)
                            break;
                        tc_fence_after();
                        if (elect_one())
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                weighted(i);
                        __syncwarp();
                        ok = wait(&sh.p_ready[s], p_phase[s], sh, status);
                        p_phase[s] ^= 1;
                        if (!ok)
                            break;
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int i = 4; i < 8; ++i)
                                weighted(i);
                            if (s == (j < it.tiles1))
                                umma_commit(&sh.empty[slot]);
                            if (j == mine - 1)
                                umma_commit(&sh.o_done[s]);
                        }
                        __syncwarp();
                        if (j + 1 < mine) {
                            ok = arrived(2 * j + 2);
                            if (ok)
                                scores(s, j + 1);
                        }
                    }
                }
                tile += 2 * n;
            }
        } else if (warp == kLoadWarp) {
            // ---------------------------------------------------------- copies
            uint32_t tile = 0, q_phase = 1;
            Items items;
            Item it;
            bool ok = true;
            if (lane == 0) {
                tma_prefetch_map(&map_q);
                tma_prefetch_map(&map_k);
                tma_prefetch_map(&map_v);
            }
            while (ok && items.next(it, sh, status)) {
                const int n = max(it.tiles0, it.tiles1);
                ok = wait(&sh.q_empty, q_phase, sh, status);
                q_phase ^= 1;
                if (ok && lane == 0) {
                    const int streams = it.tiles1 > 0 ? 2 : 1;
                    mbar_arrive_expect_tx(&sh.q_full, streams * (D / 64) * p.Gp * p.TB * 128);
                    for (int s = 0; s < streams; ++s)
                        for (int h = 0; h < D / 64; ++h)
                            tma_load_3d(tiles + s * P::kTile + h * P::kHalf, &map_q, h * 64, it.head * p.G + it.g0, it.start + it.token + s * p.TB,
                                        &sh.q_full);
                }
                __syncwarp();
#pragma unroll 1
                for (int e = 0; ok && e < 2 * n; ++e, ++tile) {
                    const uint32_t slot = tile % kSlots;
                    ok = wait(&sh.empty[slot], ((tile / kSlots) & 1) ^ 1, sh, status);
                    if (ok && lane == 0) {
                        const int j = e >> 1;
                        const bool value = e & 1;
                        uint64_t *bar = value && j * kKeys + kKeys - 1 > it.token ? &sh.go[slot] : &sh.full[slot];
                        mbar_arrive_expect_tx(bar, P::kTile);
                        for (int h = 0; h < D / 64; ++h)
                            tma_load_3d(tiles + P::kQ + slot * P::kTile + h * P::kHalf, value ? &map_v : &map_k, h * 64, it.head, it.start + j * kKeys, bar);
                    }
                    __syncwarp();
                }
            }
        } else if (warp == kCleanWarp) {
            // ---------------------------------------------------------- the last tiles' values
            uint32_t tile = 0, go_phase = 0;  // bit s: of go[s]
            Items items;
            Item it;
            for (int turn = 0; items.next(it, sh, status); ++turn) {
                const int n = max(it.tiles0, it.tiles1);
                // (the softmax warps are past their use of this word: to have the item before, they ended the ones before it)
                if (lane == 0)
                    *reinterpret_cast<volatile int *>(&sh.wild[turn & 3]) = 0;
                __syncwarp();
#pragma unroll 1
                for (int j = it.token / kKeys; j < n; ++j) {
                    if (j * kKeys + kKeys - 1 <= it.token)
                        continue;
                    const uint32_t slot = (tile + 2 * j + 1) % kSlots;
                    wait(&sh.go[slot], (go_phase >> slot) & 1, sh, status);
                    go_phase ^= 1u << slot;
                    uint4 *const at = reinterpret_cast<uint4 *>(tiles + P::kQ + slot * P::kTile);
                    bool found = false;
#pragma unroll 1
                    for (int i = lane; i < P::kTile / 16; i += 32 * 8) {
                        uint4 w[8];
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            w[c] = at[i + 32 * c];
                        uint32_t odd = 0;
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            odd |= odd_bits(w[c].x) | odd_bits(w[c].y) | odd_bits(w[c].z) | odd_bits(w[c].w);
                        if (!(odd & 0x80008000u))
                            continue;
                        found = true;
#pragma unroll 1
                        for (int c = 0; c < 8; ++c) {
                            uint32_t *u = reinterpret_cast<uint32_t *>(&at[i + 32 * c]);
                            for (int b = 0; b < 4; ++b) {
                                uint32_t y = u[b];
                                y = (y & 0x7F80u) == 0x7F80u ? y & 0xFFFF0000u : y;
                                y = (y & 0x7F800000u) == 0x7F800000u ? y & 0x0000FFFFu : y;
                                u[b] = y;
                            }
                        }
                    }
                    if (__any_sync(0xFFFFFFFFu, found)) {
                        if (lane == 0)
                            *reinterpret_cast<volatile int *>(&sh.wild[turn & 3]) = 1;
                        __syncwarp();
                        fence_async_shared();
                        __syncwarp();
                    }
                    if (lane == 0)
                        mbar_arrive(&sh.full[slot]);
                }
                tile += 2 * n;
            }
        } else {
            // ---------------------------------------------------------- the next block
            Rounds rounds;
            rounds.init(p, sh);
            // The grid has a CTA for each block; one that runs takes the place of one that has not begun, as long as
            // there are any, and keeps its TMEM, its barriers and its roles.
            int next = blockIdx.x;
            bool more = true;
            for (uint32_t count = 0; more; ++count) {
                const int slot = count & 1;
                Item it;
                if (count > 0) {
                    if (lane == 0) {
                        fence_async_shared();
                        mbar_arrive_expect_tx(&sh.taken, 16);
                        asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                                     ::"r"(smem_addr(&sh.answer)), "r"(smem_addr(&sh.taken)) : "memory");
                    }
                    __syncwarp();
                    more = wait(&sh.taken, (count - 1) & 1, sh, status);
                    uint32_t yes = 0, id = 0;
                    asm volatile("{\n\t.reg .pred p;\n\t.reg .b128 r;\n\tld.shared.b128 r, [%2];\n\t"
                                 "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\tselp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
                                 "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, _, _, _}, r;\n\t}"
                                 : "=r"(yes), "=r"(id) : "r"(smem_addr(&sh.answer)) : "memory");
                    __syncwarp();
                    more = more && yes;
                    next = (int)id;
                }
                more = more && rounds.find(p, next, sh, it);
                if (!wait(&sh.item_empty[slot], ((count >> 1) & 1) ^ 1, sh, status))
                    break;
                if (lane == 0) {
                    sh.item[slot] = it;
                    sh.last[slot] = !more;
                    mbar_arrive(&sh.item_full[slot]);
                }
                __syncwarp();
            }
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

template <int D>
cudaError_t launch(const PromptAttnParams &p, const uint16_t *q, long q_stride, const uint16_t *k, long k_stride, cudaStream_t stream)
{
    auto *kernel = hc_prompt_attn_kernel<D>;
    static_assert(Plan<D>::kTotal + sizeof(Shared) <= 227 * 1024, "shared memory");
    int per_sm = 1;
    const cudaError_t e = attn_ready(reinterpret_cast<const void *>(kernel), kThreads, Plan<D>::kTotal, &per_sm);
    if (e != cudaSuccess)
        return e;
    CUtensorMap map_q{}, map_k{}, map_v{};
    if (!tc_make_map_heads(&map_q, q, p.N, p.q_heads, D, q_stride, p.Gp, p.TB) || !tc_make_map_heads(&map_k, k, p.N, p.kv_heads, D, k_stride, 1, kKeys) ||
        !tc_make_map_heads(&map_v, p.v, p.N, p.kv_heads, D, p.v_stride, 1, kKeys))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t lc{};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = at;
    lc.numAttrs = 1;
    lc.stream = stream;
    lc.blockDim = dim3(kThreads);
    lc.gridDim = dim3((unsigned)prompt_attn_blocks(p.N, p.S, p.q_heads, p.kv_heads));
    lc.dynamicSmemBytes = Plan<D>::kTotal;
    return cudaLaunchKernelEx(&lc, kernel, p, map_q, map_k, map_v);
}

}  // namespace

// Query heads that share a block: all of a key head's where 32 or fewer, else the largest part of them that is.
int prompt_attn_heads(int G)
{
    for (int g = std::min(G, 32);; --g)
        if (G % g == 0)
            return g;
}

long prompt_attn_blocks(int N, int S, int q_heads, int kv_heads)
{
    const int Gp = prompt_attn_heads(q_heads / kv_heads);
    return ((long)N / (2 * (128 / Gp)) + S) * (q_heads / Gp);
}

cudaError_t launch_prompt_attention(PromptAttnParams p, const uint16_t *q, long q_stride, const uint16_t *k, long k_stride, int D,
                                    const LaunchCfg &, cudaStream_t stream)
{
    p.G = p.q_heads / p.kv_heads;
    p.Gp = prompt_attn_heads(p.G);
    p.TB = 128 / p.Gp;
    return D == 64 ? launch<64>(p, q, q_stride, k, k_stride, stream) : launch<128>(p, q, q_stride, k, k_stride, stream);
}

}  // namespace tshc
