// hc_logprobs.cu -- log probabilities of given tokens, the distribution's entropy
// and its best alternatives (ts_hc_logprobs in include/ts_hc.h).
//
//   log p_v = x_v - m - log Z,  Z = sum_v e^(x_v - m),  m = max_v x_v
//   entropy = -sum_v p_v log p_v = log Z - S / Z,  S = sum_v (x_v - m) e^(x_v - m)
//
// One pass over the logits: each thread keeps a running maximum and Z and S
// relative to it, in fp32, and they are joined in a fixed order. Where one token has nearly all of the
// probability, Z is 1 and little more, and log Z would have the rounding of 1 for its error (5e-7, of 4e-4 a
// thousandth): the sum without the thread that holds the maximum is kept beside Z, that thread's few elements are
// taken again without the maximum, and log Z is log1p of the two.
//
// The best alternatives come from the same pass. An element is a 64-bit key, its
// value in an order that unsigned comparison keeps above its index's complement, so
// that keys are distinct and the larger key is the larger value or, of equal ones,
// the lower index. The n-th largest of the maxima of 120 groups of a row's first
// 7680 elements is a threshold that n elements reach; what passes it goes to shared
// memory (some 20 elements of each further 7680), and is ranked at the row's end by
// counting, for each key, the larger ones. Rows in whose order too many pass it, a
// rising one say, are read a second time, with a threshold a chunk: at most n groups
// hold an element that reaches one, which bounds what is kept for any logits.
//
// 4099 rows of 65537 bf16, eight tokens each, take 111 us for 0.54 GB, 0.72 of the measured copy rate; 2048 rows of
// 128001 fp32 with the twenty best 212 us for 1.05 GB, 0.73, without them 152; 4096 rows of 65537 bf16 with the twenty best 237,
// 0.33: what a row's alternatives cost does not depend on its length. All issue 2.3 to 2.7 of 4 instructions a cycle from two
// blocks a SM; a block that ranks a row leaves the SM to the other. With alternatives the kernels spill 24 to 48 bytes in their 64
// registers, a third block's would not fit. One row of 32768: 7.9 us, a launch, 16 KB a CTA, a ranking and a join
// through the cluster. (Loads to registers, without copies ahead: 218 and 355 us. Without keeping the largest term apart: 106, 210,
// 148, 234 and 7.5.)
#include <algorithm>
#include <type_traits>

#include "hc_prompt.h"
#include "hc_attn.cuh"
#include "umma.cuh"

namespace tshc {

namespace {

constexpr unsigned kStatusInvalidArg = 1u;  // TS_ERR_INVALID_ARG of ts_hc.h
constexpr int kThreads = 480, kWarps = kThreads / 32;  // that take the elements; one more warp asks for copies
constexpr int kBlock = kThreads + 32;
constexpr int kHold = 16;                    // elements of a chunk that a thread holds
constexpr int kGroups = kThreads / 4;        // of four threads each
constexpr int kMaxTop = 32;
constexpr int kKeep = 4096;                  // keys kept; a chunk's threshold leaves at most kMaxTop * 4 * kHold of it
constexpr int kRank = kThreads / 4;          // keys that are ranked without a threshold first
constexpr int kEach = (kKeep + kThreads - 1) / kThreads;  // kept keys of a thread
constexpr int kFew = 1184;                   // keys that a compaction leaves, at most kMaxTop * 4 * kEach
static_assert(kGroups % 8 == 0, "quarters in pairs");
static_assert(kMaxTop * 4 * kHold <= kKeep / 2, "a chunk's keys");
static_assert(kMaxTop * 4 * kEach <= kFew, "what a compaction leaves");
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLeast = -200.f;           // of d: 2^d is 0 from -127 on, and d 2^d no NaN
constexpr float kNearlyOne = 1.25f;        // from here on log Z is right to 6 times what the sum is
constexpr float kNaN = __builtin_nanf("");

__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// mbar_wait_bounded, for warps that have nothing else to do: each attempt may take a microsecond of the
// hardware's own waiting, so that the others have the issue slots. One wait that runs out is all of `limit`: the next ones
// end after an attempt.
__device__ __forceinline__ bool wait_bounded(uint64_t *bar, uint32_t parity, uint32_t &limit)
{
    const uint64_t t0 = global_timer_ns();
    for (;;) {
        uint32_t done;
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(done) : "r"(smem_addr(bar)), "r"(parity), "r"(1000u) : "memory");
        if (done)
            return true;
        if (global_timer_ns() - t0 > limit) {
            limit = 0;
            return false;
        }
    }
}

// A value's and index's key, and back.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t i)
{
    const uint32_t u = __float_as_uint(x + 0.f);  // -0 is 0
    return (uint64_t)(u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u)) << 32 | (0xFFFFFFFFu - i);
}

__device__ __forceinline__ float key_value(uint64_t k)
{
    const uint32_t u = (uint32_t)(k >> 32);
    return __uint_as_float((u & 0x80000000u) ? u ^ 0x80000000u : ~u);
}

__device__ __forceinline__ uint32_t key_index(uint64_t k) { return 0xFFFFFFFFu - (uint32_t)k; }

// A distribution's part: its largest logit m, Z = sum 2^d and S = sum d 2^d over d = (x - m) log2 e, and Z without the
// thread that has m (the first of several), `who`: these where Z is less than kNearlyOne.
struct Part {
    float m, z, s, rest;
    int who;
};
__device__ __forceinline__ Part no_part() { return Part{-INFINITY, 0.f, 0.f, 0.f, 0}; }

// The parts of a warp's lanes.
__device__ __forceinline__ Part join_warp(Part a)
{
    const uint32_t u = __float_as_uint(a.m);
    const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u));
    const float m = __uint_as_float((most & 0x80000000u) ? most ^ 0x80000000u : ~most);
    const float d = max_nan((a.m - (m == -INFINITY ? 0.f : m)) * kLog2e, kLeast), f = ex2(d);
    float z = a.z * f, s = f * fmaf(d, a.z, a.s);
    const float mine = z;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
        s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    }
    if (!(z < kNearlyOne))   // nor is the row's then, if m is its maximum
        return Part{m, z, s, 0.f, 0};
    const int first = __ffs(__ballot_sync(0xFFFFFFFFu, a.m == m)) - 1;
    float rest = (threadIdx.x & 31) == first ? a.rest : mine;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        rest += __shfl_xor_sync(0xFFFFFFFFu, rest, o);
    return Part{m, z, s, rest, __shfl_sync(0xFFFFFFFFu, a.who, first)};
}

struct Shared {
    uint64_t keep[kKeep];
    uint64_t few[kFew];
    alignas(16) uint64_t group[kGroups];
    uint64_t top[kMaxTop];   // this block's, best first; a block of a cluster reads the others'
    uint64_t all[8 * kMaxTop];
    uint64_t threshold[2];
    Part part[2][kWarps];    // by rows in turn
    Part whole;
    uint64_t full[4], empty[4];
    int kept, left, dead;
};

// A barrier of the threads that take the elements.
__device__ __forceinline__ void sync() { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); }

// The n-th largest of the groups' largest keys (0 if fewer than n groups have one). Threads may still be reading it in
// `word` when others go on, up to the next barrier: the next call before one takes the other word.
__device__ __forceinline__ uint64_t threshold_of(uint64_t best, int n, Shared &sh, int word = 0)
{
    best = max(best, __shfl_xor_sync(0xFFFFFFFFu, best, 1));
    best = max(best, __shfl_xor_sync(0xFFFFFFFFu, best, 2));
    const int tid = threadIdx.x;
    if ((tid & 3) == 0)
        sh.group[tid >> 2] = best;
    if (tid == 0)
        sh.threshold[word] = 0;
    sync();
    // a group's four threads have a quarter of the others each
    constexpr int kQuarter = kGroups / 4;
    int larger = 0;
#pragma unroll 5
    for (int i = 0; i < kQuarter; i += 2) {
        const ulonglong2 two = *reinterpret_cast<const ulonglong2 *>(&sh.group[(tid & 3) * kQuarter + i]);
        larger += (two.x > best) + (two.y > best);
    }
    larger += __shfl_xor_sync(0xFFFFFFFFu, larger, 1);
    larger += __shfl_xor_sync(0xFFFFFFFFu, larger, 2);
    if ((tid & 3) == 0 && larger == n - 1 && best != 0)  // keys are distinct
        sh.threshold[word] = best;
    sync();
    return sh.threshold[word];
}

// Replaces the kept keys by the n largest of them, best first (0 where there are fewer).
__device__ __forceinline__ void compact(int n, Shared &sh)
{
    const int tid = threadIdx.x, kept = sh.kept;
    int left = kept;
    const uint64_t *from = sh.keep;
    if (tid < kMaxTop)
        sh.top[tid] = 0;
    if (kept > kRank) {  // what cannot be among the n best goes first
        uint64_t best = 0, k[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            k[i] = i * kThreads + tid < kept ? sh.keep[i * kThreads + tid] : 0;
            best = max(best, k[i]);
        }
        if (tid == 0)
            sh.left = 0;
        const uint64_t least = threshold_of(best, n, sh);
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (k[i] != 0 && k[i] >= least)
                sh.few[atomicAdd(&sh.left, 1)] = k[i];
        sync();
        left = sh.left;
        from = sh.few;
    } else {
        sync();
    }
    for (int i0 = 0; i0 < left; i0 += kThreads / 4) {  // four threads a key, with a quarter of the others each
        const int i = i0 + (tid >> 2);
        const uint64_t mine = i < left ? from[i] : ~0ull;
        int larger = 0;
#pragma unroll 4
        for (int j = tid & 3; j < left; j += 4)
            larger += from[j] > mine;
        larger += __shfl_xor_sync(0xFFFFFFFFu, larger, 1);
        larger += __shfl_xor_sync(0xFFFFFFFFu, larger, 2);
        if ((tid & 3) == 0 && i < left && larger < n)
            sh.top[larger] = mine;
    }
    sync();
    if (tid < n)
        sh.keep[tid] = sh.top[tid];
    if (tid == 0)
        sh.kept = min(left, n);
    sync();
}

// Elements of a row as vectors of 16 bytes, the ends perhaps in part. Vectors are copied to shared memory by the
// chunk, but where the logits begin or end inside one: its elements are loaded one by one.
template <bool kBf16>
struct Row {
    static constexpr int kPer = kBf16 ? 8 : 4;             // elements of a vector
    static constexpr int kVecs = kHold / kPer;             // a thread's of a chunk
    static constexpr int kStep = kThreads * kVecs;         // a chunk's
    static constexpr int kStages = kBf16 ? 4 : 2;          // chunks in shared memory: 64 KB of them
    static constexpr int kRing = kStages * kStep * 16;
    const char *base, *at;                                 // the row, and the multiple of 128 at or before it, so that copies
                                                           // begin on whole lines
    int lead, V;                                           // elements between them
    int w0, w1;                                            // vectors that lie in the logits whole
    int in0, in1;                                          // the block's whose elements are all the row's
    int v0, v1, chunks;                                    // the block's vectors

    __device__ __forceinline__ Row(const LogprobParams &p, long row, int rank, int ranks)
    {
        base = static_cast<const char *>(p.logits) + row * p.stride * (kBf16 ? 2 : 4);
        lead = (int)(reinterpret_cast<uintptr_t>(base) & 127) / (kBf16 ? 2 : 4);
        at = base - lead * (kBf16 ? 2 : 4);
        V = p.V;
        const int vecs = (lead + V + kPer - 1) / kPer, per = (vecs + ranks - 1) / ranks;
        v0 = rank * per;
        v1 = min(vecs, v0 + per);
        const char *first = static_cast<const char *>(p.logits), *last = first + ((p.N - 1) * p.stride + V) * (kBf16 ? 2 : 4);
        w0 = at >= first ? 0 : (int)((first - at + 15) >> 4);
        w1 = (int)min((long)vecs, (long)(last - at) >> 4);
        in0 = (lead + kPer - 1) / kPer;
        in1 = min(v1, (lead + V) / kPer);
        chunks = v0 < v1 ? (v1 - v0 + kStep - 1) / kStep : 0;
    }
    __device__ __forceinline__ float logit(int i) const
    {
        return kBf16 ? __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(base)[i] << 16) : reinterpret_cast<const float *>(base)[i];
    }
    // Whether a vector can be read whole: in the row, or at its end with bytes of the rows beside it.
    __device__ __forceinline__ bool whole(int vec) const { return vec >= w0 && vec < w1; }
    // ... and, of one that can, the row's elements, the others -infinity
    __device__ __forceinline__ uint4 trim(uint4 x, int vec) const
    {
        uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (!exists(vec, i)) {
                if (kBf16)
                    w[i / 2] = i & 1 ? (w[i / 2] & 0xFFFFu) | 0xFF800000u : (w[i / 2] & 0xFFFF0000u) | 0xFF80u;
                else
                    w[i & 3] = 0xFF800000u;
            }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ uint4 none()
    {
        const uint32_t w = kBf16 ? 0xFF80FF80u : 0xFF800000u;  // -infinity
        return make_uint4(w, w, w, w);
    }
    __device__ __forceinline__ uint4 part(int vec) const
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = vec * kPer - lead + i;
            const float x = e >= 0 && e < V ? logit(e) : -INFINITY;
            if (kBf16)
                w[i / 2] = i & 1 ? w[i / 2] | (__float_as_uint(x) & 0xFFFF0000u) : __float_as_uint(x) >> 16;
            else
                w[i & 3] = __float_as_uint(x);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ bool exists(int vec, int c) const { return vec < v1 && vec * kPer + c >= lead && vec * kPer + c < lead + V; }
    // the vectors of chunk c that can be read whole to `to`
    __device__ __forceinline__ void copy(int c, uint8_t *to, uint64_t *bar) const
    {
        const int first = v0 + c * kStep;
        const int lo = max(first, max(w0, lead / kPer)), hi = min(min(v1, first + kStep), w1);
        const uint32_t bytes = lo < hi ? (uint32_t)(hi - lo) * 16 : 0;
        mbar_arrive_expect_tx(bar, bytes);
        if (bytes)
            bulk_copy_g2s(to + (lo - first) * 16, at + (long)lo * 16, bytes, bar);
    }
};

template <bool kBf16>
__device__ __forceinline__ void unpack(uint4 w, float (&x)[kBf16 ? 8 : 4])
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if (kBf16) {
            x[2 * c] = bf16_lo(u[c]);
            x[2 * c + 1] = bf16_hi(u[c]);
        } else {
            x[c] = __uint_as_float(u[c]);
        }
    }
}

// Keeps the thread's elements that `pass` names, by their keys (0: not after all). Few threads have any, and few of
// their fours of elements.
template <typename R, typename Pass, typename Key>
__device__ __forceinline__ void keep_four(const float (&x)[R::kVecs][R::kPer], const Pass &pass, const Key &key, Shared &sh)
{
#pragma unroll
    for (int f = 0; f < R::kVecs * R::kPer / 4; ++f) {
        const int i = f * 4 / R::kPer, c0 = f * 4 % R::kPer;
        const float *const e = &x[i][c0];
        if (!pass(fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3]))))
            continue;
        uint32_t over = (pass(e[0]) ? 1u : 0u) | (pass(e[1]) ? 2u : 0u) | (pass(e[2]) ? 4u : 0u) | (pass(e[3]) ? 8u : 0u);
#pragma unroll 1
        for (; over; over &= over - 1) {
            const int c = __ffs(over) - 1;
            const uint64_t k = key(c < 2 ? (c == 0 ? e[0] : e[1]) : c == 2 ? e[2] : e[3], i, c0 + c);
            if (k != 0) {
                const int place = atomicAdd(&sh.kept, 1);
                if (place < kKeep)
                    sh.keep[place] = k;
            }
        }
    }
}

// The first chunk's threshold: keeps what reaches it among the thread's elements that `in` names (all, where it is
// `inside`), whose largest is `top`. Returns it (0: fewer than n groups have an element).
template <typename R, typename In>
__device__ __forceinline__ uint64_t keep_first(const float (&x)[R::kVecs][R::kPer], float top, int first, bool inside, int n, const In &in, Shared &sh)
{
    const auto key = [&](float y, int i, int c) { return key_of(y, (uint32_t)(first + i * kThreads * R::kPer + c)); };
    uint64_t best = 0;
    if (__all_sync(0xFFFFFFFFu, inside)) {  // the first of the largest
        int at = 0;
#pragma unroll
        for (int i = R::kVecs - 1; i >= 0; --i)
#pragma unroll
            for (int c = R::kPer - 1; c >= 0; --c)
                at = x[i][c] == top ? i * kThreads * R::kPer + c : at;
        best = key_of(top, (uint32_t)(first + at));
    } else {
#pragma unroll
        for (int i = 0; i < R::kVecs; ++i)
#pragma unroll
            for (int c = 0; c < R::kPer; ++c)
                if (in(i, c))
                    best = max(best, key(x[i][c], i, c));
    }
    const uint64_t least = threshold_of(best, n, sh);
    const float limit = least != 0 ? key_value(least) : -INFINITY;
    if (best != 0 && best >= least)
        keep_four<R>(x, [&](float y) { return y >= limit; }, [&](float y, int i, int c) {
            const uint64_t k = key(y, i, c);
            return k >= least && in(i, c) ? k : 0;
        }, sh);
    return least;
}

// Any chunk's threshold, for rows that are read again: keeps what reaches it among the thread's elements that
// `in` names. Returns it (0: fewer than n groups have an element).
template <typename R, typename In>
__device__ __forceinline__ uint64_t keep_best(const float (&x)[R::kVecs][R::kPer], int first, int n, const In &in, Shared &sh)
{
    const auto key = [&](int i, int c) { return key_of(x[i][c], (uint32_t)(first + i * kThreads * R::kPer + c)); };
    uint64_t best = 0;
#pragma unroll
    for (int i = 0; i < R::kVecs; ++i)
#pragma unroll
        for (int c = 0; c < R::kPer; ++c)
            if (in(i, c))
                best = max(best, key(i, c));
    const uint64_t least = threshold_of(best, n, sh);
    if (best != 0 && best >= least) {
#pragma unroll
        for (int i = 0; i < R::kVecs; ++i)
#pragma unroll
            for (int c = 0; c < R::kPer; ++c)
                if (in(i, c)) {
                    const uint64_t k = key(i, c);
                    if (k >= least)
                        sh.keep[atomicAdd(&sh.kept, 1)] = k;
                }
    }
    return least;
}

// The n best of the block's part of a row in bounded space, for rows whose order let too many elements pass the
// first chunk's threshold: each chunk has a threshold of its own, and the kept keys are ranked in between.
template <typename R>
__device__ __noinline__ void keep_again(const LogprobParams &p, long row, int rank, int ranks, Shared &sh)
{
    const R r(p, row, rank, ranks);
    const int tid = threadIdx.x, n = p.top;
    float limit = -INFINITY;
    bool has = false;
    sync();             // everyone has seen that too many were kept
    if (tid == 0)
        sh.kept = 0;
    for (int ch = 0; ch < r.chunks; ++ch) {
        const int v = r.v0 + ch * R::kStep + tid;
        float x[R::kVecs][R::kPer];
#pragma unroll
        for (int i = 0; i < R::kVecs; ++i) {
            const int at = v + i * kThreads;
            unpack<R::kPer == 8>(at >= r.v1 ? R::none() : r.whole(at) ? r.trim(*reinterpret_cast<const uint4 *>(r.at + (long)at * 16), at) : r.part(at), x[i]);
        }
        const uint64_t least = keep_best<R>(x, v * R::kPer - r.lead, n, [&](int i, int c) { return has ? x[i][c] > limit : r.exists(v + i * kThreads, c); }, sh);
        if (least != 0) {
            limit = key_value(least);
            has = true;
        }
        sync();
        if (sh.kept > kKeep / 2) {
            compact(n, sh);
            limit = key_value(sh.top[n - 1]);
            has = true;
        }
    }
    sync();
}

// Thread `who`'s sum of 2^d, of the row's part that it had, but for its elements that are the maximum: by a warp, its
// chunks' 16 elements two chunks at a time, eight loads ahead. (The others go on with the next row meanwhile.)
template <typename R>
__device__ __noinline__ float rest_of(const LogprobParams &p, long row, int ranks, int who, float m)
{
    constexpr int kAhead = 8, kStride = 32 / kHold * R::kStep * R::kPer;
    const R r(p, row, who / kThreads, ranks);
    const int lane = threadIdx.x & 31, c = lane % kHold;
    const int end = min(r.V, r.v1 * R::kPer - r.lead);
    float sum = 0.f;
    int at = (r.v0 + lane / kHold * R::kStep + c / R::kPer * kThreads + who % kThreads) * R::kPer + c % R::kPer - r.lead;
    if (at < 0)
        at += kStride;  // an element before the row
#pragma unroll 1
    for (; at < end; at += kAhead * kStride) {
        float x[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            x[j] = at + (long)j * kStride < end ? r.logit(at + j * kStride) : -INFINITY;
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            sum += x[j] < m ? ex2(fmaxf((x[j] - m) * kLog2e, kLeast)) : 0.f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    return sum;
}

// kRanks: CTAs of the cluster that shares a row; kTop: alternatives are asked for. The grid takes rows in turn; the copies run ahead of the chunk at
// hand, past the end of a row, so that a row's joins and lists do not stop them.
template <bool kBf16, int kRanks, bool kTop>
__global__ void __launch_bounds__(kBlock, 2) hc_logprobs_kernel(const LogprobParams p)
{
    using R = Row<kBf16>;
    constexpr int kPer = R::kPer, kVecs = R::kVecs, kStages = R::kStages;
    extern __shared__ uint4 ring[];
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        sh.kept = 0;
        sh.dead = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], kWarps);
        }
        mbar_fence_init();
    }
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();
    const int rank = kRanks == 1 ? 0 : (int)cluster_rank();
    const int rows = gridDim.x / kRanks, n = kTop ? p.top : 0;  // rows of the grid at a time
    const long row0 = blockIdx.x / kRanks;

    if (warp == kWarps) {
        if (lane == 0) {
            unsigned asked = 0;
            bool ok = true;
            for (long row = row0; ok && row < p.N; row += rows) {
                const R r(p, row, rank, kRanks);
                for (int c = 0; ok && c < r.chunks; ++c, ++asked) {
                    const unsigned stage = asked % kStages, use = asked / kStages;
                    ok = use == 0 || mbar_wait_bounded(&sh.empty[stage], (use & 1) ^ 1);  // (else the waits for it run out and say so)
                    if (ok)
                        r.copy(c, reinterpret_cast<uint8_t *>(ring + stage * R::kStep), &sh.full[stage]);
                }
            }
        }
        if (kRanks > 1) {
            cluster_sync();
            cluster_sync();
        }
        return;
    }

    const int back = kThreads - 1 - tid;             // results are the last threads'
    unsigned taken = 0;                              // chunks that came
    int turn = 0;                                    // rows, in turn
    uint32_t wait_limit = kWaitLimitNs;
#pragma unroll 1
    for (long row = row0; row < p.N; row += rows, turn ^= 1) {
        const R r(p, row, rank, kRanks);
        // a given token's logit is asked for before the pass
        const bool asks = rank == 0 && back < p.J;
        int token = -1;
        float given = 0.f;
        if (asks) {
            token = p.tokens[row * p.J + back];
            if (token >= 0 && token < p.V)
                given = r.logit(token);
        }
        Part a = no_part();                          // the thread's
        float limit = -INFINITY;                     // values up to this one are not among the n best
#pragma unroll 1
        for (int ch = 0; ch < r.chunks; ++ch, ++taken) {
            const int v = r.v0 + ch * R::kStep + tid, stage = (int)(taken % kStages);
            const uint32_t phase = (taken / kStages) & 1;
            if (kTop && ch == 3 && n > 2) {
                // The threads' maxima so far give a higher threshold (its elements come before this chunk's, so that of
                // equal ones none is missed). 20 of 128001: some 140 are kept in all, 320 with the first alone; 221 us for
                // 2048 rows, with two such thresholds 222, without 229; for one alternative 188, 193, 182.
                const uint64_t least = threshold_of(key_of(a.m, tid), n, sh, 1);  // (no barrier since chunk 0's)
                limit = fmaxf(limit, key_value(least));
            }
            if (!wait_bounded(&sh.full[stage], phase, wait_limit)) {
                *reinterpret_cast<volatile int *>(&sh.dead) = 1;
                if (p.status)
                    atomicExch(p.status, kStatusTimeout);
            }
            float x[kVecs][kPer];
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int at = v + i * kThreads;
                uint4 w = ring[stage * R::kStep + i * kThreads + tid];
                if (at < r.in0 || at >= r.in1)  // an end of the row, or past it
                    w = at >= r.v1 ? R::none() : r.whole(at) ? r.trim(w, at) : r.part(at);
                unpack<kBf16>(w, x[i]);
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.empty[stage]);
            float top = x[0][0];
            if (v - lane < r.v1) {  // the warp has some of the chunk
#pragma unroll
                for (int i = 0; i < kVecs; ++i)
#pragma unroll
                    for (int c = 0; c < kPer; ++c)
                        top = fmaxf(top, x[i][c]);
                if (top > a.m) {
                    const float d = max_nan((a.m - top) * kLog2e, kLeast), f = ex2(d);
                    a.s = f * fmaf(d, a.z, a.s);
                    a.z *= f;
                    a.m = top;
                }
                // Two elements an instruction. A -infinity makes the chunk's S a NaN: it is taken again with d bounded.
                const float ref = a.m == -INFINITY ? 0.f : a.m;
                const auto add = [&](auto bounded) {
                    const uint64_t by = f32x2(kLog2e, kLog2e), off = f32x2(-ref, -ref);
                    uint64_t z = 0, s = 0;
#pragma unroll
                    for (int i = 0; i < kVecs; ++i)
#pragma unroll
                        for (int c = 0; c < kPer; c += 2) {
                            uint64_t d = ffma2(fadd2(f32x2(x[i][c], x[i][c + 1]), off), by, 0x8000000080000000ull);  // (x - m) log2 e
                            float y0, y1;
                            f32x2_unpack(d, y0, y1);
                            if (decltype(bounded)::value) {
                                y0 = max_nan(y0, kLeast);
                                y1 = max_nan(y1, kLeast);
                                d = f32x2(y0, y1);
                            }
                            const uint64_t e = f32x2(ex2(y0), ex2(y1));
                            z = fadd2(z, e);
                            s = ffma2(d, e, s);
                        }
                    float z0, z1, s0, s1;
                    f32x2_unpack(z, z0, z1);
                    f32x2_unpack(s, s0, s1);
                    s0 += s1;
                    if (!decltype(bounded)::value && s0 != s0)
                        return false;
                    a.z += z0 + z1;
                    a.s += s0;
                    return true;
                };
                if (!add(std::false_type{}))
                    add(std::true_type{});
            }
            if (!kTop)
                continue;
            const int first = v * kPer - r.lead;
            if (ch == 0) {
                const uint64_t least = keep_first<R>(x, top, first, v >= r.in0 && v + (kVecs - 1) * kThreads < r.in1, n,
                                                     [&](int i, int c) { return r.exists(v + i * kThreads, c); }, sh);
                limit = least != 0 ? key_value(least) : INFINITY;  // (0: then there is no second chunk)
            } else if (top > limit) {
                keep_four<R>(x, [&](float y) { return y > limit; }, [&](float y, int i, int c) {
                    return key_of(y, (uint32_t)(first + i * kThreads * kPer + c));
                }, sh);
            }
        }
        a.who = tid;
        a = join_warp(a);
        if (lane == 0)
            sh.part[turn][warp] = a;
        sync();
        if (kTop) {
            if (sh.kept > kKeep)
                keep_again<R>(p, row, rank, kRanks, sh);
            compact(n, sh);
            if (tid == 0)
                sh.kept = 0;
        }
        if (kRanks == 1 && back - 31 + lane >= max(p.J, max(n, 1)))
            continue;                                // the warp has no results to write
        a = lane < kWarps ? sh.part[turn][lane] : no_part();
        a = join_warp(a);
        if (kRanks > 1) {
            if (tid == 0)
                sh.whole = a;
            cluster_sync();
            if (rank == 0) {
                a = no_part();
                if (lane < kRanks) {
                    const uint32_t from = dsmem_addr(&sh.whole, lane);
                    a = Part{dsmem_ld_f32(from), dsmem_ld_f32(from + 4), dsmem_ld_f32(from + 8), dsmem_ld_f32(from + 12),
                             __float_as_int(dsmem_ld_f32(from + 16)) + lane * kThreads};
                }
                a = join_warp(a);
                if (kTop && tid < n * kRanks) {  // the ranks' lists, n keys each
                    const uint32_t from = dsmem_addr(&sh.top[tid % max(n, 1)], tid / max(n, 1));
                    sh.all[tid] = (uint64_t)__float_as_uint(dsmem_ld_f32(from + 4)) << 32 | __float_as_uint(dsmem_ld_f32(from));
                }
            }
            cluster_sync();  // the others' memory has been read
            if (rank != 0)
                break;       // (a cluster has one row)
            if (tid < n * kRanks && sh.all[tid] != 0) {
                const uint64_t mine = sh.all[tid];
                int larger = 0;
                for (int j = 0; j < n * kRanks; ++j)
                    larger += sh.all[j] > mine;
                if (larger < n)
                    sh.top[larger] = mine;
            }
            sync();
        }
        // a row with a NaN, with +infinity, or with nothing but -infinity is no distribution
        const bool bad = !(a.m > -INFINITY && a.m < INFINITY) || !(a.z >= 0.f);
        const float log_z = bad ? kNaN : a.z < kNearlyOne ? log1pf(a.rest + rest_of<R>(p, row, kRanks, a.who, a.m)) : logf(a.z);
        bool wrong = bad;
        if (asks) {
            for (int j = back; j < p.J; j += kThreads) {
                if (j != back) {
                    token = p.tokens[row * p.J + j];
                    if (token >= 0 && token < p.V)
                        given = r.logit(token);
                }
                wrong |= token >= p.V;
                p.logp[row * p.J + j] = token < 0 ? 0.f : token >= p.V ? kNaN : (given - a.m) - log_z;
            }
        }
        if (back == 0 && p.entropy)
            p.entropy[row] = log_z - a.s * kLn2 / a.z;
        if (back < n) {
            const uint64_t k = sh.top[back];
            p.top_ids[row * n + back] = bad ? -1 : (int)key_index(k);
            p.top_logp[row * n + back] = (key_value(k) - a.m) - log_z;
        }
        if (wrong && p.status)
            atomicExch(p.status, kStatusInvalidArg);
    }
    if (*reinterpret_cast<volatile int *>(&sh.dead)) {  // a copy may still be in flight: give it time before the memory goes
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 50000000ull) {}
    }
}

template <bool kBf16, int kRanks>
cudaError_t launch(const LogprobParams &p, const LaunchCfg &cfg, cudaStream_t stream)
{
    auto *kernel = p.top > 0 ? hc_logprobs_kernel<kBf16, kRanks, true> : hc_logprobs_kernel<kBf16, kRanks, false>;
    int per_sm = 1;
    const cudaError_t e = attn_ready(reinterpret_cast<const void *>(kernel), kBlock, Row<kBf16>::kRing, &per_sm);
    if (e != cudaSuccess)
        return e;
    const int grid = kRanks > 1 ? p.N * kRanks : std::min(p.N, per_sm * cfg.sm_count);
    return launch_pdl(kernel, dim3((unsigned)grid), dim3(kBlock), Row<kBf16>::kRing, true, stream, p, kRanks);
}

template <bool kBf16>
cudaError_t launch_type(const LogprobParams &p, const LaunchCfg &cfg, cudaStream_t stream)
{
    // CTAs share a row, a cluster's, while all have SMs of their own (eight: while half of the SMs do) and each still has 4096
    // elements. With 1, 2, 4 and 8 of them, us, fp32, the five best: a row of 4096 7.5, 8.5, 8.3, 8.4; of 32768 12.7, 11.7,
    // 9.8, 9.1; of 128001 22.9, 18.2, 14.1, 12.5; 16 rows of 32768 12.7, 12.2, 10.3, 11.6; 40 rows of 128001 23.5, 19.2, 19.3,
    // 27.0; 80 rows of 32768 13.2, 16.0, 20.2, 30.8.
    int ranks = 1;
    while (ranks < 8 && (long)p.N * ranks * 2 <= cfg.sm_count / (ranks == 4 ? 2 : 1) && p.V / (ranks * 2) >= 4096)
        ranks *= 2;
    switch (ranks) {
    case 1: return launch<kBf16, 1>(p, cfg, stream);
    case 2: return launch<kBf16, 2>(p, cfg, stream);
    case 4: return launch<kBf16, 4>(p, cfg, stream);
    default: return launch<kBf16, 8>(p, cfg, stream);
    }
}

}  // namespace

cudaError_t launch_logprobs(const LogprobParams &p, bool bf16, const LaunchCfg &cfg, cudaStream_t stream)
{
    return bf16 ? launch_type<true>(p, cfg, stream) : launch_type<false>(p, cfg, stream);
}

}  // namespace tshc
