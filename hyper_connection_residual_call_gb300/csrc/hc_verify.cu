// hc_verify.cu -- which drafted tokens hold, and the token after them
// (ts_hc_verify in include/ts_hc.h).
//
// From the root: p the target's distribution at the node reached, q the draft's.
// What is left of p after rejections is R = max(p - c q, 0) with sum S:
//   c = 0, S = 1;  a child with token x holds iff u S q[x] < R[x];
//   a rejection makes c += S and S = sum_v max(p_v - c q_v, 0),
// since max(max(p - c q, 0) - S q, 0) = max(p - (c + S) q, 0): R is never stored,
// and a rejection costs one pass over the row for the new sum. The next token is
// argmax_v R_v / noise_v.
//
// A walk is a chain of passes over rows of V floats, each followed by a decision,
// and it needs only the rows that it reaches: with a tree of T nodes and a path of
// a few, reading all B T rows would cost many times the bytes. So a sequence is
// walked by one cluster of up to 8 CTAs, each with a slice of the vocabulary, and
// what counts is the latency of a step of the chain:
//   - a thread keeps its words of the target's row, and of the draft's once a child
//     was rejected, in registers (32 of each; longer slices read the rest again), so
//     that a pass is one round of loads and a further rejection none;
//   - the first child's row, the draft's row and the noise are asked into L2 while
//     the row at hand is worked on, and the first child's two probabilities are
//     loaded before the sums are there;
//   - a reduction has one cluster barrier: each warp leaves its result, and every warp
//     of the cluster reads all of them through distributed shared memory and joins them
//     in the same order, so that every CTA takes the same decisions.
// GPU times of calls replayed back to back in a CUDA graph: a chain of 5 nodes over 32768
// words 18 us, a node some 3 us (greedy 15). 16 trees of 26 nodes over 128001 words: 49 to 52 us,
// where the walks' 25 MB would take 4 (greedy 30, and 1.2): the longest walk's passes, one
// after the other, each a round of loads, the sums and an exchange between the CTAs.
#include <algorithm>

#include "hc_spec.h"
#include "ptx.cuh"

namespace tshc {

namespace {

constexpr unsigned kStatusInvalidArg = 1u;  // TS_ERR_INVALID_ARG of ts_hc.h
constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr float kLog2e = 1.4426950408889634f;

struct Pair {
    float a;
    float b;                  // a sum, or an index's bits
};

__device__ __forceinline__ float ex2f(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A float's bits in an order that unsigned comparison keeps, and back.
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t u = __float_as_uint(x);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

__device__ __forceinline__ float unordered(uint32_t u) { return __uint_as_float((u & 0x80000000u) ? u ^ 0x80000000u : ~u); }

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// The ways in which partial results meet, N of each lane: a maximum by one warp-wide
// integer reduction, sums by shuffles in a fixed order.
struct Softmax {              // (maximum, sum of 2^((l - maximum) k)); k is the caller's
    float k;
    template <int N>
    __device__ __forceinline__ Pair operator()(const Pair (&x)[N]) const
    {
        float m = x[0].a;
#pragma unroll
        for (int i = 1; i < N; ++i)
            m = fmaxf(m, x[i].a);
        m = unordered(__reduce_max_sync(0xFFFFFFFFu, ordered(m)));
        const float ref = m > -INFINITY ? m : 0.f;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i)
            sum += x[i].b * ex2f((x[i].a - ref) * k);
        return Pair{m, warp_sum(sum)};
    }
};

struct Sum {
    template <int N>
    __device__ __forceinline__ Pair operator()(const Pair (&x)[N]) const
    {
        float sum = x[0].a;
#pragma unroll
        for (int i = 1; i < N; ++i)
            sum += x[i].a;
        return Pair{warp_sum(sum), 0.f};
    }
};

struct Best {                 // (value, index): the largest value, the lowest index of equal ones
    static __device__ __forceinline__ Pair better(Pair x, Pair y)
    {
        const int i = __float_as_int(x.b), j = __float_as_int(y.b);
        return y.a > x.a || (y.a == x.a && j < i) ? y : x;
    }
    template <int N>
    __device__ __forceinline__ Pair operator()(const Pair (&x)[N]) const
    {
        Pair v = x[0];
#pragma unroll
        for (int i = 1; i < N; ++i)
            v = better(v, x[i]);
        const float m = unordered(__reduce_max_sync(0xFFFFFFFFu, ordered(v.a)));
        return Pair{m, __int_as_float(__reduce_min_sync(0xFFFFFFFFu, v.a == m ? __float_as_int(v.b) : 0x7FFFFFFF))};
    }
};

constexpr int kHold = 32;     // words of a row that a thread keeps
constexpr int kSmallTree = 1024;  // nodes whose parents and tokens are kept in shared memory

struct Scratch {
    Pair part[2][kVerifyWarps];  // the warps' results, by turns: one barrier a reduction is enough
    int parent[kSmallTree], token[kSmallTree];
};

// kRanks: CTAs of the cluster.
template <int kRanks, typename Op>
__device__ __forceinline__ Pair reduce(Pair v, const Op &op, const Pair none, Scratch &sc, int &turn)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Pair own[1] = {v};
    v = op(own);
    if (lane == 0)
        sc.part[turn][warp] = v;
    constexpr int kParts = kRanks * kVerifyWarps;  // 16 a CTA
    if (kRanks > 1)
        cluster_sync();
    else
        __syncthreads();
    Pair w[(kParts + 31) / 32];
#pragma unroll
    for (int i = 0; i < (kParts + 31) / 32; ++i) {
        const int at = i * 32 + lane;
        w[i] = none;
        if (kRanks > 1) {
            const uint32_t a = dsmem_addr(&sc.part[turn][at % kVerifyWarps], at / kVerifyWarps);
            w[i] = Pair{dsmem_ld_f32(a), dsmem_ld_f32(a + 4)};
        } else if (at < kParts) {
            w[i] = sc.part[turn][at];
        }
    }
    turn ^= 1;
    return op(w);
}

// Asks L2 for n floats, a line of 128 bytes a thread and step.
__device__ __forceinline__ void ask_l2(const float *p, int n)
{
    for (int i = threadIdx.x * 32; i < n; i += kVerifyThreads * 32)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p + i) : "memory");
}

template <int kRanks>
__global__ void __launch_bounds__(kVerifyThreads) hc_verify_kernel(const VerifyParams p)
{
    __shared__ Scratch sc;
    pdl_launch_dependents();
    pdl_wait();
    const int rank = kRanks == 1 ? 0 : (int)cluster_rank();
    const int b = blockIdx.x / kRanks, tid = threadIdx.x, lane = tid & 31;
    const int part = (p.V + kRanks - 1) / kRanks;
    const int v0 = min(p.V, rank * part), v1 = min(p.V, v0 + part);
    const bool lead = rank == 0 && tid == 0;
    const int32_t *parents = p.parents ? p.parents + (long)b * p.parents_stride : nullptr;
    const int32_t *tokens = p.tokens + (size_t)b * p.T;
    const float temp = p.draft ? p.temperature[b] : 0.f;
    const bool greedy = !(temp > 0.f);
    const float k = greedy ? 0.f : kLog2e / temp;
    const bool small = p.T <= kSmallTree;
    int turn = 0, cur = 0, count = 0;

    if (!greedy)
        ask_l2(p.noise + (size_t)b * p.V + v0, v1 - v0);
    if (small)
        for (int i = tid; i < p.T; i += kVerifyThreads) {
            sc.parent[i] = parents ? parents[i] : i - 1;
            sc.token[i] = tokens[i];
        }
    for (int i = rank * kVerifyThreads + tid; i < p.T; i += kRanks * kVerifyThreads)
        p.path[(size_t)b * p.T + i] = i == 0 ? 0 : -1;
    if (kRanks > 1)
        cluster_sync();  // the marks precede the accepted nodes, which the leader writes
    else
        __syncthreads();
    const auto parent_of = [&](int i) { return small ? sc.parent[i] : parents ? parents[i] : i - 1; };
    // The children of `node` among 32 nodes from i0 on, as a mask; and the first child (or -1).
    const auto kids_at = [&](int node, int i0) {
        const int i = i0 + lane;
        return __ballot_sync(0xFFFFFFFFu, i < p.T && parent_of(i) == node);
    };

    for (;;) {
        // the target's row at cur
        const float *row = p.logits + ((size_t)b * p.T + cur) * p.V;
        const float *draft = p.draft ? p.draft + ((size_t)b * p.T + cur) * p.V : nullptr;
        float l[kHold], q[kHold];
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            const int v = v0 + tid + i * kVerifyThreads;
            l[i] = v < v1 ? row[v] : -INFINITY;
        }
        int i0 = cur + 1;
        unsigned kids = 0;
        for (; i0 < p.T; i0 += 32) {
            kids = kids_at(cur, i0);
            if (kids)
                break;
        }
        const int first = kids ? i0 + __ffs(kids) - 1 : -1;
        float first_l = 0.f, first_q = 0.f, first_u = 0.f;
        if (first >= 0) {
            ask_l2(p.logits + ((size_t)b * p.T + first) * p.V + v0, v1 - v0);
            if (!greedy) {
                const int x = small ? sc.token[first] : tokens[first];
                if (x >= 0 && x < p.V) {
                    first_l = row[x];
                    first_q = draft[x];
                    first_u = p.u[(size_t)b * p.T + first];
                }
                ask_l2(draft + v0, v1 - v0);
            }
        }
        Pair st;
        if (greedy) {
            const Pair none{-INFINITY, __int_as_float(0x7FFFFFFF)};
            const Best best;
            st = none;
            bool nan = false;  // which better() passes over
#pragma unroll
            for (int i = 0; i < kHold; ++i) {
                if (v0 + tid + i * kVerifyThreads < v1)
                    st = best.better(st, Pair{l[i], __int_as_float(v0 + tid + i * kVerifyThreads)});
                nan |= l[i] != l[i];
            }
            for (int v = v0 + tid + kHold * kVerifyThreads; v < v1; v += kVerifyThreads) {
                const float x = row[v];
                st = best.better(st, Pair{x, __int_as_float(v)});
                nan |= x != x;
            }
            if (nan)  // before every other
                st = Pair{INFINITY, __int_as_float(-1)};
            st = reduce<kRanks>(st, best, none, sc, turn);
        } else {
            const Pair none{-INFINITY, 0.f};
            st = none;
#pragma unroll
            for (int i = 0; i < kHold; ++i)
                st.a = fmaxf(st.a, l[i]);
            const float ref = st.a > -INFINITY ? st.a : 0.f;
#pragma unroll
            for (int i = 0; i < kHold; ++i)
                st.b += ex2f((l[i] - ref) * k);
#pragma unroll 8
            for (int v = v0 + tid + kHold * kVerifyThreads; v < v1; v += kVerifyThreads) {
                const float x = row[v];
                if (x > st.a) {
                    st.b *= ex2f((st.a - x) * k);  // 0 at the first
                    st.a = x;
                }
                st.b += ex2f((x - (st.a > -INFINITY ? st.a : 0.f)) * k);
            }
            st = reduce<kRanks>(st, Softmax{k}, none, sc, turn);
        }
        const float m = st.a, inv = greedy || !(m > -INFINITY) ? 0.f : 1.f / st.b;
        const int top = greedy ? __float_as_int(st.b) : -1;
        // A NaN, and for a softmax an infinity or nothing but -infinity, is no distribution: the walk ends here.
        if (greedy ? top < 0 : !(st.b > 0.f))
            kids = 0;
        const auto prob = [&](float x) { return m > -INFINITY ? ex2f((x - m) * k) * inv : 0.f; };

        // its children, in their order
        float taken = 0.f, left = 1.f;
        int next = -1;
        bool have = false;  // whether l and q hold probabilities
        while (kids && next < 0) {
            const int node = i0 + __ffs(kids) - 1;
            kids &= kids - 1;
            const int x = small ? sc.token[node] : tokens[node];
            if (x < 0 || x >= p.V) {
                if (lead && p.status)
                    atomicExch(p.status, kStatusInvalidArg);
            } else if (greedy) {
                if (x == top)
                    next = node;
            } else {
                const float qx = node == first ? first_q : draft[x], lx = node == first ? first_l : row[x];
                const float ux = node == first ? first_u : p.u[(size_t)b * p.T + node];
                const float r = fmaxf(fmaf(-taken, qx, prob(lx)), 0.f);
                if (ux * left * qx < r) {
                    next = node;
                } else {
                    if (!have) {
                        have = true;
#pragma unroll
                        for (int i = 0; i < kHold; ++i) {
                            const int v = v0 + tid + i * kVerifyThreads;
                            q[i] = v < v1 ? draft[v] : 0.f;
                        }
#pragma unroll
                        for (int i = 0; i < kHold; ++i)
                            l[i] = prob(l[i]);
                    }
                    taken += left;
                    Pair sum{0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < kHold; ++i)
                        sum.a += fmaxf(fmaf(-taken, q[i], l[i]), 0.f);
#pragma unroll 8
                    for (int v = v0 + tid + kHold * kVerifyThreads; v < v1; v += kVerifyThreads)
                        sum.a += fmaxf(fmaf(-taken, draft[v], prob(row[v])), 0.f);
                    left = reduce<kRanks>(sum, Sum{}, Pair{0.f, 0.f}, sc, turn).a;
                }
            }
            while (!kids && next < 0 && parents && i0 + 32 < p.T) {
                i0 += 32;
                kids = kids_at(cur, i0);
            }
        }
        if (next >= 0) {
            cur = next;
            ++count;
            if (lead)
                p.path[(size_t)b * p.T + count] = cur;
            continue;
        }

        // no child is left: the next token
        int token = top;
        if (!greedy && st.b > 0.f) {
            const Best best;
            const Pair none{-1.f, __int_as_float(0x7FFFFFFF)};
            Pair win = none;
            const float *noise = p.noise + (size_t)b * p.V;
            const bool rest = have && left > 0.f;
#pragma unroll
            for (int i = 0; i < kHold; ++i) {
                const int v = v0 + tid + i * kVerifyThreads;
                if (v < v1) {
                    float r = have ? l[i] : prob(l[i]);
                    if (rest)
                        r = fmaxf(fmaf(-taken, q[i], r), 0.f);
                    win = best.better(win, Pair{__fdiv_rn(r, noise[v]), __int_as_float(v)});
                }
            }
#pragma unroll 8
            for (int v = v0 + tid + kHold * kVerifyThreads; v < v1; v += kVerifyThreads) {
                float r = prob(row[v]);
                if (rest)
                    r = fmaxf(fmaf(-taken, draft[v], r), 0.f);
                win = best.better(win, Pair{__fdiv_rn(r, noise[v]), __int_as_float(v)});
            }
            win = reduce<kRanks>(win, best, none, sc, turn);
            token = __float_as_int(win.b);
        }
        if (lead) {
            const bool found = token >= 0 && token < p.V;
            if (!found && p.status)
                atomicExch(p.status, kStatusInvalidArg);
            p.n_accepted[b] = count;
            p.next_token[b] = found ? token : 0;
        }
        break;
    }
    if (kRanks > 1)
        cluster_sync();  // no CTA's shared memory goes before the others have read it
}

}  // namespace

cudaError_t launch_verify(const VerifyParams &p, const LaunchCfg &cfg, cudaStream_t stream)
{
    // As many CTAs a sequence as the SMs hold (up to 8, a portable cluster), with
    // no fewer than 2048 words of a row for each. A chain of 5 over 32768 words: 18.4 us with
    // 8 or 4 CTAs, 23.8 with 2, 36 with 1; 8 trees of 8 over 16384: 20.2 with 4, 22.3 with 2.
    int ranks = 8;
    while (ranks > 1 && ((long)p.B * ranks > cfg.sm_count || p.V / ranks < 2048))
        ranks /= 2;
    cudaLaunchConfig_t lc{};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = ranks;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    lc.attrs = at;
    lc.numAttrs = 2;
    lc.stream = stream;
    lc.blockDim = dim3(kVerifyThreads);
    lc.gridDim = dim3((unsigned)(p.B * ranks));
    switch (ranks) {
    case 8: return cudaLaunchKernelEx(&lc, hc_verify_kernel<8>, p);
    case 4: return cudaLaunchKernelEx(&lc, hc_verify_kernel<4>, p);
    case 2: return cudaLaunchKernelEx(&lc, hc_verify_kernel<2>, p);
    default: return cudaLaunchKernelEx(&lc, hc_verify_kernel<1>, p);
    }
}

}  // namespace tshc
