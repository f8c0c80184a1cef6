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
// walked by one cluster of up to 8 CTAs, each with a slice of the vocabulary; the
// sums and maxima of the slices meet through distributed shared memory, in rank
// order, and every CTA takes the same decisions from them.
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

// The ways in which two partial results meet.
struct Softmax {              // (maximum, sum of 2^((l - maximum) k)); k is the caller's
    float k;
    __device__ __forceinline__ Pair operator()(Pair x, Pair y) const
    {
        const float m = fmaxf(x.a, y.a);
        if (m == -INFINITY)
            return Pair{m, x.b + y.b};
        return Pair{m, x.b * ex2f((x.a - m) * k) + y.b * ex2f((y.a - m) * k)};
    }
};

struct Sum {
    __device__ __forceinline__ Pair operator()(Pair x, Pair y) const { return Pair{x.a + y.a, 0.f}; }
};

struct Best {                 // (value, index): the largest value, the lowest index of equal ones
    __device__ __forceinline__ Pair operator()(Pair x, Pair y) const
    {
        const int i = __float_as_int(x.b), j = __float_as_int(y.b);
        return y.a > x.a || (y.a == x.a && j < i) ? y : x;
    }
};

struct Scratch {
    Pair warp[kVerifyWarps];
    Pair slot[2];             // this CTA's result, by turns, so that one cluster barrier a reduction is enough
};

template <typename Op>
__device__ __forceinline__ Pair reduce(Pair v, const Op &op, Scratch &sc, int &turn, int ranks)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const Pair w{__shfl_xor_sync(0xFFFFFFFFu, v.a, o), __shfl_xor_sync(0xFFFFFFFFu, v.b, o)};
        v = (lane & o) ? op(w, v) : op(v, w);  // the same order in both lanes
    }
    if (lane == 0)
        sc.warp[warp] = v;
    __syncthreads();
    v = sc.warp[0];
#pragma unroll
    for (int w = 1; w < kVerifyWarps; ++w)
        v = op(v, sc.warp[w]);
    if (ranks == 1) {
        __syncthreads();  // sc.warp is free again
        return v;
    }
    if (threadIdx.x == 0)
        sc.slot[turn] = v;
    cluster_sync();
    for (int r = 0; r < ranks; ++r) {
        const uint32_t at = dsmem_addr(&sc.slot[turn], r);
        const Pair w{dsmem_ld_f32(at), dsmem_ld_f32(at + 4)};
        v = r == 0 ? w : op(v, w);
    }
    turn ^= 1;
    return v;
}

__global__ void __launch_bounds__(kVerifyThreads) hc_verify_kernel(const VerifyParams p, const int ranks)
{
    __shared__ Scratch sc;
    pdl_launch_dependents();
    pdl_wait();
    const int rank = ranks == 1 ? 0 : (int)cluster_rank();
    const int b = blockIdx.x / ranks, tid = threadIdx.x, lane = tid & 31;
    const int part = (p.V + ranks - 1) / ranks;
    const int v0 = min(p.V, rank * part), v1 = min(p.V, v0 + part);
    const bool lead = rank == 0 && tid == 0;
    const int32_t *parents = p.parents ? p.parents + (long)b * p.parents_stride : nullptr;
    const int32_t *tokens = p.tokens + (size_t)b * p.T;
    const float temp = p.draft ? p.temperature[b] : 0.f;
    const bool greedy = !(temp > 0.f);
    const float k = greedy ? 0.f : kLog2e / temp;
    int turn = 0, cur = 0, count = 0;

    for (int i = (rank * kVerifyThreads + tid); i < p.T; i += ranks * kVerifyThreads)
        if (i > 0)
            p.path[(size_t)b * p.T + i] = -1;
    if (lead)
        p.path[(size_t)b * p.T] = 0;
    if (ranks > 1)
        cluster_sync();  // the marks precede the accepted nodes, which the leader writes
    else
        __syncthreads();

    for (;;) {
        // the target at cur
        const float *row = p.logits + ((size_t)b * p.T + cur) * p.V;
        const float *draft = p.draft ? p.draft + ((size_t)b * p.T + cur) * p.V : nullptr;
        Pair st{-INFINITY, greedy ? __int_as_float(0x7FFFFFFF) : 0.f};
        if (greedy) {
            const Best best;
#pragma unroll 8
            for (int v = v0 + tid; v < v1; v += kVerifyThreads)
                st = best(st, Pair{row[v], __int_as_float(v)});
            st = reduce(st, best, sc, turn, ranks);
        } else {
            const Softmax soft{k};
#pragma unroll 8
            for (int v = v0 + tid; v < v1; v += kVerifyThreads) {
                const float l = row[v];
                if (l > st.a) {
                    st.b *= ex2f((st.a - l) * k);  // 0 at the first
                    st.a = l;
                }
                if (st.a > -INFINITY)
                    st.b += ex2f((l - st.a) * k);
            }
            st = reduce(st, soft, sc, turn, ranks);
        }
        const float m = st.a, inv = greedy || !(m > -INFINITY) ? 0.f : 1.f / st.b;
        const int top = greedy ? __float_as_int(st.b) : 0;
        const auto prob = [&](float l) { return m > -INFINITY ? ex2f((l - m) * k) * inv : 0.f; };

        // its children, in their order
        float taken = 0.f, left = 1.f;
        int next = -1;
        for (int i0 = cur + 1; i0 < p.T && next < 0; i0 += 32) {
            const int i = i0 + lane;
            unsigned kids = __ballot_sync(0xFFFFFFFFu, i < p.T && (parents ? parents[i] == cur : i == cur + 1));
            while (kids && next < 0) {
                const int node = i0 + __ffs(kids) - 1;
                kids &= kids - 1;
                const int x = tokens[node];
                if (x < 0 || x >= p.V) {
                    if (lead && p.status)
                        atomicExch(p.status, kStatusInvalidArg);
                    continue;
                }
                if (greedy) {
                    if (x == top)
                        next = node;
                    continue;
                }
                const float q = draft[x], r = fmaxf(fmaf(-taken, q, prob(row[x])), 0.f);
                if (p.u[(size_t)b * p.T + node] * left * q < r) {
                    next = node;
                    continue;
                }
                taken += left;
                Pair sum{0.f, 0.f};
#pragma unroll 8
                for (int v = v0 + tid; v < v1; v += kVerifyThreads)
                    sum.a += fmaxf(fmaf(-taken, draft[v], prob(row[v])), 0.f);
                left = reduce(sum, Sum{}, sc, turn, ranks).a;
            }
            if (!parents)
                break;  // a chain: the only child was looked at
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
        if (!greedy) {
            const Best best;
            Pair win{-1.f, __int_as_float(0x7FFFFFFF)};
            const float *noise = p.noise + (size_t)b * p.V;
            const bool rest = taken > 0.f && left > 0.f;
#pragma unroll 8
            for (int v = v0 + tid; v < v1; v += kVerifyThreads) {
                float r = prob(row[v]);
                if (rest)
                    r = fmaxf(fmaf(-taken, draft[v], r), 0.f);
                win = best(win, Pair{__fdiv_rn(r, noise[v]), __int_as_float(v)});
            }
            win = reduce(win, best, sc, turn, ranks);
            token = __float_as_int(win.b);
        }
        if (lead) {
            p.n_accepted[b] = count;
            p.next_token[b] = token >= 0 && token < p.V ? token : 0;
        }
        break;
    }
    if (ranks > 1)
        cluster_sync();  // no CTA's shared memory goes before the others have read it
}

}  // namespace

cudaError_t launch_verify(const VerifyParams &p, const LaunchCfg &cfg, cudaStream_t stream)
{
    // As many CTAs a sequence as the SMs hold (up to 8, a portable cluster), with
    // no fewer than 2048 words of a row for each.
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
    return cudaLaunchKernelEx(&lc, hc_verify_kernel, p, ranks);
}

}  // namespace tshc
