// hc_logprobs.cu -- log probabilities of given tokens, the distribution's entropy
// and its best alternatives (ts_hc_logprobs in include/ts_hc.h).
//
//   log p_v = x_v - m - log Z,  Z = sum_v e^(x_v - m),  m = max_v x_v
//   entropy = -sum_v p_v log p_v = log Z - S / Z,  S = sum_v (x_v - m) e^(x_v - m)
//
// One pass over the logits: each thread keeps a running maximum and Z and S
// relative to it, in fp32, and they are joined in a fixed order.
//
// The best alternatives come from the same pass. An element is a 64-bit key, its
// value in an order that unsigned comparison keeps above its index's complement, so
// that keys are distinct and the larger key is the larger value or, of equal ones,
// the lower index. A chunk of 8192 elements lies in the block's registers, and a
// threshold, which n elements are known to reach, says which of them are kept in
// shared memory: the n-th largest of the maxima of 128 groups of a chunk's elements
// is such a threshold, and at most n groups hold an element that reaches it. So what
// is kept is bounded for any logits, and the few hundred keys that a vocabulary leaves
// are ranked by counting, for each, the larger ones.
#include <algorithm>

#include "hc_prompt.h"
#include "ptx.cuh"

namespace tshc {

namespace {

constexpr unsigned kStatusInvalidArg = 1u;  // TS_ERR_INVALID_ARG of ts_hc.h
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kHold = 16;                    // elements of a chunk that a thread holds
constexpr int kGroups = kThreads / 4;        // of four threads each
constexpr int kMaxTop = 32;
constexpr int kDirect = 128;                 // threads that may keep elements without a new threshold
constexpr int kKeep = 4096;                  // keys kept; a chunk adds at most kMaxTop * 4 * kHold = kDirect * kHold
constexpr int kFew = 1024;                   // keys that a compaction leaves, at most kMaxTop * 4 * (kKeep / kThreads)
static_assert(kMaxTop * 4 * kHold <= kKeep / 2 && kDirect * kHold <= kKeep / 2, "a chunk's keys");
static_assert(kMaxTop * 4 * (kKeep / kThreads) <= kFew, "what a compaction leaves");
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNaN = __builtin_nanf("");

__device__ __forceinline__ float ex2f(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
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

// A distribution's part: its largest logit, and Z and S (in log2 units) relative to it.
struct Part {
    float m, z, s;
};

__device__ __forceinline__ Part join(Part a, Part b)
{
    const float m = fmaxf(a.m, b.m), ref = m == -INFINITY ? 0.f : m;
    const float da = max_nan((a.m - ref) * kLog2e, -200.f), db = max_nan((b.m - ref) * kLog2e, -200.f);
    const float fa = ex2f(da), fb = ex2f(db);
    return Part{m, a.z * fa + b.z * fb, fa * fmaf(da, a.z, a.s) + fb * fmaf(db, b.z, b.s)};
}

struct Shared {
    uint64_t keep[kKeep];
    uint64_t few[kFew];
    uint64_t group[kGroups];
    uint64_t top[kMaxTop];   // this block's, best first; a block of a cluster reads the others'
    uint64_t all[8 * kMaxTop];
    uint64_t threshold;
    Part part[kWarps];
    Part whole;
    int kept, left;
};

// The n-th largest of the groups' largest keys (0 if fewer than n groups have one).
__device__ __forceinline__ uint64_t threshold_of(uint64_t best, int n, Shared &sh)
{
    best = max(best, __shfl_xor_sync(0xFFFFFFFFu, best, 1));
    best = max(best, __shfl_xor_sync(0xFFFFFFFFu, best, 2));
    const int tid = threadIdx.x;
    if ((tid & 3) == 0)
        sh.group[tid >> 2] = best;
    if (tid == 0)
        sh.threshold = 0;
    __syncthreads();
    if (tid < kGroups) {
        const uint64_t mine = sh.group[tid];
        int larger = 0;
#pragma unroll 8
        for (int i = 0; i < kGroups; ++i)
            larger += sh.group[i] > mine;
        if (larger == n - 1 && mine != 0)  // keys are distinct
            sh.threshold = mine;
    }
    __syncthreads();
    return sh.threshold;
}

// Replaces the kept keys by the n largest of them, best first (0 where there are fewer).
__device__ __forceinline__ void compact(int n, Shared &sh)
{
    const int tid = threadIdx.x, kept = sh.kept;
    uint64_t best = 0, k[kKeep / kThreads];
#pragma unroll
    for (int i = 0; i < kKeep / kThreads; ++i) {
        k[i] = i * kThreads + tid < kept ? sh.keep[i * kThreads + tid] : 0;
        best = max(best, k[i]);
    }
    if (tid == 0)
        sh.left = 0;
    if (tid < kMaxTop)
        sh.top[tid] = 0;
    const uint64_t least = threshold_of(best, n, sh);
#pragma unroll
    for (int i = 0; i < kKeep / kThreads; ++i)
        if (k[i] != 0 && k[i] >= least)
            sh.few[atomicAdd(&sh.left, 1)] = k[i];
    __syncthreads();
    const int left = sh.left;
    for (int i = tid; i < left; i += kThreads) {
        const uint64_t mine = sh.few[i];
        int larger = 0;
#pragma unroll 4
        for (int j = 0; j < left; ++j)
            larger += sh.few[j] > mine;
        if (larger < n)
            sh.top[larger] = mine;
    }
    __syncthreads();
    if (tid < n)
        sh.keep[tid] = sh.top[tid];
    if (tid == 0)
        sh.kept = min(left, n);
    __syncthreads();
}

// Elements of a row as vectors of 16 bytes, the first and the last perhaps in part.
template <bool kBf16>
struct Row {
    static constexpr int kPer = kBf16 ? 8 : 4;  // elements of a vector
    const char *at;                             // a multiple of 16
    int lead, V;                                // elements before the row's first, in the first vector
    __device__ __forceinline__ void load(int vec, float (&x)[kPer]) const
    {
        const int first = vec * kPer - lead;
        const char *src = at + (long)vec * 16;
        if (first >= 0 && first + kPer <= V) {
            const uint4 w = __ldcs(reinterpret_cast<const uint4 *>(src));
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (kBf16) {
                    x[2 * i] = bf16_lo(u[i]);
                    x[2 * i + 1] = bf16_hi(u[i]);
                } else {
                    x[i] = __uint_as_float(u[i]);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                x[i] = -INFINITY;
                if (first + i >= 0 && first + i < V)
                    x[i] = kBf16 ? __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(src)[i] << 16)
                                 : reinterpret_cast<const float *>(src)[i];
            }
        }
    }
};

// kRanks: CTAs of the cluster that shares a row.
template <bool kBf16, int kRanks>
__global__ void __launch_bounds__(kThreads, 2) hc_logprobs_kernel(const LogprobParams p)
{
    constexpr int kPer = Row<kBf16>::kPer, kVecs = kHold / kPer;
    __shared__ Shared sh;
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = kRanks == 1 ? 0 : (int)cluster_rank();
    const long row = blockIdx.x / kRanks;
    const int n = p.top;
    Row<kBf16> r;
    const char *base = static_cast<const char *>(p.logits) + row * p.stride * (kBf16 ? 2 : 4);
    r.lead = (int)(reinterpret_cast<uintptr_t>(base) & 15) / (kBf16 ? 2 : 4);
    r.at = base - r.lead * (kBf16 ? 2 : 4);
    r.V = p.V;
    const int vecs = (r.lead + p.V + kPer - 1) / kPer, per = (vecs + kRanks - 1) / kRanks;
    const int v0 = rank * per, v1 = min(vecs, v0 + per);

    // a given token's logit is asked for before the pass
    const bool asks = rank == 0 && tid < p.J;
    int token = -1;
    float given = 0.f;
    const auto logit = [&](int t) {
        return kBf16 ? __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(base)[t] << 16) : reinterpret_cast<const float *>(base)[t];
    };
    if (asks) {
        token = p.tokens[row * p.J + tid];
        if (token >= 0 && token < p.V)
            given = logit(token);
    }
    if (tid == 0)
        sh.kept = 0;

    float x[kVecs][kPer], m = -INFINITY;
    float z[2] = {0.f, 0.f}, s[2] = {0.f, 0.f};
    float limit = -INFINITY;     // values up to this one are not among the n best (once there is a threshold)
    bool has = false;            // a threshold
    const auto fetch = [&](int v, float(&y)[kVecs][kPer]) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int at = v + i * kThreads + tid;
            if (at < v1) {
                r.load(at, y[i]);
            } else {
#pragma unroll
                for (int c = 0; c < kPer; ++c)
                    y[i][c] = -INFINITY;
            }
        }
    };
    if (v0 < v1)
        fetch(v0, x);
#pragma unroll 1
    for (int v = v0; v < v1; v += kVecs * kThreads) {
        float next[kVecs][kPer];
        const bool more = v + kVecs * kThreads < v1;
        if (more)
            fetch(v + kVecs * kThreads, next);
        float top = x[0][0];
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
#pragma unroll
            for (int c = 0; c < kPer; ++c)
                top = fmaxf(top, x[i][c]);
        if (top > m) {
            const float d = max_nan((m - top) * kLog2e, -200.f), f = ex2f(d);
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                s[a] = f * fmaf(d, z[a], s[a]);
                z[a] *= f;
            }
            m = top;
        }
        const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
#pragma unroll
            for (int c = 0; c < kPer; ++c) {
                const float d = max_nan((x[i][c] - ref) * kLog2e, -200.f), e = ex2f(d);
                z[c & 1] += e;
                s[c & 1] = fmaf(d, e, s[c & 1]);
            }
        if (n > 0) {
            const auto exists = [&](int i, int c) {
                const int at = v + i * kThreads + tid, e = at * kPer + c - r.lead;
                return at < v1 && e >= 0 && e < p.V;
            };
            const auto key = [&](int i, int c) { return key_of(x[i][c], (uint32_t)((v + i * kThreads + tid) * kPer + c - r.lead)); };
            const bool some = !has || top > limit;
            const int many = __syncthreads_count(some);
            if (many > 0) {
                uint64_t least = 0;
                if (many > kDirect) {
                    uint64_t best = 0;
                    if (some) {
#pragma unroll
                        for (int i = 0; i < kVecs; ++i)
#pragma unroll
                            for (int c = 0; c < kPer; ++c)
                                if (exists(i, c) && (!has || x[i][c] > limit))
                                    best = max(best, key(i, c));
                    }
                    least = threshold_of(best, n, sh);
                }
                if (some) {
#pragma unroll
                    for (int i = 0; i < kVecs; ++i)
#pragma unroll
                        for (int c = 0; c < kPer; ++c)
                            if (exists(i, c) && (!has || x[i][c] > limit)) {
                                const uint64_t k = key(i, c);
                                if (k >= least)
                                    sh.keep[atomicAdd(&sh.kept, 1)] = k;
                            }
                }
                __syncthreads();
                if (least != 0) {
                    limit = key_value(least);
                    has = true;
                }
                if (more && sh.kept > kKeep / 2) {
                    compact(n, sh);
                    if (sh.kept == n) {
                        limit = key_value(sh.top[n - 1]);
                        has = true;
                    }
                }
            }
        }
        if (more) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
#pragma unroll
                for (int c = 0; c < kPer; ++c)
                    x[i][c] = next[i][c];
        }
    }
    Part a{m, z[0] + z[1], s[0] + s[1]};
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        a = join(a, Part{__shfl_xor_sync(0xFFFFFFFFu, a.m, o), __shfl_xor_sync(0xFFFFFFFFu, a.z, o), __shfl_xor_sync(0xFFFFFFFFu, a.s, o)});
    if (lane == 0)
        sh.part[warp] = a;
    __syncthreads();
    if (n > 0)
        compact(n, sh);
    if (warp == 0) {
        a = lane < kWarps ? sh.part[lane] : Part{-INFINITY, 0.f, 0.f};
#pragma unroll
        for (int o = kWarps / 2; o > 0; o >>= 1)
            a = join(a, Part{__shfl_xor_sync(0xFFFFFFFFu, a.m, o), __shfl_xor_sync(0xFFFFFFFFu, a.z, o), __shfl_xor_sync(0xFFFFFFFFu, a.s, o)});
        if (lane == 0)
            sh.whole = a;
    }
    if (kRanks > 1) {
        cluster_sync();
        if (rank == 0) {
            if (warp == 0) {
                a = Part{-INFINITY, 0.f, 0.f};
                if (lane < kRanks) {
                    const uint32_t from = dsmem_addr(&sh.whole, lane);
                    a = Part{dsmem_ld_f32(from), dsmem_ld_f32(from + 4), dsmem_ld_f32(from + 8)};
                }
#pragma unroll
                for (int o = kRanks / 2; o > 0; o >>= 1)
                    a = join(a, Part{__shfl_xor_sync(0xFFFFFFFFu, a.m, o), __shfl_xor_sync(0xFFFFFFFFu, a.z, o), __shfl_xor_sync(0xFFFFFFFFu, a.s, o)});
            } else if (warp <= n * kRanks / 32 + 1) {  // the ranks' lists, n keys each
                const int i = tid - 32;
                if (i < n * kRanks) {
                    const uint32_t from = dsmem_addr(&sh.top[i % n], i / n);
                    sh.all[i] = (uint64_t)__float_as_uint(dsmem_ld_f32(from + 4)) << 32 | __float_as_uint(dsmem_ld_f32(from));
                }
            }
        }
        cluster_sync();  // the others' memory has been read
        if (rank != 0)
            return;
        if (tid == 0)
            sh.whole = a;
        if (n > 0) {
            if (tid < n * kRanks && sh.all[tid] != 0) {
                const uint64_t mine = sh.all[tid];
                int larger = 0;
                for (int j = 0; j < n * kRanks; ++j)
                    larger += sh.all[j] > mine;
                if (larger < n)
                    sh.top[larger] = mine;
            }
        }
    }
    __syncthreads();
    a = sh.whole;
    // a row with a NaN, with +infinity, or with nothing but -infinity is no distribution
    const bool bad = !(a.m > -INFINITY && a.m < INFINITY) || !(a.z >= 0.f);
    const float log_z = bad ? kNaN : logf(a.z);
    bool wrong = bad;
    if (asks) {
        for (int j = tid; j < p.J; j += kThreads) {
            if (j != tid) {
                token = p.tokens[row * p.J + j];
                if (token >= 0 && token < p.V)
                    given = logit(token);
            }
            wrong |= token >= p.V;
            p.logp[row * p.J + j] = token < 0 ? 0.f : token >= p.V ? kNaN : (given - a.m) - log_z;
        }
    }
    if (tid == 0 && p.entropy)
        p.entropy[row] = log_z - a.s * kLn2 / a.z;
    if (tid < n) {
        const uint64_t k = sh.top[tid];
        p.top_ids[row * n + tid] = bad ? -1 : (int)key_index(k);
        p.top_logp[row * n + tid] = (key_value(k) - a.m) - log_z;
    }
    if (wrong && p.status)
        atomicExch(p.status, kStatusInvalidArg);
}

template <bool kBf16, int kRanks>
cudaError_t launch(const LogprobParams &p, cudaStream_t stream)
{
    return launch_pdl(hc_logprobs_kernel<kBf16, kRanks>, dim3((unsigned)p.N * kRanks), dim3(kThreads), 0, true, stream, p, kRanks);
}

template <bool kBf16>
cudaError_t launch_type(const LogprobParams &p, const LaunchCfg &cfg, cudaStream_t stream)
{
    // CTAs share a row while there are not rows enough for two a SM and each still has 2048 elements.
    int ranks = 1;
    while (ranks < 8 && (long)p.N * ranks < cfg.sm_count && p.V / (ranks * 2) >= 2048)
        ranks *= 2;
    switch (ranks) {
    case 1: return launch<kBf16, 1>(p, stream);
    case 2: return launch<kBf16, 2>(p, stream);
    case 4: return launch<kBf16, 4>(p, stream);
    default: return launch<kBf16, 8>(p, stream);
    }
}

}  // namespace

cudaError_t launch_logprobs(const LogprobParams &p, bool bf16, const LaunchCfg &cfg, cudaStream_t stream)
{
    return bf16 ? launch_type<true>(p, cfg, stream) : launch_type<false>(p, cfg, stream);
}

}  // namespace tshc
