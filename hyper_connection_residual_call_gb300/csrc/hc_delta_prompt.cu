// hc_delta_prompt.cu -- the gated delta rule over packed prompts, in chunks of 64
// tokens on the tensor cores (ts_hc_delta_prompt in include/ts_hc.h).
//
// Within a chunk that begins with the state S0 (D x D), with G_i the sum of the decays'
// logarithms up to token i, k_i and q_i of norm 1 (their norms' inverses are r_i and, with
// the scale, s_i), the updates u_i of
//     S <- e^g S,  u = beta (v - S^T k),  S <- S + k u^T,  o = scale S^T q
// are the rows of  U = T R,  with
//     R_i = v_i - e^(G_i) r_i (S0^T k_i),       T = (I + A)^-1 diag(beta),
//     A_ij = beta_i r_i r_j (k_i . k_j) e^(G_i - G_j)  for j < i, else 0,
// and then
//     o_i = e^(G_i) s_i (S0^T q_i) + sum_{j <= i} P_ij u_j,   P_ij = s_i r_j (q_i . k_j) e^(G_i - G_j)
//     S1  = e^(G_64) S0 + sum_j k_j w_j u_j^T,                 w_j = r_j e^(G_64 - G_j).
//
// What does not depend on the state is one kernel's, a block a chunk and key head: the
// products of keys and queries with keys, T by inverting blocks of 16 and joining them, P
// and the factors, in fp32; T and P are written as sums of two bf16 and in the order in
// which the second kernel's tensor cores want them, so that they come by one bulk copy.
//
// The second kernel walks a sequence's chunks, a block a value head. A TMEM lane is a
// column of the state. Two threads a lane keep that column in fp32 registers, half each;
// every operand that is made on the way (the state, R, U, w U) goes back to TMEM as an A
// operand's rows, so that nothing is exchanged between threads, and keys, queries, T and P
// are B operands as they lie in shared memory:
//     X = S0^T K^T   ->  R  ->   U = R T^T   ->   w U   ->   dS = (w U)^T K   ->   S1
// and beside that chain Y = S0^T Q^T and Z = U P^T, the outputs' two parts.
//
// Each of these operands is split into two bf16 (16 bits of significand), and each product
// into two or three: a state is off by some 2^-17 of the terms that made it, a chunk. (With
// one bf16 an operand it would be 2^-9.) Keys and queries are bf16 as they are; their norms
// are in the factors.
//
// What bounds it: the chain. A chunk's products take 1400 cycles of it, the work in between
// some 1000 instructions a scheduler, and there are three round trips.
//
// An infinity or a NaN reaches the outputs from its token on and the state, and nothing
// before: factors of a chunk's tokens from a bad key, decay or beta on make R a NaN, and a
// lane sets its R to 0 from the first that is not finite, and its outputs and state to NaN.
#include <cuda_bf16.h>

#include <algorithm>

#include "hc_attn.cuh"
#include "hc_prompt.h"
#include "hc_tc.h"
#include "umma.cuh"

namespace tshc {

namespace {

constexpr unsigned kStatusInvalidArg = 1u;   // TS_ERR_INVALID_ARG of ts_hc.h
constexpr int kChunk = 64;
constexpr int kTile = kChunk * 128;           // bytes of a 64 x 64 bf16 tile
// A record: T's and P's two parts (64 rows of 128 bytes, swizzled), then the factors.
constexpr int kTh = 0, kTl = kTile, kPh = 2 * kTile, kPl = 3 * kTile, kFactors = 4 * kTile;
constexpr int kRecord = kFactors + 1024;
struct Factors {
    float c[kChunk];          // -e^(G_i) r_i
    float w[kChunk];          // r_j e^(G_64 - G_j)
    float y[kChunk];          // e^(G_i) s_i
    float keep;               // e^(G_64)
};
static_assert(sizeof(Factors) <= kRecord - kFactors, "a record's factors");
constexpr float kNoDecay = -120.f;            // e^-120 is 0 in fp32; sums of -infinities would be no numbers
constexpr float kNaN = __builtin_nanf("");

// Records lie by value head, and within one by the sequence's first token / 64, plus the sequence, plus the chunk:
// no two sequences' overlap, and nobody needs a sum over the sequences before.
__host__ __device__ inline long record_slots(int N, int S) { return (long)N / kChunk + S; }
__device__ __forceinline__ long record_of(int start, int seq, int chunk) { return (long)(start / kChunk) + seq + chunk; }

// A sequence's rows; false for one that is out of range (recorded).
__device__ __forceinline__ bool rows_of(const DeltaPromptParams &p, int s, int &lo, int &n)
{
    lo = p.starts[s];
    const int hi = p.starts[s + 1];
    n = hi - lo;
    if (lo >= 0 && hi >= lo && hi <= p.N)
        return true;
    if (p.status && threadIdx.x == 0)
        atomicExch(p.status, kStatusInvalidArg);
    return false;
}

// ------------------------------------------------------------------ T, P and the factors

constexpr int kPrepThreads = 256;
constexpr int kPitch = 68;    // floats of a row of a 64 x 64 matrix in shared memory

template <int D>
struct PrepShared {
    uint16_t k[kChunk][D + 8], q[kChunk][D + 8];
    float kk[kChunk][kPitch], qk[kChunk][kPitch];
    float a[kChunk][kPitch], t[kChunk][kPitch], tmp[32][36];
    float r[kChunk], s[kChunk];                    // the inverse norms
    float gh[kChunk], gl[kChunk], beta[kChunk];    // G in two parts
    int bad_key, bad;                              // the first token with an infinity or a NaN
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], const void *at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(smem_addr(at)) : "memory");
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Eight values as two bf16 each, to piece x of row i of two tiles.
__device__ __forceinline__ void put8(uint8_t *hi, uint8_t *lo, int i, int x, const float (&v)[8])
{
    uint32_t h[4], l[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        h[c] = pack2_bf16(v[2 * c], v[2 * c + 1]);
        l[c] = pack2_bf16(v[2 * c] - bf16_lo(h[c]), v[2 * c + 1] - bf16_hi(h[c]));
    }
    const int at = i * 128 + ((x ^ (i & 7)) << 4);
    *reinterpret_cast<uint4 *>(hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4 *>(lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
}

template <int D>
__global__ void __launch_bounds__(kPrepThreads) hc_delta_prep_kernel(const DeltaPromptParams p)
{
    extern __shared__ uint4 smem4[];
    auto &sh = *reinterpret_cast<PrepShared<D> *>(smem4);
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long slots = record_slots(p.N, p.S);
    const long slot = blockIdx.x / p.Hk;
    const int hk = (int)(blockIdx.x - slot * p.Hk);
    // the sequence whose records this one is among: the last that begins at or before it
    int seq = 0;
    for (int lo = 0, hi = p.S - 1; lo < hi;) {
        const int mid = (lo + hi + 1) / 2;
        if (record_of(p.starts[mid], mid, 0) <= slot)
            lo = mid;
        else
            hi = mid - 1;
        seq = lo;
    }
    int first, len;
    if (!rows_of(p, seq, first, len))
        return;
    const long chunk = slot - record_of(first, seq, 0);
    if (chunk < 0 || chunk * kChunk >= len)
        return;
    first += (int)chunk * kChunk;
    const int n = min(kChunk, len - (int)chunk * kChunk);
    if (tid == 0)
        sh.bad_key = n;
    __syncthreads();

    // keys and queries, zeros after the last token, and their norms: D / 8 lanes a row
    constexpr int kPieces = D / 8;
    for (int i = tid; i < kChunk * kPieces * 2; i += kPrepThreads) {
        const bool query = i >= kChunk * kPieces;
        const int r = i / kPieces % kChunk, x = i % kPieces;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (r < n)
            w = *reinterpret_cast<const uint4 *>((query ? p.q + (size_t)(first + r) * p.q_stride : p.k + (size_t)(first + r) * p.k_stride) +
                                                 (size_t)hk * D + x * 8);
        *reinterpret_cast<uint4 *>(query ? &sh.q[r][x * 8] : &sh.k[r][x * 8]) = w;
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        float sum = 0.f;
        bool odd = false;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            sum = fmaf(bf16_lo(u[c]), bf16_lo(u[c]), sum);
            sum = fmaf(bf16_hi(u[c]), bf16_hi(u[c]), sum);
            odd |= !(fabsf(bf16_lo(u[c])) < INFINITY) || !(fabsf(bf16_hi(u[c])) < INFINITY);
        }
#pragma unroll
        for (int o = kPieces / 2; o > 0; o >>= 1)
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (odd && !query)
            atomicMin(&sh.bad_key, r);
        if (x == 0) {
            const float inv = p.norm_eps >= 0.f ? 1.f / sqrtf(sum + p.norm_eps) : 1.f;
            if (query)
                sh.s[r] = inv * p.scale;
            else
                sh.r[r] = inv;
        }
    }
    __syncthreads();

    // keys with keys (warps 0-3) and queries with keys (4-7), 16 rows a warp
    {
        const int row = (warp & 3) * 16;
        const bool query = warp >= 4;
        float d[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                d[i][c] = 0.f;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
            uint32_t a[4];
            const int ar = row + (lane & 15), ac = s * 16 + (lane >> 4) * 8;
            ldmatrix4(a, query ? &sh.q[ar][ac] : &sh.k[ar][ac]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // 16 columns: two tiles' two halves of the sum's 16 terms
                uint32_t b[4];
                ldmatrix4(b, &sh.k[i * 16 + (lane >> 4) * 8 + (lane & 7)][s * 16 + ((lane >> 3) & 1) * 8]);
                mma16816(d[2 * i], a, b[0], b[1]);
                mma16816(d[2 * i + 1], a, b[2], b[3]);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float *to = query ? &sh.qk[row + (lane >> 2)][i * 8 + (lane & 3) * 2] : &sh.kk[row + (lane >> 2)][i * 8 + (lane & 3) * 2];
            *reinterpret_cast<float2 *>(to) = make_float2(d[i][0], d[i][1]);
            *reinterpret_cast<float2 *>(to + 8 * kPitch) = make_float2(d[i][2], d[i][3]);
        }
    }

    const int group = p.Hv / p.Hk;
    for (int g = 0; g < group; ++g) {
        const int h = hk * group + g;
        uint8_t *const rec = p.work + ((size_t)h * slots + slot) * kRecord;
        auto &f = *reinterpret_cast<Factors *>(rec + kFactors);
        __syncthreads();                           // the products, and the head before
        if (warp == 0) {
            // the decays' sums in 64 bits, kept as two floats: differences of near ones are right after strong decays too
            double x[2];
            float bt[2];
            int bad = sh.bad_key;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 2 * lane + i;
                float d = 0.f;
                bt[i] = 0.f;
                if (r < n) {
                    d = p.decay[(size_t)(first + r) * p.Hv + h];
                    bt[i] = p.beta[(size_t)(first + r) * p.Hv + h];
                    if (!(d < INFINITY) || !(fabsf(bt[i]) < INFINITY) || !(sh.r[r] < INFINITY))
                        bad = min(bad, r);
                    d = fmaxf(d, kNoDecay);
                }
                x[i] = d;
            }
            bad = __reduce_min_sync(0xFFFFFFFFu, bad);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (2 * lane + i >= bad) {
                    x[i] = 0.0;
                    bt[i] = 0.f;
                }
            x[1] += x[0];
            double pre = x[1];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double y = __shfl_up_sync(0xFFFFFFFFu, pre, o);
                if (lane >= o)
                    pre += y;
            }
            const double all = __shfl_sync(0xFFFFFFFFu, pre, 31), before = pre - x[1];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 2 * lane + i;
                const double G = before + x[i];
                sh.gh[r] = (float)G;
                sh.gl[r] = (float)(G - (float)G);
                sh.beta[r] = bt[i];
                const float e = expf((float)G);
                f.c[r] = r < bad ? -e * sh.r[r] : r < n ? kNaN : 0.f;
                f.w[r] = r < bad ? expf((float)(all - G)) * sh.r[r] : 0.f;
                f.y[r] = e * sh.s[r];
            }
            if (lane == 0) {
                f.keep = expf((float)all);
                sh.bad = bad;
            }
        }
        __syncthreads();
        const int bad = sh.bad;
        // A and P, 8 columns of a row a time
        for (int u = tid; u < kChunk * 8; u += kPrepThreads) {
            const int i = u >> 3, x = u & 7;
            const float gh = sh.gh[i], gl = sh.gl[i], bi = sh.beta[i] * sh.r[i], si = sh.s[i];
            float pv[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const int j = x * 8 + c;
                const bool in = j <= i && i < bad;
                const float e = in ? expf((gh - sh.gh[j]) + (gl - sh.gl[j])) * sh.r[j] : 0.f;
                sh.a[i][j] = in && j < i ? bi * sh.kk[i][j] * e : 0.f;
                pv[c] = in ? si * sh.qk[i][j] * e : 0.f;
            }
            put8(rec + kPh, rec + kPl, i, x, pv);
        }
        __syncthreads();
        // T = (I + A)^-1: the blocks of 16 on the diagonal, a thread a column; the others' upper halves are 0
        if (tid < kChunk) {
            const int b = tid & 48, j = tid & 15;
            float t[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float sum = 0.f;
#pragma unroll
                for (int k = 0; k < i; ++k)
                    sum = fmaf(sh.a[b + i][b + k], t[k], sum);
                t[i] = i < j ? 0.f : i == j ? 1.f : -sum;
                sh.t[b + i][b + j] = t[i];
            }
        } else {
            for (int u = tid - kChunk; u < kChunk * kChunk; u += kPrepThreads - kChunk)
                if ((u & 63) >> 4 > u >> 10)
                    sh.t[u >> 6][u & 63] = 0.f;
        }
        __syncthreads();
        // (T11 0; T21 T22) has T21 = -T22 A21 T11: two pairs of blocks of 16, then one of 32
        {
            const int pair = tid >> 7, i = (tid >> 3) & 15, j = (tid & 7) * 2, b = pair * 32;
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const float a = sh.a[b + 16 + i][b + k];
                s0 = fmaf(a, sh.t[b + k][b + j], s0);
                s1 = fmaf(a, sh.t[b + k][b + j + 1], s1);
            }
            sh.tmp[pair * 16 + i][j] = s0;
            sh.tmp[pair * 16 + i][j + 1] = s1;
            __syncthreads();
            s0 = s1 = 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const float a = sh.t[b + 16 + i][b + 16 + k];
                s0 = fmaf(a, sh.tmp[pair * 16 + k][j], s0);
                s1 = fmaf(a, sh.tmp[pair * 16 + k][j + 1], s1);
            }
            sh.t[b + 16 + i][b + j] = -s0;
            sh.t[b + 16 + i][b + j + 1] = -s1;
            __syncthreads();
        }
        {
            const int i = tid >> 3, j = (tid & 7) * 4;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
            for (int k = 0; k < 32; ++k) {
                const float a = sh.a[32 + i][k];
                const float4 t = *reinterpret_cast<const float4 *>(&sh.t[k][j]);
                s = make_float4(fmaf(a, t.x, s.x), fmaf(a, t.y, s.y), fmaf(a, t.z, s.z), fmaf(a, t.w, s.w));
            }
            *reinterpret_cast<float4 *>(&sh.tmp[i][j]) = s;
            __syncthreads();
            s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
            for (int k = 0; k < 32; ++k) {
                const float a = sh.t[32 + i][32 + k];
                const float4 t = *reinterpret_cast<const float4 *>(&sh.tmp[k][j]);
                s = make_float4(fmaf(a, t.x, s.x), fmaf(a, t.y, s.y), fmaf(a, t.z, s.z), fmaf(a, t.w, s.w));
            }
            *reinterpret_cast<float4 *>(&sh.t[32 + i][j]) = make_float4(-s.x, -s.y, -s.z, -s.w);
            __syncthreads();
        }
        for (int u = tid; u < kChunk * 8; u += kPrepThreads) {
            const int i = u >> 3, x = u & 7;
            float tv[8];
#pragma unroll
            for (int c = 0; c < 8; ++c)
                tv[c] = sh.t[i][x * 8 + c] * sh.beta[x * 8 + c];
            put8(rec + kTh, rec + kTl, i, x, tv);
        }
    }
}

// ------------------------------------------------------------------ the walk over the chunks

constexpr int kColThreads = 256, kThreads = kColThreads + 128;  // two threads a column; the products, the copies, and two idle warps
constexpr int kMmaWarp = 8, kLoadWarp = 9;
constexpr int kColRegs = 216, kOtherRegs = 72;  // 256 * 216 + 128 * 72 = 64512 = 384 * 168, what the launch has
constexpr uint32_t kTmemCols = 512;
// TMEM columns. Where an operand takes an accumulator's place, each half of the threads writes over the 32 columns
// that it read itself: the high parts of its 32 tokens, then the low ones.
constexpr uint32_t kS = 0, kX = 128, kU = 192, kY = 256, kZ = 320, kDS = 384;  // kX: X, R, U; kU: U, w U

template <int D>
struct Stage {
    static constexpr int kRows = kChunk * D * 2;   // bytes of a chunk's keys, queries or values
    static constexpr int kK = 0, kQ = kRows, kV = 2 * kRows, kMat = 3 * kRows;
    static constexpr int kBytes = 3 * kRows + kRecord;                 // a multiple of 1024
    static constexpr int kTotal = 2 * kBytes + 1024;
    static_assert(kBytes % 1024 == 0, "a tile's alignment");
};

struct Shared {
    uint64_t full[2], empty[2];
    uint64_t s_ready, r_ready, w_ready, y_free;  // of the columns' threads
    uint64_t x_done, u_done, d_done, o_done;     // of the products
    uint32_t tmem;
    int dead;
    int bad[2][128];                             // by chunks in turn: a lane's first token that is not finite
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

// Two values as two bf16 each.
__device__ __forceinline__ void split2(uint64_t v, uint32_t &hi, uint32_t &lo)
{
    float a, z;
    f32x2_unpack(v, a, z);
    hi = pack2_bf16(a, z);
    f32x2_unpack(fadd2(v, f32x2(-bf16_lo(hi), -bf16_hi(hi))), a, z);
    lo = pack2_bf16(a, z);
}

__device__ __forceinline__ uint64_t pair_of(const uint32_t (&x)[32], int c) { return f32x2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])); }

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
hc_delta_scan_kernel(const __grid_constant__ DeltaPromptParams p, const __grid_constant__ CUtensorMap map_q,
                     const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v)
{
    using St = Stage<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Shared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t *const smem = smem_raw + (base - smem_addr(smem_raw));
    unsigned *const status = p.status;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1 + kColThreads / 32);
        }
        mbar_init(&sh.s_ready, kColThreads);
        mbar_init(&sh.r_ready, kColThreads);
        mbar_init(&sh.w_ready, kColThreads);
        mbar_init(&sh.y_free, kColThreads);
        mbar_init(&sh.x_done, 1);
        mbar_init(&sh.u_done, 1);
        mbar_init(&sh.d_done, 1);
        mbar_init(&sh.o_done, 1);
        sh.dead = 0;
        mbar_fence_init();
        fence_async_shared();
    }
    if (tid < 256)
        sh.bad[tid >> 7][tid & 127] = kChunk;
    if (warp == kMmaWarp) {
        tmem_alloc(&sh.tmem, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    pdl_launch_dependents();
    pdl_wait();
    const int seq = blockIdx.x / p.Hv, h = blockIdx.x - seq * p.Hv, hk = h / (p.Hv / p.Hk);
    int first, len;
    if (!rows_of(p, seq, first, len))
        len = 0;
    const int chunks = (len + kChunk - 1) / kChunk;

    if (warp < kMmaWarp) {
        // ---------------------------------------------------------- a column's two threads
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kColRegs));
        const int half = warp >> 2, col = (warp & 3) * 32 + lane;
        const bool there = col < D;
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        constexpr int kMine = D / 2;                // elements of the column that a thread has
        const size_t state_at = (((size_t)seq * p.Hv + h) * D + half * kMine) * D + col;
        float s[kMine];
#pragma unroll
        for (int i = 0; i < kMine; ++i)
            s[i] = there ? p.state_in[state_at + (size_t)i * D] : 0.f;
        const auto state_out = [&] {                // the state as an A operand: D / 4 columns a half and part
            uint32_t hi[16], lo[16];
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kMine / 32; ++i) {
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    split2(f32x2(s[32 * i + 2 * c], s[32 * i + 2 * c + 1]), hi[c], lo[c]);
                tmem_st16_async(lane_base + kS + half * (D / 2) + 16 * i, hi);
                tmem_st16_async(lane_base + kS + half * (D / 2) + D / 4 + 16 * i, lo);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&sh.s_ready);
        };
        if (chunks > 0)
            state_out();
        // (A wait that ran out ends nothing here: the warps go on through the same barriers, on whatever lies
        // there, and every further wait returns at once.)
#pragma unroll 1
        for (int ch = 0; ch < chunks; ++ch) {
            const int stage = ch & 1, n = min(kChunk, len - ch * kChunk), t0 = half * 32;
            const uint32_t phase = ch & 1;
            const uint8_t *const at = smem + stage * St::kBytes;
            const auto &f = *reinterpret_cast<const Factors *>(at + St::kMat + kFactors);
            uint32_t x[32], hi[16], lo[16];
            // R
            wait(&sh.full[stage], (ch >> 1) & 1, sh, status);
            uint32_t v[32];
#pragma unroll
            for (int c = 0; c < 32; ++c)
                v[c] = there && t0 + c < n ? (uint32_t) reinterpret_cast<const uint16_t *>(at + St::kV)[(t0 + c) * D + col] << 16 : 0u;
            wait(&sh.x_done, phase, sh, status);
            tc_fence_after();
            if (half == 0)                          // both threads of the column have read the last chunk's
                *reinterpret_cast<volatile int *>(&sh.bad[stage ^ 1][col]) = kChunk;
            tmem_ld32(lane_base + kX + t0, x);
            uint64_t odd = 0;                       // 0 times every element: a NaN if one is not finite
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                const float2 k = *reinterpret_cast<const float2 *>(&f.c[t0 + 2 * c]);
                const uint64_t r = ffma2(pair_of(x, c), f32x2(k.x, k.y), pair_of(v, c));
                odd = ffma2(r, 0, odd);
                split2(r, hi[c], lo[c]);
            }
            float odd0, odd1;
            f32x2_unpack(odd, odd0, odd1);
            const bool fine = odd0 == 0.f && odd1 == 0.f;
            if (!__all_sync(0xFFFFFFFFu, fine || !there)) {  // zeros from the first that is not finite
                bool gone = false;
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    const float r = fmaf(__uint_as_float(x[c]), f.c[t0 + c], __uint_as_float(v[c]));
                    if (!gone && !(fabsf(r) < INFINITY)) {
                        gone = true;
                        atomicMin(&sh.bad[stage][col], t0 + c);
                    }
                    if (gone) {
                        hi[c / 2] &= c & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                        lo[c / 2] &= c & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                    }
                }
            }
            __syncwarp();
            tmem_st16_async(lane_base + kX + t0, hi);
            tmem_st16_async(lane_base + kX + t0 + 16, lo);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&sh.r_ready);
            // U and w U
            wait(&sh.u_done, phase, sh, status);
            tc_fence_after();
            tmem_ld32(lane_base + kU + t0, x);
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                const float2 w = *reinterpret_cast<const float2 *>(&f.w[t0 + 2 * c]);
                split2(ffma2(pair_of(x, c), f32x2(w.x, w.y), 0x8000000080000000ull), hi[c], lo[c]);
            }
            tmem_st16_async(lane_base + kU + t0, hi);
            tmem_st16_async(lane_base + kU + t0 + 16, lo);
#pragma unroll
            for (int c = 0; c < 16; ++c)
                split2(pair_of(x, c), hi[c], lo[c]);
            tmem_st16_async(lane_base + kX + t0, hi);
            tmem_st16_async(lane_base + kX + t0 + 16, lo);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&sh.w_ready);
            // the state
            const float keep = f.keep;
            wait(&sh.d_done, phase, sh, status);
            tc_fence_after();
            const int bad = *reinterpret_cast<volatile int *>(&sh.bad[stage][col]);
#pragma unroll
            for (int i = 0; i < kMine / 32; ++i) {
                tmem_ld32(lane_base + kDS + half * kMine + 32 * i, x);
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    s[32 * i + c] = fmaf(s[32 * i + c], keep, __uint_as_float(x[c]));
            }
            if (bad < kChunk)
#pragma unroll
                for (int i = 0; i < kMine; ++i)
                    s[i] = kNaN;
            if (ch + 1 < chunks)
                state_out();
            // the outputs
            wait(&sh.o_done, phase, sh, status);
            tc_fence_after();
            tmem_ld32(lane_base + kY + t0, x);
            tmem_ld32(lane_base + kZ + t0, v);
            tc_fence_before();
            mbar_arrive(&sh.y_free);
            uint16_t *const out = p.out + ((size_t)(first + ch * kChunk + t0) * p.Hv + h) * D + col;
#pragma unroll
            for (int c = 0; c < 32; ++c) {
                float o = fmaf(f.y[t0 + c], __uint_as_float(x[c]), __uint_as_float(v[c]));
                o = t0 + c >= bad ? kNaN : o;
                if (there && t0 + c < n)
                    out[(size_t)c * p.Hv * D] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.empty[stage]);
        }
        if (there && (chunks > 0 || p.state_out != p.state_in))
#pragma unroll
            for (int i = 0; i < kMine; ++i)
                p.state_out[state_at + (size_t)i * D] = s[i];
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kMmaWarp) {
            // ---------------------------------------------------------- products
            constexpr uint32_t kIdesc = umma_idesc_bf16(128, kChunk), kIdescS = umma_idesc_bf16(128, D) | kIdescBMnMajor;
            bool ok = true;
#pragma unroll 1
            for (int ch = 0; ok && ch < chunks; ++ch) {
                const int stage = ch & 1, n = min(kChunk, len - ch * kChunk);
                const uint32_t phase = ch & 1, at = base + stage * St::kBytes;
                ok = wait(&sh.full[stage], (ch >> 1) & 1, sh, status);
                if (!ok)
                    break;
                if (n < kChunk) {  // keys after the last are another sequence's: their products with zeros have to be zeros
                    for (int i = lane; i < (kChunk - n) * (D / 8); i += 32) {
                        const int r = n + i / (D / 8), x = i % (D / 8);
                        *reinterpret_cast<uint4 *>(smem + stage * St::kBytes + St::kK + (x >> 3) * kTile + r * 128 + (x & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_async_shared();
                    __syncwarp();
                }
                const uint32_t k = desc_lo(at + St::kK, 16), q = desc_lo(at + St::kQ, 16);
                // one operand of D terms in TMEM (the state), the other's rows in shared memory
                const auto by_state = [&](uint32_t to, uint32_t b) {
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            const int of = i / (D / 32), in = i % (D / 32);  // the half of the column
                            umma_bf16_ts_lo(tmem + to, tmem + kS + of * (D / 2) + part * (D / 4) + in * 8, b + (((i >> 2) * kTile + (i & 3) * 32) >> 4), kIdesc,
                                            part + i > 0);
                        }
                };
                // ... of 64 tokens, and 64 rows of a record's tile
                const auto by_tokens = [&](uint32_t to, uint32_t from, int part, int tile, uint32_t more) {
                    const uint32_t b = desc_lo(at + St::kMat + tile, 16);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        umma_bf16_ts_lo(tmem + to, tmem + from + (i >> 1) * 32 + part * 16 + (i & 1) * 8, b + ((i * 32) >> 4), kIdesc, more + i > 0);
                };
                ok = wait(&sh.s_ready, phase, sh, status);
                if (!ok)
                    break;
                tc_fence_after();
                if (elect_one()) {
                    by_state(kX, k);
                    umma_commit(&sh.x_done);
                }
                __syncwarp();
                if (ch > 0) {
                    ok = wait(&sh.y_free, phase ^ 1, sh, status);
                    if (!ok)
                        break;
                    tc_fence_after();
                }
                if (elect_one())
                    by_state(kY, q);
                __syncwarp();
                ok = wait(&sh.r_ready, phase, sh, status);
                if (!ok)
                    break;
                tc_fence_after();
                if (elect_one()) {
                    by_tokens(kU, kX, 0, kTh, 0);
                    by_tokens(kU, kX, 1, kTh, 1);
                    by_tokens(kU, kX, 0, kTl, 1);
                    umma_commit(&sh.u_done);
                }
                __syncwarp();
                ok = wait(&sh.w_ready, phase, sh, status);
                if (!ok)
                    break;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t km = desc_lo(at + St::kK, kTile);
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            umma_bf16_ts_lo(tmem + kDS, tmem + kU + (i >> 1) * 32 + part * 16 + (i & 1) * 8, km + i * (2048 >> 4), kIdescS, part + i > 0);
                    umma_commit(&sh.d_done);
                    by_tokens(kZ, kX, 0, kPh, 0);
                    by_tokens(kZ, kX, 1, kPh, 1);
                    by_tokens(kZ, kX, 0, kPl, 1);
                    umma_commit(&sh.o_done);
                    umma_commit(&sh.empty[stage]);
                }
                __syncwarp();
            }
        } else if (warp == kLoadWarp) {
            // ---------------------------------------------------------- copies
            const long slots = record_slots(p.N, p.S);
            const uint8_t *const rec = p.work + ((size_t)h * slots + record_of(first, seq, 0)) * kRecord;
            bool ok = true;
#pragma unroll 1
            for (int ch = 0; ok && ch < chunks; ++ch) {
                const int stage = ch & 1;
                ok = wait(&sh.empty[stage], ((ch >> 1) & 1) ^ 1, sh, status);
                if (ok && lane == 0) {
                    uint8_t *const to = smem + stage * St::kBytes;
                    uint64_t *bar = &sh.full[stage];
                    const int row = first + ch * kChunk;
                    mbar_arrive_expect_tx(bar, 3 * St::kRows + kRecord);
                    for (int i = 0; i < D / 64; ++i)
                        tma_load_3d(to + St::kK + i * kTile, &map_k, i * 64, hk, row, bar);
                    bulk_copy_g2s(to + St::kMat, rec + (size_t)ch * kRecord, kRecord, bar);
                    for (int i = 0; i < D / 64; ++i)
                        tma_load_3d(to + St::kQ + i * kTile, &map_q, i * 64, hk, row, bar);
                    tma_load_3d(to + St::kV, &map_v, 0, h, row, bar);
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
cudaError_t launch(const DeltaPromptParams &p, cudaStream_t stream)
{
    int per_sm = 1;
    cudaError_t e = attn_ready(reinterpret_cast<const void *>(hc_delta_prep_kernel<D>), kPrepThreads, (int)sizeof(PrepShared<D>), &per_sm);
    if (e == cudaSuccess)
        e = attn_ready(reinterpret_cast<const void *>(hc_delta_scan_kernel<D>), kThreads, Stage<D>::kTotal, &per_sm);
    if (e != cudaSuccess)
        return e;
    static_assert(Stage<D>::kTotal + sizeof(Shared) <= 227 * 1024 && sizeof(PrepShared<D>) <= 227 * 1024, "shared memory");
    CUtensorMap map_q{}, map_k{}, map_v{};
    if (p.N > 0 && (!tc_make_map_heads(&map_q, p.q, p.N, p.Hk, D, p.q_stride, 1, kChunk) ||
                    !tc_make_map_heads(&map_k, p.k, p.N, p.Hk, D, p.k_stride, 1, kChunk) ||
                    !tc_make_map_heads(&map_v, p.v, p.N, p.Hv, D, p.v_stride, 1, kChunk, true)))
        return cudaErrorInvalidValue;
    e = launch_pdl(hc_delta_prep_kernel<D>, dim3((unsigned)(record_slots(p.N, p.S) * p.Hk)), dim3(kPrepThreads), sizeof(PrepShared<D>), true, stream, p);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t lc{};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = at;
    lc.numAttrs = 1;
    lc.stream = stream;
    lc.blockDim = dim3(kThreads);
    lc.gridDim = dim3((unsigned)(p.S * p.Hv));
    lc.dynamicSmemBytes = Stage<D>::kTotal;
    return cudaLaunchKernelEx(&lc, hc_delta_scan_kernel<D>, p, map_q, map_k, map_v);
}

}  // namespace

size_t delta_prompt_bytes(int N, int S, int Hv) { return (size_t)record_slots(N, S) * Hv * kRecord; }

cudaError_t launch_delta_prompt(const DeltaPromptParams &p, const LaunchCfg &, cudaStream_t stream)
{
    return p.D == 64 ? launch<64>(p, stream) : launch<128>(p, stream);
}

}  // namespace tshc
