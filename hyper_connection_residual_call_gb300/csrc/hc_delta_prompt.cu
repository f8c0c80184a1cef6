// hc_delta_prompt.cu -- the gated delta rule over packed prompts, in chunks of 64
// tokens on the tensor cores (ts_hc_delta_prompt in include/ts_hc.h).
//
// Within a chunk that begins with the state S0 (D x D), with G_i the sum of the decays'
// logarithms up to token i, and r_i, s_i the inverses of the norms of k_i, q_i (s_i with the
// scale), the updates u_i of
//     S <- e^g S,  u = beta (v - S^T k),  S <- S + k u^T,  o = scale S^T q
// are the rows of  U = T R,  with
//     R_i = v_i - e^(G_i) r_i X_i,   X_i = S0^T k_i,     T = (I + A)^-1 diag(beta),
//     A_ij = beta_i r_i r_j (k_i . k_j) e^(G_i - G_j)  for j < i, else 0,
// and then
//     o_i = e^(G_i) s_i (S0^T q_i) + sum_{j <= i} P_ij u_j,   P_ij = s_i r_j (q_i . k_j) e^(G_i - G_j)
//     S1  = e^(G_64) S0 + sum_j k_j w_j u_j^T,                 w_j = r_j e^(G_64 - G_j).
//
// What does not depend on the state is one kernel's, a block a chunk and key head: the
// products of keys and queries with keys, T by inverting blocks of 16 and joining them, P
// and the factors, in fp32, written in the order in which the second kernel's tensor cores
// want them, so that they come by bulk copies.
//
// The second kernel walks a sequence's chunks, a CTA a value head. A TMEM lane is a column of
// the state. Operands that are made on the way (the state, R, U, w U) go back to TMEM as
// rows of A operands, from the threads that own the lane, so that but for the largest element
// nothing is exchanged between threads; keys, queries, T and P are B operands in shared memory. From chunk to
// chunk, X would have to wait for the state; but with S1 put in,
//     X' = e^(G_64) (S0^T K'^T) + (w U)^T M^T,   M = K' K^T  of this chunk's and the next one's keys,
// whose first part needs the state before and whose second needs no state: so the chain from
// chunk to chunk is  M's product -> R -> T's product -> w U,  and what is the state's (its
// update, its split, the next chunk's S0^T K'^T) and the outputs fall into the waits for T's and
// for M's product. A column has four threads; the state stays in their fp32 registers.
//
// Each operand is scaled by a power of two (a column of the state, of R and of U by its own, a
// row of P, a key and a query by its own, T by one) and rounded to fp16: to the sum of two, 22
// bits of significand, wherever it goes on into the state, and to one, 11 bits, where it goes to
// the outputs alone, which are bf16. Keys and queries are exact (down to 2^-25 of their
// row's largest). As sums of two bf16, 16 bits, states were off by some 1e-5; so it is that
// of fp32's own sums.
//
// An infinity or a NaN reaches the outputs from its token on and the state, and nothing
// before: factors of a chunk's tokens from a bad key, decay or beta on make R a NaN, and a
// lane sets its R to 0 from the first that is not finite, and its outputs and state to NaN.
//
// Few long sequences leave SMs idle and are cut into segments (segment_chunks): three launches instead of the second.
//
// 8192 tokens of 32 heads of 128 take 394 us: the first kernel, 138 in one piece, which issues 1.75 of 4 instructions a cycle
// (barriers, shared memory and the serial inversions of 16 rows), a third of it beside the first walks; twice 140 the walks of
// a third of the chunks each; 13 the states between (less where one kernel's end and the next's begin overlap). A
// chunk's turn is some 6300 cycles, two chains of a product, its way to registers, a column's largest element, the split
// and its way back. 24 prompts of up to 1500 tokens, 8 heads of 64: 165 us, 100 and 70 of them. The bytes are 31 and
// 13 us' worth.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "hc_attn.cuh"
#include "hc_delta_plan.h"
#include "hc_prompt.h"
#include "hc_tc.h"
#include "umma.cuh"

namespace tshc {

namespace {

constexpr unsigned kStatusInvalidArg = 1u;   // TS_ERR_INVALID_ARG of ts_hc.h
constexpr int kTile = kChunk * 128;           // bytes of a 64 x 64 fp16 tile: 64 rows of 128 bytes, swizzled
struct Factors {
    float c[kChunk];          // -e^(G_i) r_i, r with the key's power of two
    float w[kChunk];          // r_j e^(G_64 - G_j), by a power of two so that the largest is in [1, 2)
    float y[kChunk];          // e^(G_i) s_i, s with the query's power of two
    float p[kChunk];          // what undoes the powers of two of P's rows
    float keep;               // e^(G_64)
    float t, w_undo;          // what undoes T's power of two, and w's
};
constexpr int kFactorBytes = 1040;
static_assert(sizeof(Factors) <= kFactorBytes && kFactorBytes % 16 == 0, "a record's factors");
// What the first kernel leaves: of a chunk and key head, keys, the chunk's keys with the one's before (M, two parts),
// queries; of a chunk and value head, T's two parts, P, the factors.
template <int D>
struct Record {
    static constexpr int kRows = kChunk * D * 2;  // bytes of a chunk's keys, queries or values
    static constexpr int kK = 0, kM = kRows, kQ = kRows + 2 * kTile, kKeyBytes = 2 * kRows + 2 * kTile;
    static constexpr int kT = 0, kP = 2 * kTile, kFactors = 3 * kTile, kValueBytes = 3 * kTile + kFactorBytes;
};
constexpr float kNoDecay = -120.f;            // e^-120 is 0 in fp32; sums of -infinities would be no numbers
constexpr float kNaN = __builtin_nanf("");

// Records lie by head, and within one by the sequence's first token / 64, plus the sequence, plus the chunk:
// no two sequences' overlap, and nobody needs a sum over the sequences before.
__host__ __device__ inline long record_slots(int N, int S) { return (long)N / kChunk + S; }
__device__ __forceinline__ long record_of(int start, int seq, int chunk) { return (long)(start / kChunk) + seq + chunk; }

// Whose part of the first kernel a launch does.
enum { kAllSegments, kFirstSegments, kLastSegments };
__device__ __forceinline__ long segment_of(const DeltaPromptParams &p, int seq)
{
    return (long)(min(max(p.starts[seq], 0), p.N) / kChunk / p.seg) + seq;  // (one that is out of range keeps its state)
}

constexpr size_t kBegunBytes = 16;            // a word behind the ends

size_t records_bytes(int N, int S, int Hk, int Hv, int D)
{
    const size_t slots = record_slots(N, S);
    return D == 64 ? slots * ((size_t)Hk * Record<64>::kKeyBytes + (size_t)Hv * Record<64>::kValueBytes)
                   : slots * ((size_t)Hk * Record<128>::kKeyBytes + (size_t)Hv * Record<128>::kValueBytes);
}

// The last sequence that `of` has at or before the slot.
template <typename Of>
__device__ __forceinline__ int sequence_at(int S, long slot, Of of)
{
    int lo = 0;
    for (int hi = S - 1; lo < hi;) {
        const int mid = (lo + hi + 1) / 2;
        if (of(mid) <= slot)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}
template <int D>
__device__ __forceinline__ uint8_t *key_record(const DeltaPromptParams &p, int hk, long slot)
{
    return p.work + ((size_t)hk * record_slots(p.N, p.S) + slot) * Record<D>::kKeyBytes;
}
template <int D>
__device__ __forceinline__ uint8_t *value_record(const DeltaPromptParams &p, int h, long slot)
{
    const size_t slots = record_slots(p.N, p.S);
    return p.work + (size_t)p.Hk * slots * Record<D>::kKeyBytes + ((size_t)h * slots + slot) * Record<D>::kValueBytes;
}

// The power of two that brings values of up to `most` (bits of a float) to less than 2^14, and what undoes it: fp16
// holds 2^-24 of them, and what is left of the first of two parts 2^-38.
struct Scale {
    float by, undo;
    __device__ __forceinline__ explicit Scale(uint32_t most)
    {
        const uint32_t e = min(267u - (most >> 23), 253u);
        by = __uint_as_float(e << 23);
        undo = __uint_as_float((254u - e) << 23);
    }
};

// Eight values times `by` (a pair of factors for each pair of them) as two fp16 each. In the order written: one pair
// after the other, as a compiler short of registers has it, it is a chain of some 30 cycles a pair.
__device__ __forceinline__ void split8(const uint64_t v0, const uint64_t v1, const uint64_t v2, const uint64_t v3, const uint64_t by, uint32_t *hi,
                                       uint32_t *lo)
{
    asm volatile(
        "{\n\t.reg .b64 t0, t1, t2, t3;\n\t.reg .f32 a0, a1, a2, a3, z0, z1, z2, z3;\n\t.reg .b32 m0, m1, m2, m3;\n\t"
        ".reg .b16 l0, l1, l2, l3, h0, h1, h2, h3;\n\t"
        "mul.rn.f32x2 t0, %8, %12;\n\tmul.rn.f32x2 t1, %9, %12;\n\tmul.rn.f32x2 t2, %10, %12;\n\tmul.rn.f32x2 t3, %11, %12;\n\t"
        "mov.b64 {a0, z0}, t0;\n\tmov.b64 {a1, z1}, t1;\n\tmov.b64 {a2, z2}, t2;\n\tmov.b64 {a3, z3}, t3;\n\t"
        "cvt.rn.f16x2.f32 %0, z0, a0;\n\tcvt.rn.f16x2.f32 %1, z1, a1;\n\tcvt.rn.f16x2.f32 %2, z2, a2;\n\tcvt.rn.f16x2.f32 %3, z3, a3;\n\t"
        "xor.b32 m0, %0, 0x80008000;\n\txor.b32 m1, %1, 0x80008000;\n\txor.b32 m2, %2, 0x80008000;\n\txor.b32 m3, %3, 0x80008000;\n\t"
        "mov.b32 {l0, h0}, m0;\n\tmov.b32 {l1, h1}, m1;\n\tmov.b32 {l2, h2}, m2;\n\tmov.b32 {l3, h3}, m3;\n\t"
        "add.f32.f16 a0, l0, a0;\n\tadd.f32.f16 a1, l1, a1;\n\tadd.f32.f16 a2, l2, a2;\n\tadd.f32.f16 a3, l3, a3;\n\t"
        "add.f32.f16 z0, h0, z0;\n\tadd.f32.f16 z1, h1, z1;\n\tadd.f32.f16 z2, h2, z2;\n\tadd.f32.f16 z3, h3, z3;\n\t"
        "cvt.rn.f16x2.f32 %4, z0, a0;\n\tcvt.rn.f16x2.f32 %5, z1, a1;\n\tcvt.rn.f16x2.f32 %6, z2, a2;\n\tcvt.rn.f16x2.f32 %7, z3, a3;\n\t}"
        : "=&r"(hi[0]), "=&r"(hi[1]), "=&r"(hi[2]), "=&r"(hi[3]), "=&r"(lo[0]), "=&r"(lo[1]), "=&r"(lo[2]), "=&r"(lo[3])
        : "l"(v0), "l"(v1), "l"(v2), "l"(v3), "l"(by));
}

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

// ------------------------------------------------------------------ keys and queries, T, P and the factors

__device__ __forceinline__ uint32_t load_acquire(const unsigned *at)
{
    uint32_t x;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(x) : "l"(at) : "memory");
    return x;
}
__device__ __forceinline__ void store_release(unsigned *at, uint32_t x)
{
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(at), "r"(x) : "memory");
}

constexpr int kPrepThreads = 256;
constexpr int kPitch = 68;    // floats of a row of a 64 x 64 matrix in shared memory
constexpr int kGates = 4;     // value heads whose gates are added up at once, a warp each

template <int D>
struct PrepShared {
    uint16_t k[kChunk][D + 8];                     // fp16
    union {                                        // one after the other
        uint16_t q[kChunk][D + 8];
        alignas(16) float t[kChunk][kPitch];       // T
    };
    union {
        uint16_t before[kChunk][D + 8];            // the keys of the chunk before
        alignas(16) float a[kChunk][kPitch];       // M, then A, and right of its first 32 columns an intermediate product
    };
    alignas(16) float r[kChunk], s[kChunk];        // the inverse norms, with the powers of two
    struct alignas(16) {
        float gh[kChunk], gl[kChunk], beta[kChunk];  // G in two parts
        int bad;                                   // the first token with an infinity or a NaN
        uint32_t most_t;
    } gate[kGates];                                // of some value heads
    int bad_key;                                   // the first key with one
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], const void *at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(smem_addr(at)) : "memory");
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 rows of x (from `row`) with 8 kCols rows of y (from `col`).
template <int D, int kCols>
__device__ __forceinline__ void rows_with_rows(const uint16_t (*x)[D + 8], int row, const uint16_t (*y)[D + 8], int col, float (&d)[kCols][4])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kCols; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c)
            d[i][c] = 0.f;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
        uint32_t a[4];
        ldmatrix4(a, &x[row + (lane & 15)][s * 16 + (lane >> 4) * 8]);
#pragma unroll
        for (int i = 0; i < kCols / 2; ++i) {  // 16 columns: two tiles' two halves of the sum's 16 terms
            uint32_t b[4];
            ldmatrix4(b, &y[col + i * 16 + (lane >> 4) * 8 + (lane & 7)][s * 16 + ((lane >> 3) & 1) * 8]);
            mma16816(d[2 * i], a, b[0], b[1]);
            mma16816(d[2 * i + 1], a, b[2], b[3]);
        }
    }
}

__device__ __forceinline__ int piece_at(int row, int x) { return row * 128 + ((x ^ (row & 7)) << 4); }

// Eight values as two fp16 each, to piece x of row i of two tiles.
__device__ __forceinline__ void put8(uint8_t *hi, uint8_t *lo, int i, int x, const float (&v)[8])
{
    uint32_t h[4], l[4];
    split8(f32x2(v[0], v[1]), f32x2(v[2], v[3]), f32x2(v[4], v[5]), f32x2(v[6], v[7]), f32x2(1.f, 1.f), h, l);
    *reinterpret_cast<uint4 *>(hi + piece_at(i, x)) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4 *>(lo + piece_at(i, x)) = make_uint4(l[0], l[1], l[2], l[3]);
}

// Eight elements of a row, a piece, of the D / 8 lanes that share it: scaled by a power of two so that the row's largest
// is in [1, 2), as fp16, over them. Returns the row's sum of squares (before); `undo`: the power of two back, 0 for a row of
// zeros (and of what is below bf16's range): times the inverse of its norm, an epsilon's, it would be far above the others',
// whose w it shares a scale with.
template <int D>
__device__ __forceinline__ float row_to_half(uint4 &w, float &undo, bool &odd)
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        sum = fmaf(bf16_lo(u[c]), bf16_lo(u[c]), sum);
        sum = fmaf(bf16_hi(u[c]), bf16_hi(u[c]), sum);
    }
    // exponents, whose order is that of 16-bit integers, two at a time
    uint32_t tops = __vmaxu2(__vmaxu2(u[0] & 0x7F807F80u, u[1] & 0x7F807F80u), __vmaxu2(u[2] & 0x7F807F80u, u[3] & 0x7F807F80u));
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        tops = __vmaxu2(tops, __shfl_xor_sync(0xFFFFFFFFu, tops, o));
    }
    const uint32_t most = max(tops << 16, tops & 0xFFFF0000u);
    odd = most == 0x7F800000u;
    const uint32_t e = min(most >> 23, 253u);
    const float by = e == 0 || odd ? 1.f : __uint_as_float((254u - e) << 23);
    undo = odd ? 1.f : __uint_as_float(e << 23);
    w = make_uint4(pack2_f16(bf16_lo(u[0]) * by, bf16_hi(u[0]) * by), pack2_f16(bf16_lo(u[1]) * by, bf16_hi(u[1]) * by),
                   pack2_f16(bf16_lo(u[2]) * by, bf16_hi(u[2]) * by), pack2_f16(bf16_lo(u[3]) * by, bf16_hi(u[3]) * by));
    return sum;
}

// A block a chunk and key head, with the key head's value heads one after the other. (A block a value head, which does
// the keys' part again for each, took a quarter longer. Four blocks a SM, in 64 registers, for D = 128, too: 8192 tokens of 32
// heads in 419 us, with three, in 80, 426; but 2048 of 8 heads 101 and 94, where the blocks are few. 52 bytes are spilled.)
template <int D>
__global__ void __launch_bounds__(kPrepThreads, 4) hc_delta_prep_kernel(const DeltaPromptParams p)
{
    using Rec = Record<D>;
    extern __shared__ uint4 smem4[];
    auto &sh = *reinterpret_cast<PrepShared<D> *>(smem4);
    pdl_launch_dependents();
    // The last segments' blocks run beside the first walks and do not wait for their end, but for one, after which the next
    // kernel is after the walks. What was written before the call they may read because a walk's thread that had waited for it
    // released `begun` before these blocks could be launched, and each of their threads acquires it; one that does not find
    // it waits for the walks as any kernel does.
    if (p.part != kLastSegments || blockIdx.x == 0 || load_acquire(p.begun) != 1u)
        pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (p.part == kFirstSegments && blockIdx.x == 0 && tid == 0)
        *p.begun = 0;
    const long slot = blockIdx.x / p.Hk;
    const int hk = (int)(blockIdx.x - slot * p.Hk), group = p.Hv / p.Hk;
    // the sequence whose records this one is among: the last that begins at or before it
    const int seq = sequence_at(p.S, slot, [&](int i) { return record_of(p.starts[i], i, 0); });
    int first, len;
    if (!rows_of(p, seq, first, len))
        return;
    const long chunk = slot - record_of(first, seq, 0);
    if (chunk < 0 || chunk * kChunk >= len)
        return;
    if (p.part != kAllSegments) {
        const long last = (((long)len + kChunk - 1) / kChunk - 1) / p.seg;
        if ((last > 0 && chunk / p.seg == last) != (p.part == kLastSegments))
            return;
    }
    first += (int)chunk * kChunk;
    const int n = min(kChunk, len - (int)chunk * kChunk);
    uint8_t *const key_rec = key_record<D>(p, hk, slot);
    // the gates are asked for first, by the warps that add them up: a value head a warp, some at a time
    float decay[2] = {0.f, 0.f}, beta[2] = {0.f, 0.f};
    const auto ask = [&](int g) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const bool in = warp < kGates && g < group && 2 * lane + i < n;
            const size_t at = (size_t)(first + 2 * lane + i) * p.Hv + hk * group + g;
            decay[i] = in ? p.decay[at] : 0.f;
            beta[i] = in ? p.beta[at] : 0.f;
        }
    };
    ask(warp);
    if (tid == 0)
        sh.bad_key = n;
    __syncthreads();

    // keys and queries, zeros after the last token, and their norms
    constexpr int kPieces = D / 8, kRowsAtOnce = kPrepThreads / kPieces;
    const int piece = tid % kPieces, row0 = tid / kPieces;
    const uint16_t *const k_row = p.k + (size_t)hk * D + piece * 8, *const q_row = p.q + (size_t)hk * D + piece * 8;
    uint8_t *const key_to = key_rec + (piece >> 3) * kTile;
    if (chunk > 0)                                  // (which is whole)
#pragma unroll
        for (int i = 0; i < kChunk / kRowsAtOnce; ++i) {
            const int r = row0 + i * kRowsAtOnce;
            uint4 w = *reinterpret_cast<const uint4 *>(k_row + (first - kChunk + r) * p.k_stride);
            float undo;
            bool odd;
            row_to_half<D>(w, undo, odd);
            *reinterpret_cast<uint4 *>(&sh.before[r][piece * 8]) = w;
        }
#pragma unroll
    for (int i = 0; i < 2 * kChunk / kRowsAtOnce; ++i) {
        const bool query = i >= kChunk / kRowsAtOnce;
        const int r = row0 + (i - (query ? kChunk / kRowsAtOnce : 0)) * kRowsAtOnce;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (r < n)
            w = *reinterpret_cast<const uint4 *>(query ? q_row + (first + r) * p.q_stride : k_row + (first + r) * p.k_stride);
        float undo;
        bool odd;
        const float sum = row_to_half<D>(w, undo, odd);
        *reinterpret_cast<uint4 *>(query ? &sh.q[r][piece * 8] : &sh.k[r][piece * 8]) = w;
        *reinterpret_cast<uint4 *>(key_to + (query ? Rec::kQ : Rec::kK) + piece_at(r, piece & 7)) = w;
        if (piece == 0) {
            const float inv = (p.norm_eps >= 0.f ? 1.f / sqrtf(sum + p.norm_eps) : 1.f) * undo;
            if (query) {
                sh.s[r] = inv * p.scale;
            } else {
                sh.r[r] = inv;
                if (odd || !(inv < INFINITY))
                    atomicMin(&sh.bad_key, r);
            }
        }
    }
    __syncthreads();

    // the decays' sums in 64 bits, kept as two floats: differences of near ones are right after strong decays too
    const auto gates = [&](int g) {
        if (warp >= kGates || g >= group)
            return;
        auto &gate = sh.gate[warp];
        int bad = sh.bad_key;
        double x[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (!(decay[i] < INFINITY) || !(fabsf(beta[i]) < INFINITY))
                bad = min(bad, 2 * lane + i);
            x[i] = fmaxf(decay[i], kNoDecay);
        }
        bad = __reduce_min_sync(0xFFFFFFFFu, bad);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (2 * lane + i >= bad) {
                x[i] = 0.0;
                beta[i] = 0.f;
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
        auto &f = *reinterpret_cast<Factors *>(value_record<D>(p, hk * group + g, slot) + Rec::kFactors);
        float w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 2 * lane + i;
            const double G = before + x[i];
            gate.gh[r] = (float)G;
            gate.gl[r] = (float)(G - (float)G);
            gate.beta[r] = beta[i];
            const float e = expf((float)G);
            f.c[r] = r < bad ? -e * sh.r[r] : r < n ? kNaN : 0.f;
            w[i] = r < bad ? expf((float)(all - G)) * sh.r[r] : 0.f;
            f.y[r] = e * sh.s[r];
        }
        const uint32_t top = min(max(__reduce_max_sync(0xFFFFFFFFu, max(__float_as_uint(w[0]), __float_as_uint(w[1]))) >> 23, 1u), 253u);
        const float w_by = __uint_as_float((254u - top) << 23);
        *reinterpret_cast<float2 *>(&f.w[2 * lane]) = make_float2(w[0] * w_by, w[1] * w_by);
        if (lane == 0) {
            f.keep = expf((float)all);
            f.w_undo = __uint_as_float(top << 23);
            gate.bad = bad;
            gate.most_t = 0;
        }
    };
    gates(warp);
    const int row = (warp & 3) * 16 + (lane >> 2);
    if (chunk > 0) {                                // M: the keys with those of the chunk before
        const int col = (warp >> 2) * 32;
        float m[4][4];
        rows_with_rows<D, 4>(sh.k, (warp & 3) * 16, sh.before, col, m);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float *at = &sh.a[row][col + i * 8 + (lane & 3) * 2];
            *reinterpret_cast<float2 *>(at) = make_float2(m[i][0], m[i][1]);
            *reinterpret_cast<float2 *>(at + 8 * kPitch) = make_float2(m[i][2], m[i][3]);
        }
    }
    // keys with keys (warps 0-3) and queries with keys (4-7), 16 rows a warp, in registers
    float d[8][4];                                 // of rows row and row + 8: columns 8 i + 2 (lane % 4) and the next
    rows_with_rows<D, 8>(warp >= 4 ? sh.q : sh.k, (warp & 3) * 16, sh.k, 0, d);
    __syncthreads();
    if (chunk > 0) {
        const int i = tid >> 2, x = (tid & 3) * 2;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const float4 u = *reinterpret_cast<const float4 *>(&sh.a[i][(x + c) * 8]), w = *reinterpret_cast<const float4 *>(&sh.a[i][(x + c) * 8 + 4]);
            const float v[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
            put8(key_rec + Rec::kM, key_rec + Rec::kM + kTile, i, x + c, v);
        }
        __syncthreads();
    }
    // T's blocks above the diagonal stay 0
    for (int u = tid; u < kChunk * kChunk / 4; u += kPrepThreads)
        if ((u & 15) >> 2 > u >> 8)
            *reinterpret_cast<float4 *>(&sh.t[u >> 4][(u & 15) * 4]) = make_float4(0.f, 0.f, 0.f, 0.f);

    // A row of P is by the power of two that its products without decays, which are 1 at most, call for: all value heads'.
    const int cut = (warp & 3) * 2 + 1;                // the last eight columns that a row of the warp's can see
    float p_by[2] = {1.f, 1.f}, p_undo[2] = {1.f, 1.f};
    if (warp >= 4) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t most = 0;
#pragma unroll
            for (int t = 0; t < 8; ++t)
                if (t <= cut) {
                    const float2 jr = *reinterpret_cast<const float2 *>(&sh.r[8 * t + 2 * (lane & 3)]);
                            const float a = fabsf(d[t][2 * half] * jr.x), z = fabsf(d[t][2 * half + 1] * jr.y);
                    most = max(most, max(8 * t + 2 * (lane & 3) <= row + 8 * half ? __float_as_uint(a) : 0u,
                                         8 * t + 2 * (lane & 3) + 1 <= row + 8 * half ? __float_as_uint(z) : 0u));
                }
            most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
            most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
            const Scale sp(__float_as_uint(fabsf(__uint_as_float(most) * sh.s[row + 8 * half])));
            p_by[half] = sp.by;
            p_undo[half] = sp.undo;
        }
    }
#pragma unroll 1
    for (int g = 0; g < group; ++g) {
        if (g > 0) {
            __syncthreads();                           // T has been read
            if (g % kGates == 0) {
                ask(g + warp);
                gates(g + warp);
                __syncthreads();
            }
        }
        // A, to shared memory, and P, a row by a power of two of its own
        const auto &gate = sh.gate[g % kGates];
        const int bad = gate.bad;
        uint8_t *const rec = value_record<D>(p, hk * group + g, slot);
        {
            float gh[2], gl[2], by[2];                     // of rows row and row + 8, as d
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int i = row + 8 * half;
                gh[half] = gate.gh[i];
                gl[half] = gate.gl[i];
                by[half] = warp < 4 ? gate.beta[i] * sh.r[i] : sh.s[i];
            }
            const int above = row + (warp < 4 ? 0 : 1);    // row's first column that is 0, of a row before `bad`
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                float e[4] = {0.f, 0.f, 0.f, 0.f};
                const int j = 8 * t + 2 * (lane & 3);
                if (t <= cut) {
                    const float2 jh = *reinterpret_cast<const float2 *>(&gate.gh[j]), jl = *reinterpret_cast<const float2 *>(&gate.gl[j]);
                    const float2 jr = *reinterpret_cast<const float2 *>(&sh.r[j]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int half = c >> 1;
                        // (the exponential's error, |x| 2^-24 of it or so, is at most 2^-25 of 1)
                        const float g = (gh[half] - (c & 1 ? jh.y : jh.x)) + (gl[half] - (c & 1 ? jl.y : jl.x));
                        const float x = d[t][c] * (c & 1 ? jr.y : jr.x) * by[half] * __expf(g);
                        e[c] = j + (c & 1) < above + 8 * half && row + 8 * half < bad ? x : 0.f;
                    }
                }
                if (warp >= 4) {
#pragma unroll
                    for (int half = 0; half < 2; ++half)
                        *reinterpret_cast<uint32_t *>(rec + Rec::kP + piece_at(row + 8 * half, t) + (lane & 3) * 4) =
                            pack2_f16(e[2 * half] * p_by[half], e[2 * half + 1] * p_by[half]);
                } else if (t <= cut) {
                    *reinterpret_cast<float2 *>(&sh.a[row][j]) = make_float2(e[0], e[1]);
                    *reinterpret_cast<float2 *>(&sh.a[row + 8][j]) = make_float2(e[2], e[3]);
                }
            }
            if (warp >= 4 && (lane & 3) == 0)
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    reinterpret_cast<Factors *>(rec + Rec::kFactors)->p[row + 8 * half] = p_undo[half];
        }
        __syncthreads();
        // T = (I + A)^-1: the blocks of 16 on the diagonal, a thread a column; the blocks above them are 0
        if (tid < kChunk) {
            const int b = tid & 48, j = tid & 15;
            float t[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < i; k += 4) {
                    const float4 a = *reinterpret_cast<const float4 *>(&sh.a[b + i][b + k]);  // (beyond the diagonal: 0)
                    sum[0] = fmaf(a.x, t[k], sum[0]);
                    if (k + 1 < i)
                        sum[1] = fmaf(a.y, t[k + 1], sum[1]);
                    if (k + 2 < i)
                        sum[2] = fmaf(a.z, t[k + 2], sum[2]);
                    if (k + 3 < i)
                        sum[3] = fmaf(a.w, t[k + 3], sum[3]);
                }
                t[i] = i < j ? 0.f : i == j ? 1.f : -((sum[0] + sum[1]) + (sum[2] + sum[3]));
                sh.t[b + i][b + j] = t[i];
            }
        }
        __syncthreads();
        // (T11 0; T21 T22) has T21 = -T22 A21 T11: two pairs of blocks of 16, then one of 32
        {
            const int pair = tid >> 7, i = (tid >> 3) & 15, j = (tid & 7) * 2, b = pair * 32;
            const auto sixteen = [&](const float *x, const float *y, int pitch) {  // a row's products with two columns
                float s0 = 0.f, s1 = 0.f;
#pragma unroll
                for (int k = 0; k < 16; k += 4) {
                    const float4 a = *reinterpret_cast<const float4 *>(x + k);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float2 t = *reinterpret_cast<const float2 *>(y + (k + c) * pitch);
                        const float f = c == 0 ? a.x : c == 1 ? a.y : c == 2 ? a.z : a.w;
                        s0 = fmaf(f, t.x, s0);
                        s1 = fmaf(f, t.y, s1);
                    }
                }
                return make_float2(s0, s1);
            };
            *reinterpret_cast<float2 *>(&sh.a[pair * 16 + i][32 + j]) = sixteen(&sh.a[b + 16 + i][b], &sh.t[b][b + j], kPitch);
            __syncthreads();
            const float2 s = sixteen(&sh.t[b + 16 + i][b + 16], &sh.a[pair * 16][32 + j], kPitch);
            *reinterpret_cast<float2 *>(&sh.t[b + 16 + i][b + j]) = make_float2(-s.x, -s.y);
            __syncthreads();
        }
        {
            // four terms of a row's sums for four columns
            const auto four = [&](float4 &s, const float *x, const float *y, int pitch) {
                const float4 a = *reinterpret_cast<const float4 *>(x);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float4 t = *reinterpret_cast<const float4 *>(y + c * pitch);
                    const float f = c == 0 ? a.x : c == 1 ? a.y : c == 2 ? a.z : a.w;
                    s = make_float4(fmaf(f, t.x, s.x), fmaf(f, t.y, s.y), fmaf(f, t.z, s.z), fmaf(f, t.w, s.w));
                }
            };
            // A21 T11, a warp four columns: T11's rows before the columns' are 0
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
            for (int k = warp * 4; k < 32; k += 4)
                four(s, &sh.a[32 + lane][k], &sh.t[k][warp * 4], kPitch);
            *reinterpret_cast<float4 *>(&sh.a[lane][32 + warp * 4]) = s;
            __syncthreads();
            // T22 times that, a warp four rows: T22's columns after the rows' are 0
            const int i = tid >> 3, j = (tid & 7) * 4;
            s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
            for (int k = 0; k <= warp * 4; k += 4)
                four(s, &sh.t[32 + i][32 + k], &sh.a[k][32 + j], kPitch);
            *reinterpret_cast<float4 *>(&sh.t[32 + i][j]) = make_float4(-s.x, -s.y, -s.z, -s.w);
            __syncthreads();
        }
        float tv[2][8];
        {
            const int i = tid >> 2, x = (tid & 3) * 2;
            uint32_t most = 0;
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int d = 0; d < 8; d += 4) {
                    const int j = (x + c) * 8 + d;
                    const float4 t = *reinterpret_cast<const float4 *>(&sh.t[i][j]), b = *reinterpret_cast<const float4 *>(&gate.beta[j]);
                    tv[c][d] = t.x * b.x;
                    tv[c][d + 1] = t.y * b.y;
                    tv[c][d + 2] = t.z * b.z;
                    tv[c][d + 3] = t.w * b.w;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        most = max(most, __float_as_uint(tv[c][d + e]) & 0x7FFFFFFFu);
                }
            most = __reduce_max_sync(0xFFFFFFFFu, most);
            if (lane == 0)
                atomicMax(&sh.gate[g % kGates].most_t, most);
            __syncthreads();
            const Scale st(sh.gate[g % kGates].most_t);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int d = 0; d < 8; ++d)
                    tv[c][d] *= st.by;
                put8(rec + Rec::kT, rec + Rec::kT + kTile, i, x + c, tv[c]);
            }
            if (tid == 0)
                reinterpret_cast<Factors *>(rec + Rec::kFactors)->t = st.undo;
        }
    }
}

// ------------------------------------------------------------------ the walk over the chunks

// Four threads a column (in warps w, w + 4, ..), which have 16 tokens of a chunk and a quarter of the state each and do all of
// its work; then the products, the copies, two idle warps. (Two threads a column took 6100 cycles a chunk. The chain's, the
// state's and the outputs' work in threads of their own ran side by side, but their code, some 50 KB, did not fit the
// instruction cache: 7000.)
constexpr int kColumnThreads = 512, kThreads = kColumnThreads + 128;
constexpr int kMmaWarp = 16, kLoadWarp = 17;
constexpr int kColumnRegs = 104, kOtherRegs = 64;  // 512 * 104 + 128 * 64 = 61440 = 640 * 96, what the launch has
constexpr uint32_t kTmemCols = 512;
// TMEM columns: the state's two parts; S0^T K'^T, then the second half of the state's update; M's product, then R's two
// parts; T's product, then w U's two parts; the outputs' two; the first half of the state's update, then U.
constexpr uint32_t kS = 0, kXA = 128, kXB = 192, kU = 256, kY = 320, kZ = 384, kDS = 448;

// Shared memory: what is used from one chunk into the next, three of them; the rest twice.
template <int D>
struct Plan {
    using Rec = Record<D>;
    static constexpr int kA = 3, kB = 2, kC = 2, kF = 4;                   // places of (K, M), (T, V), (Q, P), factors
    static constexpr int kABytes = Rec::kRows + 2 * kTile, kBBytes = 2 * kTile + Rec::kRows, kCBytes = Rec::kRows + kTile;
    static constexpr int kAt = 0, kBt = kA * kABytes, kCt = kBt + kB * kBBytes, kFt = kCt + kC * kCBytes;
    static constexpr int kTotal = kFt + kF * kFactorBytes + 1024;                   // and alignment
};

struct Shared {
    uint64_t a_full[3], a_empty[3], b_full[2], b_empty[2], c_full[2], c_empty[2], f_full[4];
    uint64_t s_ready, r_ready, w_ready, y_free;             // of the columns' threads
    uint64_t x_done, u_done, da_done, db_done, o_done;      // of the products
    uint32_t tmem;
    int dead;
    // What a column's threads tell one another: its first token that is not finite (by chunks in turn), largest elements.
    int bad[2][4][128];
    float top_r[4][128], top_u[4][128], top_s[4][128];
};

// Waits for the phase; false when it, or another wait of the block, ran out (recorded at the end). Short: what the loop over
// the chunks has to stay within is the instruction cache.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, Shared &sh)
{
    bool there = mbar_try_wait(bar, parity);
    if (!there) {
        const uint64_t t0 = global_timer_ns();
        do {
            there = mbar_try_wait(bar, parity);
        } while (!there && !*reinterpret_cast<volatile int *>(&sh.dead) && global_timer_ns() - t0 < kWaitLimitNs);
        if (!there)
            *reinterpret_cast<volatile int *>(&sh.dead) = 1;
    }
    return __all_sync(0xFFFFFFFFu, there);
}

template <int N>
__device__ __forceinline__ uint64_t pair_of(const uint32_t (&x)[N], int c) { return f32x2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])); }
constexpr uint64_t kMinusZeros = 0x8000000080000000ull;
__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) { return ffma2(a, b, kMinusZeros); }
// The larger of |a|, |b| and |c|: a NaN if one of them is.
__device__ __forceinline__ float most3(float a, float b, float c)
{
    float y;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
__device__ __forceinline__ float most_of(float most, uint64_t v)
{
    float a, z;
    f32x2_unpack(v, a, z);
    return most3(most, a, z);
}

// The n-th longest of up to 32 sequences, so that long walks begin first: 24 prompts of up to 1500 tokens, 8 heads
// of 64, 192 walks on 152 SMs, take 165 us; in their own order 177.
__device__ __forceinline__ int longest(const DeltaPromptParams &p, int n)
{
    const int lane = threadIdx.x & 31, len = lane < p.S ? p.starts[lane + 1] - p.starts[lane] : -1;
    int before = 0;
    for (int i = 0; i < p.S; ++i) {
        const int other = __shfl_sync(0xFFFFFFFFu, len, i);
        before += other > len || (other == len && i < lane);
    }
    return __ffs(__ballot_sync(0xFFFFFFFFu, lane < p.S && before == n)) - 1;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) hc_delta_scan_kernel(const __grid_constant__ DeltaPromptParams p, const __grid_constant__ CUtensorMap map_v)
{
    using P = Plan<D>;
    using Rec = Record<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Shared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t *const smem = smem_raw + (base - smem_addr(smem_raw));
    if (tid == 0) {
        for (int i = 0; i < 3; ++i) {
            mbar_init(&sh.a_full[i], 1);
            mbar_init(&sh.a_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.b_full[i], 1);
            mbar_init(&sh.b_empty[i], 1 + kColumnThreads / 32);
            mbar_init(&sh.c_full[i], 1);
            mbar_init(&sh.c_empty[i], 1);
        }
        for (int i = 0; i < 4; ++i)
            mbar_init(&sh.f_full[i], 1);
        mbar_init(&sh.s_ready, kColumnThreads);
        mbar_init(&sh.y_free, kColumnThreads);
        mbar_init(&sh.r_ready, kColumnThreads);
        mbar_init(&sh.w_ready, kColumnThreads);
        mbar_init(&sh.x_done, 1);
        mbar_init(&sh.u_done, 1);
        mbar_init(&sh.da_done, 1);
        mbar_init(&sh.db_done, 1);
        mbar_init(&sh.o_done, 1);
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
    // What is launched to run beside the walks relies on what they have waited for (hc_delta_prep_kernel).
    if (p.part == kAllSegments)
        pdl_launch_dependents();
    pdl_wait();
    if (p.part != kAllSegments) {
        if (blockIdx.x == 0) {
            if (tid == 0)
                store_release(p.begun, 1u);
            __syncthreads();
        }
        pdl_launch_dependents();
    }
    const int h = blockIdx.x % p.Hv, hk = h / (p.Hv / p.Hk);
    int seq = blockIdx.x / p.Hv, first, len;
    // where the state comes from and goes to; of a walk without values from the identity: its column's 1
    const float *from = nullptr;
    float *to = nullptr;
    bool with_values = true, with_outputs = true;
    long record = 0;
    if (p.seg == 0) {
        if (p.S <= 32)
            seq = longest(p, seq);
        if (!rows_of(p, seq, first, len))
            len = 0;
        record = record_of(first, seq, 0);
        from = p.state_in + ((size_t)seq * p.Hv + h) * D * D;
        to = len > 0 || p.state_out != p.state_in ? p.state_out + ((size_t)seq * p.Hv + h) * D * D : nullptr;
    } else {
        const long slots = segment_slots(p.N, p.S, p.seg);
        long slot = seq;
        with_values = slot < slots;
        slot -= with_values ? 0 : slots;
        seq = sequence_at(p.S, slot, [&](int i) { return segment_of(p, i); });
        if (!rows_of(p, seq, first, len))
            len = 0;
        const long at = slot - segment_of(p, seq), last = max(((long)len + kChunk - 1) / kChunk - 1, 0l) / p.seg;
        const auto end_of = [&](long slot, bool values) { return p.ends + (((values ? 0 : slots) + slot) * p.Hv + h) * D * D; };
        const Walk w = walk_of(at, last, with_values, p.again);
        if (w.mine) {
            from = w.from == kState ? p.state_in + ((size_t)seq * p.Hv + h) * D * D : w.from == kEndBefore ? end_of(slot - 1, true) : nullptr;
            to = w.to == kState ? p.state_out + ((size_t)seq * p.Hv + h) * D * D : w.to == kEnd ? end_of(slot, with_values) : nullptr;
            if (len == 0 && p.state_out == p.state_in)
                to = nullptr;
            with_outputs = w.outputs;
        }
        record = record_of(first, seq, 0) + at * p.seg;
        first += (int)(at * p.seg) * kChunk;
        len = w.mine ? (int)min((long)len - at * p.seg * kChunk, (long)p.seg * kChunk) : 0;
    }
    const int chunks = (len + kChunk - 1) / kChunk;
    const int col = tid & 127;                      // of the threads that have one
    const bool there = col < D;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const auto factors = [&](int ch) -> const Factors & { return *reinterpret_cast<const Factors *>(smem + P::kFt + (ch % P::kF) * kFactorBytes); };

    // (In the columns' threads a wait that ran out ends nothing: they go on through the same barriers, on
    // whatever lies there, and every further wait returns at once.)
    if (warp < kMmaWarp) {
        // ---------------------------------------------------------- the columns
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kColumnRegs));
        const int part = warp >> 2, t0 = part * 16;
        const auto meet = [&] { asm volatile("bar.sync %0, 128;" ::"r"(1 + (warp & 3)) : "memory"); };  // the four warps of these columns
        const auto most_of_all = [&](const float (&top)[4][128]) {  // after they met
            return most3(most3(top[0][col], top[1][col], top[2][col]), top[3][col], 0.f);
        };
        // of each 64 elements of the column a thread has 16
        const size_t step = (size_t)p.Hv * D;
        constexpr int kMine = D / 4;
        uint64_t s[kMine / 2];                      // two elements each
#pragma unroll
        for (int i = 0; i < kMine / 2; ++i) {
            const int d = t0 + (i >> 3) * 64 + (i & 7) * 2;
            s[i] = 0;
            if (from && there)
                s[i] = f32x2(from[d * D + col], from[(d + 1) * D + col]);
            else if (!with_values)
                s[i] = f32x2(d == col, d + 1 == col);
        }
        float keep = 1.f, s_undo, y_by = 0.f, z_by = 0.f, w_undo = 0.f;  // of the chunk before, and what undoes the scales
        int bad = kChunk;                           // of the chunk before
        const auto to_operand = [&] {               // the state, D / 2 columns a part
            float tops[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < kMine / 2; ++i)
                tops[i & 3] = most_of(tops[i & 3], s[i]);
            sh.top_s[part][col] = most3(most3(tops[0], tops[1], tops[2]), tops[3], 0.f);
            meet();
            const Scale sc(__float_as_uint(most_of_all(sh.top_s)));
            s_undo = sc.undo;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kMine / 16; ++i) {
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int c = 0; c < 8; c += 4)
                    split8(s[8 * i + c], s[8 * i + c + 1], s[8 * i + c + 2], s[8 * i + c + 3], f32x2(sc.by, sc.by), hi + c, lo + c);
                tmem_st8_async(lane_base + kS + 32 * i + 8 * part, hi);
                tmem_st8_async(lane_base + kS + D / 2 + 32 * i + 8 * part, lo);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&sh.s_ready);
        };
        // the state after chunk ch
        const auto update = [&](int ch) {
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                wait(j == 0 ? &sh.da_done : &sh.db_done, ch & 1, sh);
                tc_fence_after();
                uint32_t x[16];
                tmem_ld16_async(lane_base + (j == 0 ? kDS : kXA) + t0, x);
                tmem_wait_ld(x);
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    s[8 * j + c] = ffma2(s[8 * j + c], f32x2(keep, keep), fmul2(pair_of(x, c), f32x2(w_undo, w_undo)));
            }
            if (bad < kChunk)
#pragma unroll
                for (int i = 0; i < kMine / 2; ++i)
                    s[i] = f32x2(kNaN, kNaN);
        };
        // chunk ch's outputs
        const auto outputs = [&](int ch) {
            const Factors &f = factors(ch);
            const int n = there ? min(kChunk, len - ch * kChunk) - t0 : 0;
            wait(&sh.o_done, ch & 1, sh);
            tc_fence_after();
            uint16_t *to = p.out + (size_t)(first + ch * kChunk + t0) * step + (size_t)h * D + col;
            const bool plain = __all_sync(0xFFFFFFFFu, n >= 16 && bad == kChunk);
            const uint64_t y2 = f32x2(y_by, y_by), z2 = f32x2(z_by, z_by);
#pragma unroll 1
            for (int i = 0; i < 16; i += 4) {
                uint32_t y[4], z[4];
                __syncwarp();
                tmem_ld4_async(lane_base + kY + t0 + i, y);
                tmem_ld4_async(lane_base + kZ + t0 + i, z);
                const float4 fy = *reinterpret_cast<const float4 *>(&f.y[t0 + i]), fp = *reinterpret_cast<const float4 *>(&f.p[t0 + i]);
                tmem_wait_ld4(y);
                tmem_wait_ld4(z);
                const uint64_t o0 = ffma2(fmul2(f32x2(fy.x, fy.y), y2), pair_of(y, 0), fmul2(fmul2(f32x2(fp.x, fp.y), z2), pair_of(z, 0)));
                const uint64_t o1 = ffma2(fmul2(f32x2(fy.z, fy.w), y2), pair_of(y, 1), fmul2(fmul2(f32x2(fp.z, fp.w), z2), pair_of(z, 1)));
                float o[4];
                f32x2_unpack(o0, o[0], o[1]);
                f32x2_unpack(o1, o[2], o[3]);
                if (plain) {
                    // two tokens a word, then two columns: lanes trade halves, even ones take the tokens 0 and 2, odd ones 1 and 3
                    const uint32_t p0 = pack2_bf16(o[0], o[1]), p1 = pack2_bf16(o[2], o[3]);
                    const uint32_t q0 = __shfl_xor_sync(0xFFFFFFFFu, p0, 1), q1 = __shfl_xor_sync(0xFFFFFFFFu, p1, 1);
                    const uint32_t which = lane & 1 ? 0x3276u : 0x5410u;
                    uint16_t *const at = to + ((lane & 1) ? (long)step - 1 : 0);
                    *reinterpret_cast<uint32_t *>(at) = __byte_perm(p0, q0, which);
                    *reinterpret_cast<uint32_t *>(at + 2 * step) = __byte_perm(p1, q1, which);
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (i + c < n)
                            to[c * step] = __bfloat16_as_ushort(__float2bfloat16_rn(t0 + i + c >= bad ? kNaN : o[c]));
                }
                to += 4 * step;
            }
            tc_fence_before();
            mbar_arrive(&sh.y_free);
        };
        if (chunks > 0)
            to_operand();
#pragma unroll 1
        for (int ch = 0; ch < chunks; ++ch) {
            const int n = there && with_values ? min(kChunk, len - ch * kChunk) - t0 : 0, turn = ch & 1;
            const uint32_t phase = ch & 1;
            // R
            wait(&sh.f_full[ch % P::kF], (ch / P::kF) & 1, sh);
            wait(&sh.b_full[ch % P::kB], (ch / P::kB) & 1, sh);
            const Factors &f = factors(ch);
            const uint16_t *const v = reinterpret_cast<const uint16_t *>(smem + P::kBt + (ch % P::kB) * P::kBBytes + 2 * kTile) + t0 * D + col;
            uint32_t vw[8];                         // two tokens' values
            if (n >= 16) {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    vw[c] = v[2 * c * D] | (uint32_t)v[(2 * c + 1) * D] << 16;
            } else {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    vw[c] = (2 * c < n ? v[2 * c * D] : 0u) | (2 * c + 1 < n ? (uint32_t)v[(2 * c + 1) * D] << 16 : 0u);
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.b_empty[ch % P::kB]);
            wait(&sh.x_done, phase, sh);
            tc_fence_after();
            uint64_t r[8];
            float tops[4] = {0.f, 0.f, 0.f, 0.f};
            {
                uint32_t x[16], z[16];
                tmem_ld16_async(lane_base + kXA + t0, x);
                tmem_ld16_async(lane_base + kXB + t0, z);  // (before the second chunk: whatever lies there)
                // the first part is of the state before the chunk before
                const float xa = s_undo * keep;
                const uint64_t xa2 = f32x2(xa, xa), xb2 = f32x2(w_undo, w_undo);
                tmem_wait_ld(x);
                tmem_wait_ld(z);
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    r[c] = fmul2(pair_of(x, c), xa2);
                if (ch > 0)
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        r[c] = ffma2(pair_of(z, c), xb2, r[c]);
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float2 k = *reinterpret_cast<const float2 *>(&f.c[t0 + 2 * c]);
                r[c] = ffma2(r[c], f32x2(k.x, k.y), f32x2(bf16_lo(vw[c]), bf16_hi(vw[c])));
                tops[c & 3] = most_of(tops[c & 3], r[c]);
            }
            float most = most3(most3(tops[0], tops[1], tops[2]), tops[3], 0.f);
            int gone = kChunk;
            if (__builtin_expect(!__all_sync(0xFFFFFFFFu, most < INFINITY), 0)) {  // zeros from the first that is not finite
                most = 0.f;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    float a, z;
                    f32x2_unpack(r[c], a, z);
                    if (gone == kChunk && !(fabsf(a) < INFINITY))
                        gone = t0 + 2 * c;
                    a = gone == kChunk ? a : 0.f;
                    if (gone == kChunk && !(fabsf(z) < INFINITY))
                        gone = t0 + 2 * c + 1;
                    z = gone == kChunk ? z : 0.f;
                    r[c] = f32x2(a, z);
                    most = most_of(most, r[c]);
                }
            }
            sh.bad[turn][part][col] = gone;
            sh.top_r[part][col] = most;
            meet();                                 // (all have read their products, too)
            const Scale sr(__float_as_uint(most_of_all(sh.top_r)));
            uint32_t hi[8], lo[8];
            split8(r[0], r[1], r[2], r[3], f32x2(sr.by, sr.by), hi, lo);
            split8(r[4], r[5], r[6], r[7], f32x2(sr.by, sr.by), hi + 4, lo + 4);
            __syncwarp();
            tmem_st8_async(lane_base + kXB + t0 / 2, hi);
            tmem_st8_async(lane_base + kXB + 32 + t0 / 2, lo);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&sh.r_ready);
            // the state, while T's product runs
            if (ch > 0) {
                y_by = s_undo;                      // of the outputs of the chunk before
                update(ch - 1);
                to_operand();
            }
            // U and w U, with one scale: w is at most 2
            const float u_by = sr.undo * f.t, w_by = f.w_undo;
            wait(&sh.u_done, phase, sh);
            tc_fence_after();
            uint32_t x[16], us[8];
            tmem_ld16_async(lane_base + kU + t0, x);
            tmem_wait_ld(x);
#pragma unroll
            for (int c = 0; c < 8; ++c)
                tops[c & 3] = most3(c < 4 ? 0.f : tops[c & 3], __uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1]));
            sh.top_u[part][col] = most3(most3(tops[0], tops[1], tops[2]), tops[3], 0.f);
            meet();                                 // (all have read the state's update, too)
            const Scale su(__float_as_uint(most_of_all(sh.top_u)));  // of the products as they came
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float2 w = *reinterpret_cast<const float2 *>(&f.w[t0 + 2 * c]);
                r[c] = fmul2(pair_of(x, c), f32x2(w.x, w.y));
                us[c] = pack2_f16(__uint_as_float(x[2 * c]) * su.by, __uint_as_float(x[2 * c + 1]) * su.by);
            }
            split8(r[0], r[1], r[2], r[3], f32x2(su.by, su.by), hi, lo);
            split8(r[4], r[5], r[6], r[7], f32x2(su.by, su.by), hi + 4, lo + 4);
            __syncwarp();
            tmem_st8_async(lane_base + kU + t0 / 2, hi);
            tmem_st8_async(lane_base + kU + 32 + t0 / 2, lo);
            tmem_st8_async(lane_base + kDS + t0 / 2, us);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&sh.w_ready);
            // the outputs of the chunk before, while M's product runs
            if (ch > 0 && with_outputs)
                outputs(ch - 1);
            keep = f.keep;
            z_by = su.undo * u_by;
            w_undo = z_by * w_by;
            bad = min(min(sh.bad[turn][0][col], sh.bad[turn][1][col]), min(sh.bad[turn][2][col], sh.bad[turn][3][col]));
        }
        if (chunks > 0) {
            y_by = s_undo;
            update(chunks - 1);
            if (with_outputs)
                outputs(chunks - 1);
        }
        if (there && to)
#pragma unroll
            for (int i = 0; i < kMine / 2; ++i) {
                const int d = t0 + (i >> 3) * 64 + (i & 7) * 2;
                if (with_values)
                    f32x2_unpack(s[i], to[d * D + col], to[(d + 1) * D + col]);
                else                                // F by columns, as it is read
                    *reinterpret_cast<uint64_t *>(&to[col * D + d]) = s[i];
            }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kMmaWarp) {
            // ---------------------------------------------------------- products
            constexpr uint32_t kIdesc = umma_idesc_f16(128, kChunk);
            const auto place_a = [&](int ch) { return base + P::kAt + (ch % P::kA) * P::kABytes; };
            const auto place_b = [&](int ch) { return base + P::kBt + (ch % P::kB) * P::kBBytes; };
            const auto place_c = [&](int ch) { return base + P::kCt + (ch % P::kC) * P::kCBytes; };
            const auto full_a = [&](int ch) { return wait(&sh.a_full[ch % P::kA], (ch / P::kA) & 1, sh); };
            // the state's parts with 64 rows of D elements
            const auto by_state = [&](uint32_t to, uint32_t rows, int parts) {
                const uint32_t b = desc_lo(rows, 16);
#pragma unroll 1
                for (int part = 0; part < parts; ++part)
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
                        umma_bf16_ts_lo(tmem + to, tmem + kS + part * (D / 2) + i * 8, b + (((i >> 2) * kTile + (i & 3) * 32) >> 4), kIdesc, part + i > 0);
            };
            // 64 tokens' part at `from` with 64 rows of 64 elements
            const auto by_tokens = [&](uint32_t to, uint32_t from, uint32_t rows, uint32_t more) {
                const uint32_t b = desc_lo(rows, 16);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    umma_bf16_ts_lo(tmem + to, tmem + from + i * 8, b + i * 2, kIdesc, more + i > 0);
            };
            // ... both in two parts
            const auto by_tokens2 = [&](uint32_t to, uint32_t from, uint32_t rows) {
#pragma unroll 1
                for (int i = 0; i < 3; ++i)
                    by_tokens(to, from + (i == 1 ? 32 : 0), rows + (i == 2 ? kTile : 0), i);
            };
            // half j of the state's update
            const auto update = [&](int ch, int j) {
                const uint32_t k = desc_lo(place_a(ch) + j * kTile, kTile);
#pragma unroll 1
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        umma_bf16_ts_lo(tmem + (j == 0 ? kDS : kXA), tmem + kU + part * 32 + i * 8, k + i * (2048 >> 4), kIdesc | kIdescBMnMajor, part + i > 0);
                umma_commit(j == 0 ? &sh.da_done : &sh.db_done);
                if (j == D / 64 - 1)
                    umma_commit(&sh.a_empty[ch % P::kA]);
            };
            bool ok = chunks > 0 && full_a(0) && wait(&sh.s_ready, 0, sh);
            if (ok) {
                tc_fence_after();
                if (elect_one()) {
                    by_state(kXA, place_a(0), 2);
                    umma_commit(&sh.x_done);
                }
                __syncwarp();
            }
#pragma unroll 1
            for (int ch = 0; ok && ch < chunks; ++ch) {
                const uint32_t phase = ch & 1;
                const bool more = ch + 1 < chunks;
                ok = wait(&sh.b_full[ch % P::kB], (ch / P::kB) & 1, sh) && wait(&sh.r_ready, phase, sh);
                if (!ok)
                    break;
                tc_fence_after();
                if (elect_one()) {
                    if (D > 64 && ch > 0)           // before T's product takes w U's place, and once S0^T K^T has been read
                        update(ch - 1, 1);
                    by_tokens2(kU, kXB, place_b(ch));
                    umma_commit(&sh.u_done);
                    umma_commit(&sh.b_empty[ch % P::kB]);
                }
                __syncwarp();
                ok = (ch == 0 || wait(&sh.s_ready, phase, sh)) && (!more || full_a(ch + 1));
                if (!ok)
                    break;
                tc_fence_after();
                if (more && elect_one())
                    by_state(kXA, place_a(ch + 1), 2);
                __syncwarp();
                ok = wait(&sh.w_ready, phase, sh);
                if (!ok)
                    break;
                tc_fence_after();
                if (more && elect_one()) {
                    by_tokens2(kXB, kU, place_a(ch + 1) + Rec::kRows);
                    umma_commit(&sh.x_done);
                }
                __syncwarp();
                ok = !with_outputs || (wait(&sh.c_full[ch % P::kC], (ch / P::kC) & 1, sh) && (ch == 0 || wait(&sh.y_free, phase ^ 1, sh)));
                if (!ok)
                    break;
                tc_fence_after();
                if (elect_one()) {
                    if (with_outputs) {
                        by_state(kY, place_c(ch), 1);
                        by_tokens(kZ, kDS, place_c(ch) + Rec::kRows, 0);
                        umma_commit(&sh.o_done);
                        umma_commit(&sh.c_empty[ch % P::kC]);
                    }
                    update(ch, 0);
                    if (D > 64 && !more)
                        update(ch, 1);
                }
                __syncwarp();
            }
        } else if (warp == kLoadWarp) {
            // ---------------------------------------------------------- copies
            const uint8_t *key = key_record<D>(p, hk, record), *value = value_record<D>(p, h, record);
            bool ok = true;
#pragma unroll 1
            for (int ch = 0; ok && ch < chunks; ++ch, key += Rec::kKeyBytes, value += Rec::kValueBytes) {
                const int a = ch % P::kA, b = ch % P::kB, c = ch % P::kC, f = ch % P::kF;
                ok = wait(&sh.a_empty[a], ((ch / P::kA) & 1) ^ 1, sh);
                if (ok && lane == 0) {
                    mbar_arrive_expect_tx(&sh.a_full[a], P::kABytes);
                    bulk_copy_g2s(smem + P::kAt + a * P::kABytes, key + Rec::kK, P::kABytes, &sh.a_full[a]);
                }
                __syncwarp();
                ok = ok && wait(&sh.b_empty[b], ((ch / P::kB) & 1) ^ 1, sh);
                if (ok && lane == 0) {
                    mbar_arrive_expect_tx(&sh.b_full[b], P::kBBytes);
                    tma_load_3d(smem + P::kBt + b * P::kBBytes + 2 * kTile, &map_v, 0, h, first + ch * kChunk, &sh.b_full[b]);
                    bulk_copy_g2s(smem + P::kBt + b * P::kBBytes, value + Rec::kT, 2 * kTile, &sh.b_full[b]);
                    mbar_arrive_expect_tx(&sh.f_full[f], kFactorBytes);
                    bulk_copy_g2s(smem + P::kFt + f * kFactorBytes, value + Rec::kFactors, kFactorBytes, &sh.f_full[f]);
                }
                __syncwarp();
                ok = ok && (!with_outputs || wait(&sh.c_empty[c], ((ch / P::kC) & 1) ^ 1, sh));
                if (ok && with_outputs && lane == 0) {
                    mbar_arrive_expect_tx(&sh.c_full[c], P::kCBytes);
                    bulk_copy_g2s(smem + P::kCt + c * P::kCBytes, key + Rec::kQ, Rec::kRows, &sh.c_full[c]);
                    bulk_copy_g2s(smem + P::kCt + c * P::kCBytes + Rec::kRows, value + Rec::kP, kTile, &sh.c_full[c]);
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
        if (tid == 0 && p.status)
            atomicExch(p.status, kStatusTimeout);
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 50000000ull) {}
        __syncthreads();
    }
    if (warp == kMmaWarp)
        tmem_dealloc(tmem, kTmemCols);
}

// The states after a sequence's segments but the last, from the first one's on: S <- F S + B, over B. A block has eight
// columns of a head's; kSplit threads share a row's sum. F comes by columns, the next segment's a step ahead.
constexpr int kJoinThreads = 256, kJoinColumns = 8;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) hc_delta_join_kernel(const DeltaPromptParams p)
{
    constexpr int kSplit = kJoinThreads / D, kTerms = D / kSplit, kBlocks = D / kJoinColumns;
    __shared__ __align__(16) float cur[D][kJoinColumns], sums[kSplit - 1][2][D][4];
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, row = tid % D, part = tid / D, k0 = part * kTerms;
    const int block = blockIdx.x % kBlocks, head = blockIdx.x / kBlocks, seq = head / p.Hv, h = head - seq * p.Hv;
    int first, len;
    if (!rows_of(p, seq, first, len))
        return;
    const long slots = segment_slots(p.N, p.S, p.seg), slot = segment_of(p, seq);
    const long last = max(((long)len + kChunk - 1) / kChunk - 1, 0l) / p.seg;
    if (last < 2)
        return;
    const auto end_of = [&](long at, bool values) { return p.ends + (((values ? 0 : slots) + slot + at) * p.Hv + h) * D * D; };
    float f[kTerms];
    const auto ask = [&](long at) {
#pragma unroll
        for (int i = 0; i < kTerms; ++i)
            f[i] = end_of(at, false)[(k0 + i) * D + row];
    };
    ask(1);
    if (part == 0) {
        const float4 *const at = reinterpret_cast<const float4 *>(end_of(0, true) + row * D + block * kJoinColumns);
        *reinterpret_cast<float4 *>(&cur[row][0]) = at[0];
        *reinterpret_cast<float4 *>(&cur[row][4]) = at[1];
    }
    __syncthreads();
#pragma unroll 1
    for (long at = 1; at < last; ++at) {
        float4 *const end = reinterpret_cast<float4 *>(end_of(at, true) + row * D + block * kJoinColumns);
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f), z = s;
        if (part == 0) {
            s = end[0];
            z = end[1];
        }
#pragma unroll
        for (int i = 0; i < kTerms; ++i) {
            const float4 x = *reinterpret_cast<const float4 *>(&cur[k0 + i][0]), y = *reinterpret_cast<const float4 *>(&cur[k0 + i][4]);
            s = make_float4(fmaf(f[i], x.x, s.x), fmaf(f[i], x.y, s.y), fmaf(f[i], x.z, s.z), fmaf(f[i], x.w, s.w));
            z = make_float4(fmaf(f[i], y.x, z.x), fmaf(f[i], y.y, z.y), fmaf(f[i], y.z, z.z), fmaf(f[i], y.w, z.w));
        }
        if (at + 1 < last)
            ask(at + 1);
        if (part > 0) {
            *reinterpret_cast<float4 *>(&sums[part - 1][0][row][0]) = s;
            *reinterpret_cast<float4 *>(&sums[part - 1][1][row][0]) = z;
        }
        __syncthreads();
        if (part == 0) {
#pragma unroll
            for (int i = 0; i < kSplit - 1; ++i) {
                const float4 x = *reinterpret_cast<const float4 *>(&sums[i][0][row][0]), y = *reinterpret_cast<const float4 *>(&sums[i][1][row][0]);
                s = make_float4(s.x + x.x, s.y + x.y, s.z + x.z, s.w + x.w);
                z = make_float4(z.x + y.x, z.y + y.y, z.z + y.z, z.w + y.w);
            }
            end[0] = s;
            end[1] = z;
            *reinterpret_cast<float4 *>(&cur[row][0]) = s;
            *reinterpret_cast<float4 *>(&cur[row][4]) = z;
        }
        __syncthreads();
    }
}

template <int D>
cudaError_t launch(DeltaPromptParams p, cudaStream_t stream)
{
    static_assert(Plan<D>::kTotal + sizeof(Shared) <= 227 * 1024 && sizeof(PrepShared<D>) <= 227 * 1024, "shared memory");
    int per_sm = 1;
    cudaError_t e = attn_ready(reinterpret_cast<const void *>(hc_delta_prep_kernel<D>), kPrepThreads, (int)sizeof(PrepShared<D>), &per_sm);
    if (e == cudaSuccess)
        e = attn_ready(reinterpret_cast<const void *>(hc_delta_scan_kernel<D>), kThreads, Plan<D>::kTotal, &per_sm);
    if (e != cudaSuccess)
        return e;
    CUtensorMap map_v{};
    if (!tc_make_map_heads(&map_v, p.v, p.N, p.Hv, D, p.v_stride, 1, kChunk, true))
        return cudaErrorInvalidValue;
    p.seg = segment_chunks(p.N, p.S, p.Hv);
    const long slots = p.seg > 0 ? segment_slots(p.N, p.S, p.seg) : 0;
    p.ends = reinterpret_cast<float *>(p.work + records_bytes(p.N, p.S, p.Hk, p.Hv, D));
    p.begun = reinterpret_cast<unsigned *>(p.ends + 2 * slots * p.Hv * D * D);
    const auto prep = [&](int part) {
        p.part = part;
        return launch_pdl(hc_delta_prep_kernel<D>, dim3((unsigned)(record_slots(p.N, p.S) * p.Hk)), dim3(kPrepThreads), sizeof(PrepShared<D>), true,
                          stream, p);
    };
    e = prep(p.seg > 0 && apart(p.N, p.S, p.Hv, p.seg) ? kFirstSegments : kAllSegments);
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
    lc.dynamicSmemBytes = Plan<D>::kTotal;
    if (p.seg == 0) {
        lc.gridDim = dim3((unsigned)(p.S * p.Hv));
        return cudaLaunchKernelEx(&lc, hc_delta_scan_kernel<D>, p, map_v);
    }
    lc.gridDim = dim3((unsigned)(2 * slots * p.Hv));
    e = cudaLaunchKernelEx(&lc, hc_delta_scan_kernel<D>, p, map_v);
    if (e == cudaSuccess && p.part != kAllSegments) {
        e = prep(kLastSegments);
        p.part = kAllSegments;
    }
    if (e == cudaSuccess)
        e = launch_pdl(hc_delta_join_kernel<D>, dim3((unsigned)(p.S * p.Hv * (D / kJoinColumns))), dim3(kJoinThreads), 0, true, stream, p);
    if (e != cudaSuccess)
        return e;
    p.again = 1;
    lc.gridDim = dim3((unsigned)(slots * p.Hv));
    return cudaLaunchKernelEx(&lc, hc_delta_scan_kernel<D>, p, map_v);
}

}  // namespace

size_t delta_prompt_bytes(int N, int S, int Hk, int Hv, int D)
{
    const long slots = most_segment_slots(N, S, Hv);
    return records_bytes(N, S, Hk, Hv, D) + (slots > 0 ? sizeof(float) * 2 * (size_t)slots * Hv * D * D + kBegunBytes : 0);
}

cudaError_t launch_delta_prompt(const DeltaPromptParams &p, const LaunchCfg &, cudaStream_t stream)
{
    return p.D == 64 ? launch<64>(p, stream) : launch<128>(p, stream);
}

}  // namespace tshc
