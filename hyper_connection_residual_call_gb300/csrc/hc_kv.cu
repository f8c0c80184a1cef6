// hc_kv.cu -- the paged cache of keys and values: quantised as it is written,
// read back as bf16, and the accepted nodes' rows moved after a verification;
// and the masks of a tree of drafted tokens (ts_hc_kv_write, ts_hc_kv_read,
// ts_hc_kv_compact, ts_hc_tree_build in include/ts_hc.h).
//
//   FP8   code = e4m3(x * 2^-e), e the smallest with max|x| <= 448 * 2^e. A power
//         of two keeps every step exact: x * 2^-e loses nothing before the one
//         rounding to e4m3, the code times 2^e is a bf16, and the attention can
//         apply it to a product's sum. A floating code gains nothing from a finer
//         scale but the use of its top half octave.
//   INT4  scale = f16((max - min)/15), bias = f16(min), q = round((x - bias)/scale),
//         the same format as the library's INT4-affine weights.
//
// Writing and reading move each byte once; on a prompt bf16 and FP8 are bound by HBM, INT4
// by its instructions, and a step's few rows by launch latency. Times are the GPU's for
// calls replayed back to back in a CUDA graph (a step's calls take some 10 us each from
// Python, which is the host's time).
#include <algorithm>

#include "hc_kv.cuh"

namespace tshc {

namespace {

constexpr int kKvThreads = 256;
constexpr float kInt4Most = 57344.f;

// Where a thread works: D/16 lanes a row, of which a lane has elements [8 part, 8 part + 8)
// of each half, so that the lanes' accesses lie side by side; the key's and the value's
// row of one token and head. Rows go over a run of up to kRun tokens of one head first:
// their codes and scales lie side by side in a page, and a warp's stores of 2-byte
// scales are one piece of memory.
constexpr int kRun = 32;

template <int kLanes>
struct RowAt {
    bool valid, placed;       // placed: the row has a place in the cache (if not, that is recorded)
    int part, h;
    size_t token;             // b * T + t
    size_t row;
    __device__ __forceinline__ RowAt(const KvParams &p, unsigned idx)  // 32 bits: the host keeps the rows' lanes below 2^31
    {
        part = (int)(idx % kLanes);
        const unsigned r = idx / kLanes, r1 = p.by_run.div(r), r2 = p.by_heads.div(r1), b = p.by_runs.div(r2);
        const unsigned t = (r2 - b * p.by_runs.d) * p.by_run.d + (r - r1 * p.by_run.d);
        h = (int)(r1 - r2 * p.by_heads.d);
        token = (size_t)b * p.T + t;
        valid = b < (unsigned)p.B && t < (unsigned)p.T;
        placed = false;
        row = 0;
        if (!valid)
            return;
        const int start = p.start[b];
        const long pos = (long)start + t;
        const long page = start < 0 ? -1 : kv_page(p.c, (int)b, pos);
        placed = page >= 0;
        if (placed)
            row = kv_row(p.c, page, h, pos);
        else if (part == 0 && p.status)
            atomicExch(p.status, kStatusBadArg);
    }
};

// q = clamp(round(d / scale), 0, 15), ties to even. The quotient by the reciprocal is
// corrected once with its exact remainder (Markstein's step): a quotient that lies on a
// tie, which d and scale of few bits often do, comes out as the tie itself.
__device__ __forceinline__ float quotient(float d, float by, float inv)
{
    const float q = d * inv;
    return fmaf(fmaf(-q, by, d), inv, q);
}

__device__ __forceinline__ float int4_code(float d, float scale, float inv)
{
    constexpr float kEven = 12582912.f;  // 1.5 * 2^23: the sum is rounded to a whole number, ties to even
    return fminf(fmaxf(quotient(d, scale, inv), 0.f), 15.f) + kEven - kEven;
}

__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// bf16 pairs in an order that signed 16-bit comparison keeps (its own inverse).
__device__ __forceinline__ uint32_t ordered16x2(uint32_t w) { return w ^ (((w >> 15) & 0x00010001u) * 0x7FFFu); }

// One row's elements of this lane (a: of the first half, b: of the second), quantised and stored.
template <int kType, int kLanes>
__device__ __forceinline__ void write_row(const KvView &c, const RowAt<kLanes> &at, uint8_t *codes, uint8_t *scales, uint8_t *biases,
                                          const uint4 a, const uint4 b)
{
    if (kType == kKvBf16) {
        if (at.placed) {
            uint4 *out = reinterpret_cast<uint4 *>(codes + at.row * (kLanes * 32)) + at.part;
            out[0] = a;
            out[kLanes] = b;
        }
        return;
    }
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (kType == kKvFp8) {
        // |x| as 16-bit integers keeps its order, and infinities and NaNs are the largest
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            top = __vmaxu2(top, w[j] & 0x7FFF7FFFu);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1)
            top = __vmaxu2(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        top = max(top & 0xFFFFu, top >> 16);
        const bool bad = top >= 0x7F80u;
        const int byte = bad ? kFp8BadRow : fp8_scale_byte(__uint_as_float(top << 16));
        const float inv = __uint_as_float((uint32_t)(254 - byte) << 23);  // 2^-e, exact
        if (byte == kFp8TopRow) {  // (the same for a row's lanes, and rare)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                w[j] = (w[j] & 0x80008000u) | __vminu2(w[j] & 0x7FFF7FFFu, kFp8TopBits * 0x10001u);
        }
        uint32_t out[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(bf16_lo(w[2 * j]) * inv, bf16_hi(w[2 * j]) * inv), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi =
                __nv_cvt_float2_to_fp8x2(make_float2(bf16_lo(w[2 * j + 1]) * inv, bf16_hi(w[2 * j + 1]) * inv), __NV_SATFINITE, __NV_E4M3);
            out[j] = bad ? 0u : lo | hi << 16;
        }
        if (at.placed) {
            uint2 *to = reinterpret_cast<uint2 *>(codes + at.row * (kLanes * 16)) + at.part;
            to[0] = make_uint2(out[0], out[1]);
            to[kLanes] = make_uint2(out[2], out[3]);
            if (at.part == 0)
                scales[at.row] = (uint8_t)byte;
        }
        return;
    }
    // INT4: a group of 32 or more elements is 4 or more lanes of a half, or both halves.
    // range[k]: the largest element in the low 16 bits and the complement of the smallest in the high
    // ones, both as ordered integers, so that one signed maximum serves both.
    uint32_t range[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t most = ordered16x2(w[4 * k]), least = most;
#pragma unroll
        for (int j = 4 * k + 1; j < 4 * k + 4; ++j) {
            const uint32_t o = ordered16x2(w[j]);
            most = __vmaxs2(most, o);
            least = __vmins2(least, o);
        }
        least = ~least;
        range[k] = __vmaxs2(__byte_perm(most, least, 0x5410), __byte_perm(most, least, 0x7632));
#pragma unroll
        for (int o = 2; o > 0; o >>= 1)  // groups of 32: 4 lanes
            range[k] = __vmaxs2(range[k], __shfl_xor_sync(0xFFFFFFFFu, range[k], o));
        if (kLanes >= 8 && c.group >= 64)
            range[k] = __vmaxs2(range[k], __shfl_xor_sync(0xFFFFFFFFu, range[k], 4));
        if (kLanes >= 16 && c.group >= 128)
            range[k] = __vmaxs2(range[k], __shfl_xor_sync(0xFFFFFFFFu, range[k], 8));
    }
    if (c.group > kLanes * 8)
        range[0] = range[1] = __vmaxs2(range[0], range[1]);
    uint32_t word[2];
    __half scale[2], bias[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        // Infinities and NaNs are the largest or the smallest: from 0x7F80 on in both halves, where the
        // lowest finite bf16's complement is 0x7F7F like the highest itself.
        const bool bad = (int16_t)(range[k] & 0xFFFFu) >= 0x7F80 || (int16_t)(range[k] >> 16) >= 0x7F80;
        // Values saturate at +-57344, so that q * scale + bias stays inside fp16 for every q.
        const uint32_t most = ordered16x2(range[k] & 0xFFFFu) << 16, least = ordered16x2(~range[k] >> 16) << 16;
        const float top = fminf(fmaxf(__uint_as_float(most), -kInt4Most), kInt4Most);
        const float low = fminf(fmaxf(__uint_as_float(least), -kInt4Most), kInt4Most);
        const __half s = __float2half_rn(quotient(top - low, 15.f, 1.f / 15.f));
        bias[k] = __float2half_rn(low);
        scale[k] = bad ? __ushort_as_half(0x7E00) : s;
        const float sf = __half2float(s), bf = __half2float(bias[k]);
        const bool none = bad || !(sf > 0.f);
        const float inv = none ? 0.f : rcp(sf);
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t v = w[4 * k + i / 2];
            q[i] = int4_code(((i & 1) ? bf16_hi(v) : bf16_lo(v)) - bf, sf, inv);
        }
        // four codes are a whole number below 2^16: its bits over 2^23
        const float lo4 = fmaf(fmaf(fmaf(q[3], 16.f, q[2]), 16.f, q[1]), 16.f, q[0]) + 8388608.f;
        const float hi4 = fmaf(fmaf(fmaf(q[7], 16.f, q[6]), 16.f, q[5]), 16.f, q[4]) + 8388608.f;
        word[k] = none ? 0u : __byte_perm(__float_as_uint(lo4), __float_as_uint(hi4), 0x5410);
    }
    if (at.placed) {
        uint32_t *to = reinterpret_cast<uint32_t *>(codes + at.row * (kLanes * 8)) + at.part;
        to[0] = word[0];
        to[kLanes] = word[1];
        // a group's lanes: the first stores the first half's scale and bias, the second the other's
        const int lanes = c.group / 8, turn = at.part % lanes, groups = kLanes * 16 / c.group;
        if (turn < 2 && at.part < kLanes && !(turn == 1 && c.group > kLanes * 8)) {
            const size_t g = at.row * groups + (at.part + turn * kLanes) / lanes;
            reinterpret_cast<__half *>(scales)[g] = turn ? scale[1] : scale[0];
            reinterpret_cast<__half *>(biases)[g] = turn ? bias[1] : bias[0];
        }
    }
}

// A thread has the key's and the value's elements of its token and head: their loads
// are in flight together, and they share what finding the place costs. (Four rows of
// each a thread were no faster: the kernels are bound by their instructions as much as
// by HBM, 32768 tokens x 8 heads of FP8.) 32768 tokens x 8 heads x 128 of FP8: 31 us to
// write and 32 to read, 0.2 GB each, 0.96 of the measured copy rate, with the arithmetic
// pipe busy 63% and 37% of the time; bf16 both ways 86 us for 0.54 GB, 0.92. INT4 in
// groups of 64, both ways: 102 us for 0.34 GB (63 and 41 alone), of them 51 its bytes': 3.2 of
// 4 instructions a cycle and the arithmetic pipe busy 68% to write, 2.7 and 70% to read. A step's
// rows (8 x 13 tokens of 4 heads, both ways) take 8.3 us: two launches and their chains
// of lengths, pages and rows.
template <int kType, int kLanes>
__global__ void __launch_bounds__(kKvThreads) hc_kv_write_kernel(const KvParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    const RowAt<kLanes> at(p, blockIdx.x * kKvThreads + threadIdx.x);
    // Lanes past the last row stay for the shuffles; a whole warp of them leaves.
    if (!__any_sync(0xFFFFFFFFu, at.valid))
        return;
    uint4 k0 = make_uint4(0, 0, 0, 0), k1 = k0, v0 = k0, v1 = k0;
    if (at.valid) {
        const size_t off = (size_t)at.h * (kLanes * 16) + at.part * 8;
        const uint4 *k = reinterpret_cast<const uint4 *>(p.k + at.token * p.k_stride + off);
        const uint4 *v = reinterpret_cast<const uint4 *>(p.v + at.token * p.v_stride + off);
        k0 = k[0];
        k1 = k[kLanes];
        v0 = v[0];
        v1 = v[kLanes];
    }
    write_row<kType, kLanes>(p.c, at, p.c.k, p.c.ks, p.c.kb, k0, k1);
    write_row<kType, kLanes>(p.c, at, p.c.v, p.c.vs, p.c.vb, v0, v1);
}

// This lane's elements of a stored row (a: of the first half, b: of the second), as bf16.
template <int kType, int kLanes>
__device__ __forceinline__ void read_row(const KvView &c, const RowAt<kLanes> &at, const uint8_t *codes, const uint8_t *scales,
                                         const uint8_t *biases, uint4 &a, uint4 &b)
{
    a = b = make_uint4(0, 0, 0, 0);
    if (!at.placed)
        return;
    if (kType == kKvBf16) {
        const uint4 *in = reinterpret_cast<const uint4 *>(codes + at.row * (kLanes * 32)) + at.part;
        a = in[0];
        b = in[kLanes];
        return;
    }
    uint32_t w[8];
    if (kType == kKvFp8) {
        const uint2 *in = reinterpret_cast<const uint2 *>(codes + at.row * (kLanes * 16)) + at.part;
        const uint2 in0 = in[0], in1 = in[kLanes];
        const float s = fp8_scale(scales[at.row]);
        const uint32_t v[4] = {in0.x, in0.y, in1.x, in1.y};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(v[j / 2] >> (16 * (j & 1))), __NV_E4M3);
            const float2 f = __half22float2(__half2(h));
            const __nv_bfloat162 y = __floats2bfloat162_rn(f.x * s, f.y * s);
            w[j] = reinterpret_cast<const uint32_t &>(y);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int part = at.part + k * kLanes;
            const uint32_t in = reinterpret_cast<const uint32_t *>(codes + at.row * (kLanes * 8))[part];
            const size_t g = at.row * (size_t)(kLanes * 16 / c.group) + part / (c.group / 8);
            const float s = __half2float(reinterpret_cast<const __half *>(scales)[g]), bias = __half2float(reinterpret_cast<const __half *>(biases)[g]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t v = in >> (8 * j);
                const __nv_bfloat162 y = __floats2bfloat162_rn(fmaf((float)(v & 15u), s, bias), fmaf((float)((v >> 4) & 15u), s, bias));
                w[4 * k + j] = reinterpret_cast<const uint32_t &>(y);
            }
        }
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
    b = make_uint4(w[4], w[5], w[6], w[7]);
}

template <int kType, int kLanes>
__global__ void __launch_bounds__(kKvThreads) hc_kv_read_kernel(const KvParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    const RowAt<kLanes> at(p, blockIdx.x * kKvThreads + threadIdx.x);
    if (!at.valid)
        return;
    uint4 k0, k1, v0, v1;
    read_row<kType, kLanes>(p.c, at, p.c.k, p.c.ks, p.c.kb, k0, k1);
    read_row<kType, kLanes>(p.c, at, p.c.v, p.c.vs, p.c.vb, v0, v1);
    const size_t off = (at.token * p.c.heads + at.h) * (kLanes * 16) + at.part * 8;
    uint4 *k = reinterpret_cast<uint4 *>(p.k_out + off), *v = reinterpret_cast<uint4 *>(p.v_out + off);
    k[0] = k0;
    k[kLanes] = k1;
    v[0] = v0;
    v[kLanes] = v1;
}

// Bytes of one row's codes and of one scale array's row.
__host__ __device__ __forceinline__ int row_bytes(int type, int D) { return type == kKvBf16 ? 2 * D : type == kKvFp8 ? D : D / 2; }

// Grid (B * heads, columns). A thread owns one column of a row (16 bytes of a
// key's or value's codes, one byte of an FP8 scale, or one fp16 scale or bias)
// and moves it along the path in ascending order: the source of a later step is
// never a place that an earlier one wrote (path[j] > path[i] >= i for j > i). Each step of a
// path is a chain of dependent loads, its node, the pages and the row: 16 sequences x 8 heads
// x 128, three steps: 3.1 us bf16, 3.5 FP8, 4.3 INT4; 64 sequences, seven steps: 5.2, 6.4, 7.5.
__global__ void __launch_bounds__(kKvThreads) hc_kv_compact_kernel(const KvCompactParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    const int b = blockIdx.x / p.c.heads, h = blockIdx.x % p.c.heads;
    const int ctx = p.ctx_len[b];
    const bool lead = threadIdx.x == 0 && h == 0 && blockIdx.y == 0;
    int n = p.n_accepted[b];
    if (ctx < 0 || n < 0 || n >= p.T) {
        if (lead) {
            if (p.status)
                atomicExch(p.status, kStatusBadArg);
            if (p.new_len)
                p.new_len[b] = ctx;
        }
        return;
    }
    const int cols = row_bytes(p.c.type, p.c.D) / 16;
    const int scols = p.c.type == kKvBf16 ? 0 : p.c.type == kKvFp8 ? 1 : 2 * (p.c.D / p.c.group);
    const int per = cols + scols;
    int i = blockIdx.y * kKvThreads + threadIdx.x;
    if (i >= 2 * per)
        return;
    const bool value = i >= per;
    i -= value ? per : 0;
    uint8_t *codes = value ? p.c.v : p.c.k;
    int last = 0;
    for (int step = 1; step <= n; ++step) {
        const int node = p.path[(size_t)b * p.T + step];
        const long src = node < 0 ? -1 : kv_page(p.c, b, (long)ctx + node), dst = kv_page(p.c, b, (long)ctx + step);
        if (node <= last || node >= p.T || src < 0 || dst < 0) {  // not an ascending path, or no place
            if (i == 0 && p.status)
                atomicExch(p.status, kStatusBadArg);
            n = step - 1;
            break;
        }
        last = node;
        if (node == step)
            continue;
        const size_t s = kv_row(p.c, src, h, (long)ctx + node), d = kv_row(p.c, dst, h, (long)ctx + step);
        if (i < cols) {
            uint4 *x = reinterpret_cast<uint4 *>(codes);
            x[d * cols + i] = x[s * cols + i];
        } else if (p.c.type == kKvFp8) {
            uint8_t *x = value ? p.c.vs : p.c.ks;
            x[d] = x[s];
        } else {
            const int groups = p.c.D / p.c.group, g = (i - cols) % groups;
            uint16_t *x = reinterpret_cast<uint16_t *>(i - cols < groups ? (value ? p.c.vs : p.c.ks) : (value ? p.c.vb : p.c.kb));
            x[d * groups + g] = x[s * groups + g];
        }
    }
    if (lead && p.new_len)
        p.new_len[b] = ctx + n + 1;  // the root and the steps that were moved
}

// One thread per (sequence, node): walks up to the root. An entry that is not a
// smaller node's index ends the walk (negative for i > 0: the node is absent).
__global__ void __launch_bounds__(128) hc_tree_build_kernel(const TreeBuildParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    const long idx = (long)blockIdx.x * blockDim.x + threadIdx.x;
    if (idx >= (long)p.B * p.T)
        return;
    const int b = (int)(idx / p.T), i = (int)(idx % p.T);
    const int32_t *parents = p.parents + (long)b * p.parents_stride;
    const int words = (p.T + 31) / 32;
    uint32_t *row = p.mask ? p.mask + (size_t)idx * words : nullptr;
    if (row)
        for (int w = 0; w < words; ++w)
            row[w] = 0;
    int depth = 0, node = i;
    bool present = true;
    while (node > 0) {
        const int up = parents[node];
        if (up >= node) {
            if (p.status)
                atomicExch(p.status, kStatusBadArg);
            present = false;
            break;
        }
        if (up < 0) {
            present = false;
            break;
        }
        node = up;
        ++depth;
    }
    if (row && present)
        for (node = i;; node = parents[node]) {
            row[node >> 5] |= 1u << (node & 31);
            if (node == 0)
                break;
        }
    if (p.positions)
        p.positions[idx] = (p.ctx_len ? p.ctx_len[b] : 0) + (present ? depth : 0);
}

template <int kLanes>
cudaError_t launch_rows(const KvParams &p, bool write, cudaStream_t stream)
{
    const size_t n = (size_t)p.B * p.by_runs.d * p.by_heads.d * p.by_run.d * kLanes;
    const dim3 grid((unsigned)((n + kKvThreads - 1) / kKvThreads));
    void (*kernel)(KvParams) = nullptr;
    switch (p.c.type) {
    case kKvBf16: kernel = write ? hc_kv_write_kernel<kKvBf16, kLanes> : hc_kv_read_kernel<kKvBf16, kLanes>; break;
    case kKvFp8: kernel = write ? hc_kv_write_kernel<kKvFp8, kLanes> : hc_kv_read_kernel<kKvFp8, kLanes>; break;
    default: kernel = write ? hc_kv_write_kernel<kKvInt4, kLanes> : hc_kv_read_kernel<kKvInt4, kLanes>; break;
    }
    return launch_pdl(kernel, grid, dim3(kKvThreads), 0, true, stream, p);
}

cudaError_t launch_any(KvParams p, bool write, cudaStream_t stream)
{
    const int run = std::min(p.T, kRun);
    p.by_run = FastDiv((uint32_t)run);
    p.by_heads = FastDiv((uint32_t)p.c.heads);
    p.by_runs = FastDiv((uint32_t)((p.T + run - 1) / run));
    switch (p.c.D) {
    case 64: return launch_rows<4>(p, write, stream);
    case 128: return launch_rows<8>(p, write, stream);
    default: return launch_rows<16>(p, write, stream);
    }
}

}  // namespace

cudaError_t launch_kv_write(const KvParams &p, const LaunchCfg &, cudaStream_t stream) { return launch_any(p, true, stream); }

cudaError_t launch_kv_read(const KvParams &p, const LaunchCfg &, cudaStream_t stream) { return launch_any(p, false, stream); }

cudaError_t launch_kv_compact(const KvCompactParams &p, const LaunchCfg &, cudaStream_t stream)
{
    const int per = row_bytes(p.c.type, p.c.D) / 16 + (p.c.type == kKvBf16 ? 0 : p.c.type == kKvFp8 ? 1 : 2 * (p.c.D / p.c.group));
    return launch_pdl(hc_kv_compact_kernel, dim3((unsigned)(p.B * p.c.heads), (unsigned)((2 * per + kKvThreads - 1) / kKvThreads)),
                      dim3(kKvThreads), 0, true, stream, p);
}

cudaError_t launch_tree_build(const TreeBuildParams &p, const LaunchCfg &, cudaStream_t stream)
{
    const long n = (long)p.B * p.T;
    return launch_pdl(hc_tree_build_kernel, dim3((unsigned)((n + 127) / 128)), dim3(128), 0, true, stream, p);
}

}  // namespace tshc
