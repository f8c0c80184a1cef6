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
// All three move each byte once and are bound by HBM on a prompt and by launch
// latency on a step's few rows.
#include <algorithm>

#include "hc_kv.cuh"

namespace tshc {

namespace {

constexpr int kKvThreads = 256;
constexpr float kInt4Most = 57344.f;

// Reductions over aligned groups of W lanes.
template <int W>
__device__ __forceinline__ float group_max(float v)
{
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1)
        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

__device__ __forceinline__ float lanes_max(float v, int w)
{
    for (int o = w / 2; o > 0; o >>= 1)
        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

template <int W>
__device__ __forceinline__ bool group_any(bool v)
{
    // The mask's bits of this thread's group of W lanes (W divides 32).
    const unsigned b = __ballot_sync(0xFFFFFFFFu, v);
    const unsigned lane = threadIdx.x & 31;
    return ((b >> (lane / W * W)) & (W == 32 ? 0xFFFFFFFFu : (1u << W) - 1u)) != 0;
}

__device__ __forceinline__ bool lanes_any(bool v, int w)
{
    const unsigned b = __ballot_sync(0xFFFFFFFFu, v);
    const unsigned lane = threadIdx.x & 31;
    return ((b >> (lane & ~(unsigned)(w - 1))) & ((1u << w) - 1u)) != 0;
}

// Which row a thread works on: D/16 lanes a row, 16 elements a lane; rows in the
// order of the bf16 side ([b][t][head], keys then values), so that its accesses
// are contiguous over the block.
template <int kLanes>
struct RowAt {
    bool valid, value;        // value: a value's row, else a key's
    int part, b, h;
    int t;                    // token within the sequence
    size_t token;             // b * T + t
    __device__ RowAt(const KvParams &p, unsigned idx)  // 32-bit divisions: the host keeps 2 B T heads lanes below 2^31
    {
        part = (int)(idx % kLanes);
        unsigned r = idx / kLanes;
        const unsigned per = (unsigned)p.B * p.T * p.c.heads;
        value = r >= per;
        r -= value ? per : 0;
        valid = r < per;
        const unsigned tok = r / (unsigned)p.c.heads;
        h = (int)(r - tok * p.c.heads);
        b = (int)(tok / (unsigned)p.T);
        t = (int)(tok - (unsigned)b * p.T);
        token = tok;
    }
};

template <int kType, int kLanes>
__global__ void __launch_bounds__(kKvThreads) hc_kv_write_kernel(const KvParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    const RowAt<kLanes> at(p, blockIdx.x * kKvThreads + threadIdx.x);
    // Lanes past the last row stay for the shuffles; a whole warp of them leaves.
    if (!__any_sync(0xFFFFFFFFu, at.valid))
        return;
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    long page = -1, pos = 0;
    if (at.valid) {
        const uint4 *in = reinterpret_cast<const uint4 *>((at.value ? p.v + at.token * p.v_stride : p.k + at.token * p.k_stride)
                                                          + (size_t)at.h * (kLanes * 16) + at.part * 16);
        a = in[0];
        b = in[1];
        pos = (long)p.start[at.b] + at.t;
        page = p.start[at.b] < 0 ? -1 : kv_page(p.c, at.b, pos);
        if (page < 0 && at.part == 0 && p.status)
            atomicExch(p.status, kStatusBadArg);
    }
    const size_t row = page < 0 ? 0 : kv_row(p.c, page, at.h, pos);
    uint8_t *codes = at.value ? p.c.v : p.c.k;
    if (kType == kKvBf16) {
        if (page >= 0) {
            uint4 *out = reinterpret_cast<uint4 *>(codes + row * (kLanes * 32)) + at.part * 2;
            out[0] = a;
            out[1] = b;
        }
        return;
    }
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    float x[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        x[2 * j] = bf16_lo(w[j]);
        x[2 * j + 1] = bf16_hi(w[j]);
    }
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 16; ++j)
        bad |= !finite_f32(x[j]);
    uint8_t *scales = at.value ? p.c.vs : p.c.ks;
    if (kType == kKvFp8) {
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j)
            m = fmaxf(m, fabsf(x[j]));
        bad = group_any<kLanes>(bad);
        m = group_max<kLanes>(m);
        const int byte = bad ? kFp8BadRow : fp8_scale_byte(m);
        const float inv = bad ? 0.f : __uint_as_float((uint32_t)(254 - byte) << 23);  // 2^-e, exact
        uint32_t out[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t word = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 f = make_float2(bad ? 0.f : x[4 * j + 2 * i] * inv, bad ? 0.f : x[4 * j + 2 * i + 1] * inv);
                word |= (uint32_t)__nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3) << (16 * i);
            }
            out[j] = word;
        }
        if (page >= 0) {
            reinterpret_cast<uint4 *>(codes + row * (kLanes * 16))[at.part] = make_uint4(out[0], out[1], out[2], out[3]);
            if (at.part == 0)
                scales[row] = (uint8_t)byte;
        }
        return;
    }
    // INT4: groups of 32, 64 or 128 elements are 2, 4 or 8 lanes
    const int gl = p.c.group / 16;
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int j = 1; j < 16; ++j) {
        lo = fminf(lo, x[j]);
        hi = fmaxf(hi, x[j]);
    }
    bad = lanes_any(bad, gl);
    hi = lanes_max(hi, gl);
    lo = -lanes_max(-lo, gl);
    // Values saturate at +-57344, so that q * scale + bias stays inside fp16 for every q.
    lo = fminf(fmaxf(lo, -kInt4Most), kInt4Most);
    hi = fminf(fmaxf(hi, -kInt4Most), kInt4Most);
    const __half s = __float2half_rn(__fdiv_rn(hi - lo, 15.f));
    const __half bias = __float2half_rn(lo);
    const float sf = __half2float(s), bf = __half2float(bias);
    uint32_t out[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        float q = sf > 0.f ? rintf(__fdiv_rn(x[j] - bf, sf)) : 0.f;
        q = bad ? 0.f : fminf(fmaxf(q, 0.f), 15.f);
        out[j / 8] |= (uint32_t)(int)q << (4 * (j % 8));
    }
    if (page >= 0) {
        reinterpret_cast<uint2 *>(codes + row * (kLanes * 8))[at.part] = make_uint2(out[0], out[1]);
        if (at.part % gl == 0) {
            const size_t g = row * (size_t)(kLanes / gl) + at.part / gl;
            reinterpret_cast<__half *>(scales)[g] = bad ? __ushort_as_half(0x7E00) : s;
            reinterpret_cast<__half *>(at.value ? p.c.vb : p.c.kb)[g] = bias;
        }
    }
}

template <int kType, int kLanes>
__global__ void __launch_bounds__(kKvThreads) hc_kv_read_kernel(const KvParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    const RowAt<kLanes> at(p, blockIdx.x * kKvThreads + threadIdx.x);
    if (!at.valid)
        return;
    const long pos = (long)p.start[at.b] + at.t;
    const long page = p.start[at.b] < 0 ? -1 : kv_page(p.c, at.b, pos);
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (page >= 0) {
        const size_t row = kv_row(p.c, page, at.h, pos);
        const uint8_t *codes = at.value ? p.c.v : p.c.k, *scales = at.value ? p.c.vs : p.c.ks;
        if (kType == kKvBf16) {
            const uint4 *in = reinterpret_cast<const uint4 *>(codes + row * (kLanes * 32)) + at.part * 2;
            a = in[0];
            b = in[1];
        } else {
            float x[16];
            if (kType == kKvFp8) {
                const uint4 in = reinterpret_cast<const uint4 *>(codes + row * (kLanes * 16))[at.part];
                const float s = fp8_scale(scales[row]);
                const uint32_t w[4] = {in.x, in.y, in.z, in.w};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[j / 2] >> (16 * (j & 1))), __NV_E4M3);
                    const float2 f = __half22float2(__half2(h));
                    x[2 * j] = f.x * s;
                    x[2 * j + 1] = f.y * s;
                }
            } else {
                const int gl = p.c.group / 16;
                const uint2 in = reinterpret_cast<const uint2 *>(codes + row * (kLanes * 8))[at.part];
                const size_t g = row * (size_t)(kLanes / gl) + at.part / gl;
                const float s = __half2float(reinterpret_cast<const __half *>(scales)[g]);
                const float bias = __half2float(reinterpret_cast<const __half *>(at.value ? p.c.vb : p.c.kb)[g]);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    x[j] = fmaf((float)(((j < 8 ? in.x : in.y) >> (4 * (j & 7))) & 15u), s, bias);
            }
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
                w[j] = reinterpret_cast<const uint32_t &>(v);
            }
            a = make_uint4(w[0], w[1], w[2], w[3]);
            b = make_uint4(w[4], w[5], w[6], w[7]);
        }
    } else if (at.part == 0 && p.status) {
        atomicExch(p.status, kStatusBadArg);
    }
    uint4 *out = reinterpret_cast<uint4 *>((at.value ? p.v_out : p.k_out)
                                           + ((size_t)at.token * p.c.heads + at.h) * (kLanes * 16)) + at.part * 2;
    out[0] = a;
    out[1] = b;
}

// Bytes of one row's codes and of one scale array's row.
__host__ __device__ __forceinline__ int row_bytes(int type, int D) { return type == kKvBf16 ? 2 * D : type == kKvFp8 ? D : D / 2; }

// Grid (B * heads, columns). A thread owns one column of a row (16 bytes of a
// key's or value's codes, one byte of an FP8 scale, or one fp16 scale or bias)
// and moves it along the path in ascending order: the source of a later step is
// never a place that an earlier one wrote (path[j] > path[i] >= i for j > i).
__global__ void __launch_bounds__(kKvThreads) hc_kv_compact_kernel(const KvCompactParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    const int b = blockIdx.x / p.c.heads, h = blockIdx.x % p.c.heads;
    const int ctx = p.ctx_len[b];
    int n = p.n_accepted[b];
    if (ctx < 0 || n < 0 || n >= p.T) {
        if (threadIdx.x == 0 && h == 0 && blockIdx.y == 0) {
            if (p.status)
                atomicExch(p.status, kStatusBadArg);
            if (p.new_len)
                p.new_len[b] = ctx;
        }
        return;
    }
    if (threadIdx.x == 0 && h == 0 && blockIdx.y == 0 && p.new_len)
        p.new_len[b] = ctx + n + 1;
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
            return;
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
    const size_t n = (size_t)2 * p.B * p.T * p.c.heads * kLanes;
    const dim3 grid((unsigned)((n + kKvThreads - 1) / kKvThreads));
    void (*kernel)(KvParams) = nullptr;
    switch (p.c.type) {
    case kKvBf16: kernel = write ? hc_kv_write_kernel<kKvBf16, kLanes> : hc_kv_read_kernel<kKvBf16, kLanes>; break;
    case kKvFp8: kernel = write ? hc_kv_write_kernel<kKvFp8, kLanes> : hc_kv_read_kernel<kKvFp8, kLanes>; break;
    default: kernel = write ? hc_kv_write_kernel<kKvInt4, kLanes> : hc_kv_read_kernel<kKvInt4, kLanes>; break;
    }
    return launch_pdl(kernel, grid, dim3(kKvThreads), 0, true, stream, p);
}

cudaError_t launch_any(const KvParams &p, bool write, cudaStream_t stream)
{
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
