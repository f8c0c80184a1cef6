// hc_rope.cu -- rotary positions of query and key heads, and their table of
// cosines and sines (ts_hc_rope, ts_hc_rope_table in include/ts_hc.h).
//
//   (y0, y1) = (x0 c - x1 s, x0 s + x1 c) for pair i of a head at position pos,
//   (c, s) = table[pos][i] = magnitude * (cos, sin)(pos * f_i)
//
// The operator does 3 flops an element and is bound by its bytes: each head's
// row once in and once out, and the token's table row (rot * 4 bytes against
// heads * D * 4). GPU times of calls replayed back to back in a CUDA graph (called from
// Python, the shorter ones take some 15 us, which is the host's time): 16384 tokens x 40
// heads x 128, half of each turned: 55 us for 0.34 GB, 0.91 of the measured copy rate. 4099
// tokens x 18 heads x 64: 8.5 us for 20 MB, and one token 4.2 us: a launch, and a chain of
// two dependent loads.
#include <cuda_bf16.h>

#include <algorithm>

#include "hc_spec.h"
#include "ptx.cuh"

namespace tshc {

namespace {

constexpr unsigned kStatusInvalidArg = 1u;  // TS_ERR_INVALID_ARG of ts_hc.h
constexpr int kRopeThreads = 256;

// One thread per (pos, i). The angle is formed in 64 bits: at position 10^6 a
// 32-bit product would be off by up to 0.03 rad. Run once per model.
__global__ void __launch_bounds__(kRopeThreads) hc_rope_table_kernel(const RopeTableParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    const long idx = (long)blockIdx.x * blockDim.x + threadIdx.x;
    if (idx >= (long)p.max_pos * p.half)
        return;
    const long pos = idx / p.half;
    const int i = (int)(idx - pos * p.half);
    double f = exp(-p.log_theta * (double)i / (double)p.half);  // theta^(-2i/rot)
    if (p.type == 1) {
        f /= p.factor;
    } else if (p.type == 3) {
        const double turns = p.original * f * 0.15915494309189535;  // over 2 pi
        const double keep = fmin(fmax((turns - p.beta_slow) / (p.beta_fast - p.beta_slow), 0.0), 1.0);
        f = f * keep + f / p.factor * (1.0 - keep);
    }
    double s, c;
    sincos((double)pos * f, &s, &c);
    reinterpret_cast<float2 *>(p.table)[idx] = make_float2((float)(c * p.magnitude), (float)(s * p.magnitude));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return reinterpret_cast<const uint32_t &>(v);
}

__device__ __forceinline__ float2 turn(float x0, float x1, float2 cs)
{
    return make_float2(fmaf(x0, cs.x, -(x1 * cs.y)), fmaf(x0, cs.y, x1 * cs.x));
}

// Unit u of a head is 16 of its elements and the 8 pairs they form: vectors u and
// u + rot/16 of 8 elements (the two halves of pairs in the half layout, four pairs
// each interleaved), so that the lanes' vectors lie side by side; the units after
// rot/16 are the elements that are copied, split likewise. A thread keeps its
// unit's 8 (cos, sin) in registers and walks the heads lane, lane + lanes, ...
// of one token, so a table row is read once per `lanes` threads' units and not
// once per head. rot and D multiples of 16.
template <bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) hc_rope_kernel(const RopeParams p, int units, int lanes)
{
    pdl_launch_dependents();
    pdl_wait();
    const unsigned idx = blockIdx.x * kRopeThreads + threadIdx.x;
    const int u = (int)(idx % (unsigned)units);
    const unsigned rest = idx / (unsigned)units;
    const int lane = (int)(rest % (unsigned)lanes);
    const unsigned n = rest / (unsigned)lanes;
    if (n >= (unsigned)p.N)
        return;
    const int turned = p.rot / 16, heads = p.q_heads + p.k_heads;
    const bool rotate = u < turned;
    int v0, v1;
    if (!rotate) {
        v0 = turned * 2 + (u - turned);
        v1 = v0 + (p.D / 16 - turned);
    } else {
        v0 = u;
        v1 = u + turned;
    }
    float2 cs[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        cs[j] = make_float2(0.f, 0.f);
    if (rotate) {
        const int pos = p.positions[n];
        const bool ok = pos >= 0 && pos < p.max_pos;
        if (!ok && p.status && u == 0 && lane == 0)
            atomicExch(p.status, kStatusInvalidArg);
        const float4 *t = reinterpret_cast<const float4 *>(p.table + (size_t)(ok ? pos : 0) * p.rot);  // two pairs each
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float4 w = t[kInterleaved ? (j < 2 ? 2 * v0 + j : 2 * v1 + j - 2) : 4 * u + j];
            if (!ok)
                w = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p.inverse) {
                w.y = -w.y;
                w.w = -w.w;
            }
            cs[2 * j] = make_float2(w.x, w.y);
            cs[2 * j + 1] = make_float2(w.z, w.w);
        }
    }
    // Four heads' loads in flight. Turned and copied units take the same path, with the result chosen at
    // the end: a warp holds both kinds where a part of the head is turned.
    for (int h0 = lane; h0 < heads; h0 += 4 * lanes) {
        uint4 in[4][2];
        uint4 *out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int h = h0 + i * lanes;
            if (h < heads) {
                const bool is_q = h < p.q_heads;
                const int hh = is_q ? h : h - p.q_heads;
                const uint4 *src = reinterpret_cast<const uint4 *>((is_q ? p.q + (size_t)n * p.q_stride : p.k + (size_t)n * p.k_stride) +
                                                                   (size_t)hh * p.D);
                out[i] = reinterpret_cast<uint4 *>((is_q ? p.q_out + (size_t)n * p.q_out_stride : p.k_out + (size_t)n * p.k_out_stride) +
                                                   (size_t)hh * p.D);
                in[i][0] = src[v0];
                in[i][1] = src[v1];
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (h0 + i * lanes >= heads)
                break;
            const uint32_t aw[4] = {in[i][0].x, in[i][0].y, in[i][0].z, in[i][0].w};
            const uint32_t bw[4] = {in[i][1].x, in[i][1].y, in[i][1].z, in[i][1].w};
            uint32_t ya[4], yb[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (kInterleaved) {
                    const float2 y = turn(bf16_lo(aw[j]), bf16_hi(aw[j]), cs[j]);
                    const float2 z = turn(bf16_lo(bw[j]), bf16_hi(bw[j]), cs[4 + j]);
                    ya[j] = pack_bf16(y.x, y.y);
                    yb[j] = pack_bf16(z.x, z.y);
                } else {
                    const float2 y = turn(bf16_lo(aw[j]), bf16_lo(bw[j]), cs[2 * j]);
                    const float2 z = turn(bf16_hi(aw[j]), bf16_hi(bw[j]), cs[2 * j + 1]);
                    ya[j] = pack_bf16(y.x, z.x);
                    yb[j] = pack_bf16(y.y, z.y);
                }
                ya[j] = rotate ? ya[j] : aw[j];
                yb[j] = rotate ? yb[j] : bw[j];
            }
            out[i][v0] = make_uint4(ya[0], ya[1], ya[2], ya[3]);
            out[i][v1] = make_uint4(yb[0], yb[1], yb[2], yb[3]);
        }
    }
}

// Any even rot and any D: one thread per pair of a head, then the copied
// elements (D - rot of them, two to a thread). Taken where rot or D is not a
// multiple of 16, so that the 16-byte units do not hold. 2-byte accesses: 16384 tokens x
// 40 heads x 80 with 20 turned take 169 us (38 with 16 turned, in units), one token 4.1.
__global__ void __launch_bounds__(kRopeThreads) hc_rope_any_kernel(const RopeParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    const int half = p.rot / 2, per = p.D / 2, heads = p.q_heads + p.k_heads;
    const unsigned long idx = (unsigned long)blockIdx.x * kRopeThreads + threadIdx.x;
    const int u = (int)(idx % per);
    const unsigned long rest = idx / per;
    const int h = (int)(rest % heads);
    const unsigned long n = rest / heads;
    if (n >= (unsigned long)p.N)
        return;
    const bool is_q = h < p.q_heads;
    const int hh = is_q ? h : h - p.q_heads;
    const uint16_t *in = (is_q ? p.q + n * p.q_stride : p.k + n * p.k_stride) + (size_t)hh * p.D;
    uint16_t *out = (is_q ? p.q_out + n * p.q_out_stride : p.k_out + n * p.k_out_stride) + (size_t)hh * p.D;
    if (u >= half) {
        if (p.copy_rest)
            reinterpret_cast<uint32_t *>(out)[u] = reinterpret_cast<const uint32_t *>(in)[u];
        return;
    }
    const int pos = p.positions[n];
    const bool ok = pos >= 0 && pos < p.max_pos;
    if (!ok && p.status && u == 0 && h == 0)
        atomicExch(p.status, kStatusInvalidArg);
    float2 cs = make_float2(0.f, 0.f);
    if (ok)
        cs = reinterpret_cast<const float2 *>(p.table)[(size_t)pos * half + u];
    if (p.inverse)
        cs.y = -cs.y;
    const int i0 = p.interleaved ? 2 * u : u, i1 = p.interleaved ? 2 * u + 1 : u + half;
    const float2 y = turn(__uint_as_float((uint32_t)in[i0] << 16), __uint_as_float((uint32_t)in[i1] << 16), cs);
    out[i0] = __bfloat16_as_ushort(__float2bfloat16_rn(y.x));
    out[i1] = __bfloat16_as_ushort(__float2bfloat16_rn(y.y));
}

}  // namespace

cudaError_t launch_rope_table(const RopeTableParams &p, cudaStream_t stream)
{
    const long n = (long)p.max_pos * p.half;
    return launch_pdl(hc_rope_table_kernel, dim3((unsigned)((n + kRopeThreads - 1) / kRopeThreads)), dim3(kRopeThreads), 0, true,
                      stream, p);
}

cudaError_t launch_rope(const RopeParams &p, const LaunchCfg &cfg, cudaStream_t stream)
{
    cudaLaunchConfig_t lc{};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = at;
    lc.numAttrs = 1;
    lc.blockDim = dim3(kRopeThreads);
    lc.stream = stream;
    const int heads = p.q_heads + p.k_heads;
    if (p.rot % 16 != 0 || p.D % 16 != 0) {
        const unsigned long n = (unsigned long)p.N * heads * (p.D / 2);
        lc.gridDim = dim3((unsigned)((n + kRopeThreads - 1) / kRopeThreads));
        return cudaLaunchKernelEx(&lc, hc_rope_any_kernel, p);
    }
    // In place there is nothing to copy, so the copied units get no threads.
    const int units = p.copy_rest ? p.D / 16 : p.rot / 16;
    // A thread walks 8 heads once there are enough tokens to fill the GPU with
    // a few blocks an SM; below that one head a thread, for latency.
    const long one = (long)p.N * units * heads;
    const int walk = one > (long)cfg.sm_count * kRopeThreads * 16 ? 8 : 1;
    const int lanes = (heads + walk - 1) / walk;
    const unsigned long n = (unsigned long)p.N * units * lanes;
    lc.gridDim = dim3((unsigned)((n + kRopeThreads - 1) / kRopeThreads));
    return cudaLaunchKernelEx(&lc, p.interleaved ? hc_rope_kernel<true> : hc_rope_kernel<false>, p, units, lanes);
}

}  // namespace tshc
