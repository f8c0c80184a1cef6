// hc_qk_norm.cu -- the norms of query and key heads and their rotary positions in
// one pass (ts_hc_qk_norm_rope in include/ts_hc.h).
//
//   n_i = x_i w_i / sqrt(mean_j x_j^2 + eps),  (y0, y1) = (n0 c - n1 s, n0 s + n1 c) for
//   each turned pair, (c, s) = table[pos][i]
//
// The operator reads and writes each head's row once, like the rotation alone; a norm of
// its own would read and write them again. Sums and products are fp32, and the result is
// rounded to bf16 once.
//
// What bounds it is its bytes: 16381 tokens x 40 heads x 128, half of each turned, take 55 us for
// 0.34 GB, 0.91 of the measured copy rate, with two heads' loads in flight a thread and eight
// blocks a SM of 128 threads (four of 256: 56; loads as of passing data: 63); four heads' loads, in 94
// registers and half of the threads, took 63 to 66. One token of 24 heads takes
// 2.1 us: a launch, and a chain of two loads and a sum. (GPU times of calls replayed back to back in a
// CUDA graph, here and below.)
#include <cuda_bf16.h>

#include "hc_prompt.h"
#include "ptx.cuh"

namespace tshc {

namespace {

constexpr unsigned kStatusInvalidArg = 1u;  // TS_ERR_INVALID_ARG of ts_hc.h
constexpr int kThreads = 128;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return reinterpret_cast<const uint32_t &>(v);
}

__device__ __forceinline__ float2 turn(float x0, float x1, float2 cs)
{
    return make_float2(fmaf(x0, cs.x, -(x1 * cs.y)), fmaf(x0, cs.y, x1 * cs.x));
}

__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8])
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(u[i]);
        x[2 * i + 1] = bf16_hi(u[i]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// kUnits threads a head, each with two vectors of 8 elements: of the turned part, vectors u
// and u + rot/16 (the halves of 8 pairs, or four interleaved pairs each), of the rest
// likewise, so that the lanes' vectors lie side by side and a thread's 8 (cos, sin) serve
// every head that it walks. The sum of squares goes over the kUnits lanes. D = 16 kUnits,
// rot a multiple of 16.
template <int kUnits, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 8) hc_qk_norm_kernel(const NormRopeParams np, int lanes)
{
    constexpr int D = kUnits * 16;
    pdl_launch_dependents();
    pdl_wait();
    const RopeParams &p = np.r;
    const unsigned idx = blockIdx.x * kThreads + threadIdx.x;
    const int u = (int)(idx % kUnits);
    const unsigned rest = idx / kUnits;
    const int lane = (int)(rest % (unsigned)lanes);
    const unsigned n = rest / (unsigned)lanes;
    const bool there = n < (unsigned)p.N;  // the lanes of a head agree; all stay for the shuffles
    const int turned = p.rot / 16, heads = p.q_heads + p.k_heads;
    const bool rotate = u < turned;
    const int v0 = rotate ? u : turned * 2 + (u - turned), v1 = rotate ? u + turned : v0 + (kUnits - turned);
    float2 cs[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        cs[j] = make_float2(0.f, 0.f);
    if (rotate && there) {
        const int pos = p.positions[n];
        const bool ok = pos >= 0 && pos < p.max_pos;
        if (!ok && p.status && u == 0 && lane == 0)
            atomicExch(p.status, kStatusInvalidArg);
        if (ok) {
            const float4 *t = reinterpret_cast<const float4 *>(p.table + (size_t)pos * p.rot);  // two pairs each
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 w = t[kInterleaved ? (j < 2 ? 2 * v0 + j : 2 * v1 + j - 2) : 4 * u + j];
                cs[2 * j] = make_float2(w.x, w.y);
                cs[2 * j + 1] = make_float2(w.z, w.w);
            }
        }
    }
    constexpr int kAhead = 2;  // heads whose loads are in flight
    for (int h0 = lane; h0 < heads; h0 += kAhead * lanes) {
        uint4 in[kAhead][2];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int h = h0 + i * lanes;
            in[i][0] = in[i][1] = make_uint4(0, 0, 0, 0);
            if (h < heads && there) {
                const uint4 *src = reinterpret_cast<const uint4 *>(h < p.q_heads ? p.q + (size_t)n * p.q_stride + (size_t)h * D
                                                                                : p.k + (size_t)n * p.k_stride + (size_t)(h - p.q_heads) * D);
                in[i][0] = src[v0];
                in[i][1] = src[v1];
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int h = h0 + i * lanes;
            float a[8], b[8];
            unpack8(in[i][0], a);
            unpack8(in[i][1], b);
            float sum = 0.f, sum2 = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sum = fmaf(a[j], a[j], sum);
                sum2 = fmaf(b[j], b[j], sum2);
            }
            sum += sum2;
#pragma unroll
            for (int o = kUnits / 2; o > 0; o >>= 1)
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            if (h >= heads || !there)
                continue;
            const float inv = rsqrtf(fmaf(sum, 1.f / D, np.eps));
            const bool is_q = h < p.q_heads;
            const uint4 *w = reinterpret_cast<const uint4 *>(is_q ? np.qw : np.kw);
            float wa[8], wb[8];
            unpack8(w[v0], wa);  // (not as read-only data: that could be loaded before pdl_wait())
            unpack8(w[v1], wb);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                a[j] *= inv * wa[j];
                b[j] *= inv * wb[j];
            }
            if (rotate) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (kInterleaved) {
                        float *pair = (j < 4 ? a : b) + (j & 3) * 2;
                        const float2 y = turn(pair[0], pair[1], cs[j]);
                        pair[0] = y.x;
                        pair[1] = y.y;
                    } else {
                        const float2 y = turn(a[j], b[j], cs[j]);
                        a[j] = y.x;
                        b[j] = y.y;
                    }
                }
            }
            uint4 *out = reinterpret_cast<uint4 *>(is_q ? p.q_out + (size_t)n * p.q_out_stride + (size_t)h * D
                                                        : p.k_out + (size_t)n * p.k_out_stride + (size_t)(h - p.q_heads) * D);
            out[v0] = pack8(a);
            out[v1] = pack8(b);
        }
    }
}

// Any even rot and any D (a multiple of 8 up to 1024): one warp a head, a lane's pairs 32
// apart, then its elements of the rest. A lane reads what it writes before it writes, so the
// rows may be turned in place.
__global__ void __launch_bounds__(kThreads) hc_qk_norm_any_kernel(const NormRopeParams np)
{
    pdl_launch_dependents();
    pdl_wait();
    const RopeParams &p = np.r;
    const int lane = threadIdx.x & 31, heads = p.q_heads + p.k_heads, half = p.rot / 2;
    const unsigned long warp = (unsigned long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const unsigned long n = warp / heads;
    const int h = (int)(warp % heads);
    if (n >= (unsigned long)p.N)
        return;
    const bool is_q = h < p.q_heads;
    const int hh = is_q ? h : h - p.q_heads;
    const uint16_t *in = (is_q ? p.q + n * p.q_stride : p.k + n * p.k_stride) + (size_t)hh * p.D;
    uint16_t *out = (is_q ? p.q_out + n * p.q_out_stride : p.k_out + n * p.k_out_stride) + (size_t)hh * p.D;
    const uint16_t *w = is_q ? np.qw : np.kw;
    const auto value = [](uint16_t x) { return __uint_as_float((uint32_t)x << 16); };
    float sum = 0.f;
    for (int i = lane; i < p.D; i += 32)
        sum = fmaf(value(in[i]), value(in[i]), sum);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    const float inv = rsqrtf(sum / p.D + np.eps);
    const int pos = p.positions[n];
    const bool ok = pos >= 0 && pos < p.max_pos;
    if (!ok && p.status && lane == 0 && h == 0)
        atomicExch(p.status, kStatusInvalidArg);
    for (int u = lane; u < half; u += 32) {
        const float2 cs = ok ? reinterpret_cast<const float2 *>(p.table)[(size_t)pos * half + u] : make_float2(0.f, 0.f);
        const int i0 = p.interleaved ? 2 * u : u, i1 = p.interleaved ? 2 * u + 1 : u + half;
        const float2 y = turn(value(in[i0]) * (inv * value(w[i0])), value(in[i1]) * (inv * value(w[i1])), cs);
        out[i0] = __bfloat16_as_ushort(__float2bfloat16_rn(y.x));
        out[i1] = __bfloat16_as_ushort(__float2bfloat16_rn(y.y));
    }
    for (int i = p.rot + lane; i < p.D; i += 32)
        out[i] = __bfloat16_as_ushort(__float2bfloat16_rn(value(in[i]) * (inv * value(w[i]))));
}

template <int kUnits>
cudaError_t launch_units(const NormRopeParams &p, const LaunchCfg &cfg, cudaLaunchConfig_t &lc)
{
    // A thread walks 8 heads once there are enough tokens to fill the GPU with a few blocks a SM; below that one
    // head a thread, for latency.
    const int heads = p.r.q_heads + p.r.k_heads;
    const long one = (long)p.r.N * kUnits * heads;
    const int walk = one > (long)cfg.sm_count * 4096 ? 8 : 1;
    const int lanes = (heads + walk - 1) / walk;
    lc.gridDim = dim3((unsigned)(((unsigned long)p.r.N * kUnits * lanes + kThreads - 1) / kThreads));
    return cudaLaunchKernelEx(&lc, p.r.interleaved ? hc_qk_norm_kernel<kUnits, true> : hc_qk_norm_kernel<kUnits, false>, p, lanes);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const NormRopeParams &p, const LaunchCfg &cfg, cudaStream_t stream)
{
    cudaLaunchConfig_t lc{};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = at;
    lc.numAttrs = 1;
    lc.blockDim = dim3(kThreads);
    lc.stream = stream;
    if (p.r.rot % 16 == 0) {
        switch (p.r.D) {
        case 64: return launch_units<4>(p, cfg, lc);
        case 128: return launch_units<8>(p, cfg, lc);
        case 256: return launch_units<16>(p, cfg, lc);
        default: break;
        }
    }
    const unsigned long warps = (unsigned long)p.r.N * (p.r.q_heads + p.r.k_heads);
    lc.gridDim = dim3((unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32)));
    return cudaLaunchKernelEx(&lc, hc_qk_norm_any_kernel, p);
}

}  // namespace tshc
