// hc_delta.cu -- the gated delta rule, a few tokens at a time (ts_hc_delta_step in
// include/ts_hc.h).
//
//   S <- e^g S,  u = beta (v - S^T k),  S <- S + k u^T,  o = scale S^T q
//
// With D x D states of fp32 the bytes of the states, in and out, bound it: a token's other
// rows are D / 4 times fewer, and the 7 D^2 operations of a token and head take a tenth of
// the time that the 8 D^2 bytes do.
//
// Columns of a state do not meet, so a warp takes 32 of them for all tokens and keeps them in
// registers: 8 lanes of four columns each side by side (a 128-byte line of a row), 4 groups of
// lanes with D / 4 rows each. Its loads are all in flight at once, its sums over the rows are
// in a lane and then two shuffles, and nothing is exchanged between warps. The output needs
// no second pass over the state: S^T q = (e^g S)^T q + (k . q) u.
//
// 64 sequences x 4 tokens (2.5 on average) x 32 heads of 128: 48.8 us for 0.27 GB, 0.82 of the
// measured copy rate. With states loaded and stored as what stays in the caches, 52 (the loads or the stores alone as
// passing, 53 and 52); with a head's four warps in one block, 54, and one token of one sequence 3.7 for 2.8 us; 16 columns
// a warp 57, 8 columns 76. Ten or twelve warps a SM, in 168 registers, spill: 52.5 for 52.
#include <cuda_bf16.h>

#include "hc_prompt.h"
#include "ptx.cuh"

namespace tshc {

namespace {

constexpr unsigned kStatusInvalidArg = 1u;  // TS_ERR_INVALID_ARG of ts_hc.h
constexpr int kCols = 32;                    // of a warp
constexpr int kLanes = kCols / 4, kGroups = 32 / kLanes;  // that share a row; that share a column

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

template <int D>
__global__ void __launch_bounds__(32) hc_delta_step_kernel(const DeltaStepParams p)
{
    constexpr int kRows = D / kGroups;           // a lane's
    constexpr int kPer = D / 32;                 // elements of q and k that a lane loads
    __shared__ alignas(16) float qk[2][D];
    pdl_launch_dependents();
    pdl_wait();
    constexpr int kParts = D / kCols;
    const int lane = threadIdx.x, group = lane / kLanes;
    const int bh = blockIdx.x / kParts, b = bh / p.Hv, h = bh - b * p.Hv, hk = h / (p.Hv / p.Hk);
    const int col = (blockIdx.x % kParts) * kCols + (lane % kLanes) * 4;
    // Lane group g has rows 16 i + 4 g .. + 3, so that its reads of q and k are 16 bytes wide and the groups' side by side.
    const size_t at = ((size_t)bh * D + 4 * group) * D + col;
    const auto row = [](int i) { return (i >> 2) * (kGroups * 4) + (i & 3); };
    float4 s[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
        s[i] = __ldcs(reinterpret_cast<const float4 *>(p.state_in + at + (size_t)row(i) * D));
    int n = p.counts ? p.counts[b] : p.T;
    if (n < 0 || n > p.T) {
        if (p.status && threadIdx.x == 0 && h == 0)
            atomicExch(p.status, kStatusInvalidArg);
        n = min(max(n, 0), p.T);
    }
    float *const ks = qk[0], *const qs = qk[1];
    for (int t = 0; t < n; ++t) {
        const size_t tok = (size_t)b * p.T + t;
        const uint16_t *kp = p.k + tok * p.k_stride + (size_t)hk * D + lane * kPer, *qp = p.q + tok * p.q_stride + (size_t)hk * D + lane * kPer;
        float k[kPer], q[kPer];
#pragma unroll
        for (int i = 0; i < kPer; i += 2) {
            const uint32_t a = *reinterpret_cast<const uint32_t *>(kp + i), z = *reinterpret_cast<const uint32_t *>(qp + i);
            k[i] = bf16_lo(a);
            k[i + 1] = bf16_hi(a);
            q[i] = bf16_lo(z);
            q[i + 1] = bf16_hi(z);
        }
        const uint2 vw = *reinterpret_cast<const uint2 *>(p.v + tok * p.v_stride + (size_t)h * D + col);
        const float keep = expf(p.decay[tok * p.Hv + h]), beta = p.beta[tok * p.Hv + h];
        float kk = 0.f, qq = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            kk = fmaf(k[i], k[i], kk);
            qq = fmaf(q[i], q[i], qq);
        }
        float kn = 1.f, qn = p.scale;
        if (p.norm_eps >= 0.f) {
            kn = 1.f / sqrtf(warp_sum(kk) + p.norm_eps);
            qn = p.scale / sqrtf(warp_sum(qq) + p.norm_eps);
        }
        float kq = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            k[i] *= kn;
            q[i] *= qn;
            kq = fmaf(k[i], q[i], kq);
        }
        kq = warp_sum(kq);
        __syncwarp();                            // the last token's reads are done
#pragma unroll
        for (int i = 0; i < kPer; i += 2) {
            *reinterpret_cast<float2 *>(ks + lane * kPer + i) = make_float2(k[i], k[i + 1]);
            *reinterpret_cast<float2 *>(qs + lane * kPer + i) = make_float2(q[i], q[i + 1]);
        }
        __syncwarp();
        float4 sk = make_float4(0.f, 0.f, 0.f, 0.f), sq = sk;
#pragma unroll
        for (int i = 0; i < kRows; i += 4) {
            const float4 k4 = *reinterpret_cast<const float4 *>(ks + row(i) + 4 * group), q4 = *reinterpret_cast<const float4 *>(qs + row(i) + 4 * group);
            const float kr[4] = {k4.x, k4.y, k4.z, k4.w}, qr[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float4 &x = s[i + j];
                x = make_float4(x.x * keep, x.y * keep, x.z * keep, x.w * keep);
                sk = make_float4(fmaf(kr[j], x.x, sk.x), fmaf(kr[j], x.y, sk.y), fmaf(kr[j], x.z, sk.z), fmaf(kr[j], x.w, sk.w));
                sq = make_float4(fmaf(qr[j], x.x, sq.x), fmaf(qr[j], x.y, sq.y), fmaf(qr[j], x.z, sq.z), fmaf(qr[j], x.w, sq.w));
            }
        }
#pragma unroll
        for (int o = 16; o >= kLanes; o >>= 1) {
            sk.x += __shfl_xor_sync(0xFFFFFFFFu, sk.x, o);
            sk.y += __shfl_xor_sync(0xFFFFFFFFu, sk.y, o);
            sk.z += __shfl_xor_sync(0xFFFFFFFFu, sk.z, o);
            sk.w += __shfl_xor_sync(0xFFFFFFFFu, sk.w, o);
            sq.x += __shfl_xor_sync(0xFFFFFFFFu, sq.x, o);
            sq.y += __shfl_xor_sync(0xFFFFFFFFu, sq.y, o);
            sq.z += __shfl_xor_sync(0xFFFFFFFFu, sq.z, o);
            sq.w += __shfl_xor_sync(0xFFFFFFFFu, sq.w, o);
        }
        const float4 u = make_float4(beta * (bf16_lo(vw.x) - sk.x), beta * (bf16_hi(vw.x) - sk.y), beta * (bf16_lo(vw.y) - sk.z),
                                     beta * (bf16_hi(vw.y) - sk.w));
        if (group == 0) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(fmaf(kq, u.x, sq.x), fmaf(kq, u.y, sq.y));
            const __nv_bfloat162 hi = __floats2bfloat162_rn(fmaf(kq, u.z, sq.z), fmaf(kq, u.w, sq.w));
            *reinterpret_cast<uint2 *>(p.out + (tok * p.Hv + h) * D + col) =
                make_uint2(reinterpret_cast<const uint32_t &>(lo), reinterpret_cast<const uint32_t &>(hi));
        }
#pragma unroll
        for (int i = 0; i < kRows; i += 4) {
            const float4 k4 = *reinterpret_cast<const float4 *>(ks + row(i) + 4 * group);
            const float kr[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float4 &x = s[i + j];
                x = make_float4(fmaf(kr[j], u.x, x.x), fmaf(kr[j], u.y, x.y), fmaf(kr[j], u.z, x.z), fmaf(kr[j], u.w, x.w));
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i)
        __stcs(reinterpret_cast<float4 *>(p.state_out + at + (size_t)row(i) * D), s[i]);
}

}  // namespace

cudaError_t launch_delta_step(const DeltaStepParams &p, const LaunchCfg &, cudaStream_t stream)
{
    const dim3 grid((unsigned)p.B * p.Hv * (p.D / kCols));
    return p.D == 64 ? launch_pdl(hc_delta_step_kernel<64>, grid, dim3(32), 0, true, stream, p)
                     : launch_pdl(hc_delta_step_kernel<128>, grid, dim3(32), 0, true, stream, p);
}

}  // namespace tshc
