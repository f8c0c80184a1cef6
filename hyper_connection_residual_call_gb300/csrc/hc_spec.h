// hc_spec.h -- launch parameters and launchers of the speculative decoding
// step's kernels: rotary positions, the paged cache, tree attention and the
// verification of drafted tokens (internal; the public ABI is include/ts_hc.h).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "hc_kernels.h"

namespace tshc {

struct RopeTableParams {
    float *table;             // [max_pos][rot/2][2]
    int max_pos, half;        // half = rot/2
    double log_theta;         // of the theta in use (after TS_ROPE_NTK)
    int type;                 // ts_rope_scaling_type
    double factor, original, beta_fast, beta_slow, magnitude;
};

struct RopeParams {
    const uint16_t *q, *k;
    uint16_t *q_out, *k_out;
    long q_stride, k_stride, q_out_stride, k_out_stride;
    const int32_t *positions;
    const float *table;
    int max_pos, N, q_heads, k_heads, D, rot;
    bool interleaved, inverse, copy_rest;  // copy_rest: elements rot.. are copied (not in place)
    unsigned *status;
};

// Division of n < 2^31 by a fixed d, a multiplication and a shift (Granlund and
// Montgomery): n * mul >> (31 + L) with mul = floor(2^(31+L) / d) + 1, L = ceil(log2 d).
struct FastDiv {
    uint32_t mul, shift, d;
    FastDiv(uint32_t by = 1) : mul(0), shift(0), d(by)
    {
        uint32_t L = 0;
        while ((1ull << L) < by)
            ++L;
        if (L > 0) {
            mul = (uint32_t)((1ull << (31 + L)) / by + 1);
            shift = L - 1;
        }
    }
#ifdef __CUDACC__
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return mul ? __umulhi(n, mul) >> shift : n; }
#endif
};

// A cache's tensors; bytes per row and per row's scales by type.
struct KvView {
    int type, group, page_shift, heads, D, max_pages;
    long n_pages;
    uint8_t *k, *v, *ks, *vs, *kb, *vb;
    const int32_t *pages;
};

struct KvParams {
    KvView c;
    const uint16_t *k, *v;    // write: the rows in
    uint16_t *k_out, *v_out;  // read: the rows out
    long k_stride, v_stride;
    const int32_t *start;     // ctx_len or start
    int B, T;
    FastDiv by_run, by_heads, by_runs;  // rows run over tokens, then heads, then runs of tokens, then sequences
    unsigned *status;
};

struct KvCompactParams {
    KvView c;
    const int32_t *ctx_len, *path, *n_accepted;
    int32_t *new_len;
    int B, T;
    unsigned *status;
};

struct TreeBuildParams {
    const int32_t *parents, *ctx_len;
    long parents_stride;
    uint32_t *mask;
    int32_t *positions;
    int B, T;
    unsigned *status;
};

struct AttnParams {
    KvView c;
    const uint16_t *q;
    long q_stride;
    const int32_t *ctx_len;
    const uint32_t *mask;
    long mask_stride;         // words between sequences
    int mask_words;           // words in a mask row
    uint16_t *out;
    float *lse;
    int B, T, q_heads, G;     // G = query heads that share a key head
    int rows, row_blocks;     // rows = T * G, in blocks of the kernel's row tile
    float scale_log2;         // scale * log2(e)
    float *part;              // partial results of split items
    unsigned *status;
};

struct VerifyParams {
    const float *logits, *draft, *temperature, *u, *noise;
    const int32_t *tokens, *parents;
    long parents_stride;
    int32_t *n_accepted, *path, *next_token;
    int B, T, V;
    unsigned *status;
};

cudaError_t launch_rope_table(const RopeTableParams &p, cudaStream_t stream);
cudaError_t launch_rope(const RopeParams &p, const LaunchCfg &cfg, cudaStream_t stream);
cudaError_t launch_kv_write(const KvParams &p, const LaunchCfg &cfg, cudaStream_t stream);
cudaError_t launch_kv_read(const KvParams &p, const LaunchCfg &cfg, cudaStream_t stream);
cudaError_t launch_kv_compact(const KvCompactParams &p, const LaunchCfg &cfg, cudaStream_t stream);
cudaError_t launch_tree_build(const TreeBuildParams &p, const LaunchCfg &cfg, cudaStream_t stream);
// Bytes of partial results; an upper bound over devices, so that the host can size it without one.
size_t attn_part_bytes(int B, int T, int q_heads, const KvView &c);
cudaError_t launch_tree_attention(AttnParams p, const LaunchCfg &cfg, cudaStream_t stream);
cudaError_t launch_verify(const VerifyParams &p, const LaunchCfg &cfg, cudaStream_t stream);

// Launch with programmatic dependent launch: every kernel here waits for the
// kernel before it (pdl_wait) before it touches memory.
template <typename P>
inline cudaError_t launch_pdl(void (*kernel)(P), dim3 grid, dim3 block, size_t smem, bool pdl, cudaStream_t stream,
                              const P &p, int cluster = 1)
{
    cudaLaunchConfig_t lc{};
    lc.gridDim = grid;
    lc.blockDim = block;
    lc.dynamicSmemBytes = smem;
    lc.stream = stream;
    cudaLaunchAttribute at[2];
    int n = 0;
    if (pdl) {
        at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        at[n].id = cudaLaunchAttributeClusterDimension;
        at[n].val.clusterDim.x = cluster;
        at[n].val.clusterDim.y = 1;
        at[n++].val.clusterDim.z = 1;
    }
    lc.attrs = at;
    lc.numAttrs = n;
    return cudaLaunchKernelEx(&lc, kernel, p);
}

}  // namespace tshc
