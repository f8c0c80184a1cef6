// hc_prompt.h -- launch parameters and launchers of the operators of a prompt's
// pass and of the token after it: head norms with rotary positions, attention
// over packed prompts, the gated delta rule, log probabilities (internal; the
// public ABI is include/ts_hc.h).
#pragma once

#include "hc_spec.h"

namespace tshc {

struct NormRopeParams {
    RopeParams r;
    const uint16_t *qw, *kw;  // [D]
    float eps;
};

struct PromptAttnParams {
    const uint16_t *v;        // for the values that a row's tile could not hold (infinities, NaNs)
    long v_stride;
    const int32_t *starts;    // [S + 1]
    uint16_t *out;            // [N][q_heads][D]
    float *lse;               // [N][q_heads] or nullptr
    int N, S, q_heads, kv_heads;
    int G, Gp, TB;            // query heads a key head; of a block; tokens of 128 rows (Gp * TB <= 128)
    float scale_log2;         // scale * log2(e), > 0
    unsigned *status;
};

struct DeltaStepParams {
    const uint16_t *q, *k, *v;
    long q_stride, k_stride, v_stride;
    const float *decay, *beta;  // [B*T][Hv]
    const int32_t *counts;      // or nullptr: T
    const float *state_in;      // [B][Hv][D][D]
    float *state_out;
    uint16_t *out;              // [B*T][Hv][D]
    int B, T, Hk, Hv, D;
    float scale, norm_eps;      // norm_eps < 0: q and k as they are
    unsigned *status;
};

struct DeltaPromptParams {
    const uint16_t *q, *k, *v;
    long q_stride, k_stride, v_stride;
    const float *decay, *beta;  // [N][Hv]
    const int32_t *starts;      // [S + 1]
    const float *state_in;      // [S][Hv][D][D]
    float *state_out;
    uint16_t *out;              // [N][Hv][D]
    uint8_t *work;              // one record a chunk and head
    int N, S, Hk, Hv, D;
    float scale, norm_eps;
    unsigned *status;
    // the launch's own: chunks of a segment (0: none), which segments' part, whether it is the walk for the outputs, the
    // segments' ends
    int seg, part, again;
    float *ends;
    unsigned *begun;            // 1 once the first walks have waited for what came before the call
};

struct LogprobParams {
    const void *logits;
    long stride;              // elements between rows
    const int32_t *tokens;    // [N][J] or nullptr
    float *logp;              // [N][J]
    float *entropy;           // [N] or nullptr
    int32_t *top_ids;         // [N][top]
    float *top_logp;
    int N, V, J, top;
    unsigned *status;
};

cudaError_t launch_qk_norm_rope(const NormRopeParams &p, const LaunchCfg &cfg, cudaStream_t stream);
// q, k: the first heads; strides in elements.
cudaError_t launch_prompt_attention(PromptAttnParams p, const uint16_t *q, long q_stride, const uint16_t *k, long k_stride, int D,
                                    const LaunchCfg &cfg, cudaStream_t stream);
// The query heads of a block and the blocks that a call can have at most.
int prompt_attn_heads(int G);
long prompt_attn_blocks(int N, int S, int q_heads, int kv_heads);
cudaError_t launch_delta_step(const DeltaStepParams &p, const LaunchCfg &cfg, cudaStream_t stream);
size_t delta_prompt_bytes(int N, int S, int Hk, int Hv, int D);
cudaError_t launch_delta_prompt(const DeltaPromptParams &p, const LaunchCfg &cfg, cudaStream_t stream);
cudaError_t launch_logprobs(const LogprobParams &p, bool bf16, const LaunchCfg &cfg, cudaStream_t stream);

}  // namespace tshc
