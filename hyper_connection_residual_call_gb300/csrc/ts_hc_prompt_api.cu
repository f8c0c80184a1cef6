// ts_hc_prompt_api.cu -- the C ABI of the operators of a prompt's pass and of the
// token after it in include/ts_hc.h (head norms with rotary positions,
// attention over packed prompts, the gated delta rule, log probabilities): argument validation on the host, then the
// launches.
#include <climits>
#include <cmath>

#include "hc_prompt.h"
#include "ts_hc.h"
#include "ts_hc_checks.h"

namespace {

using tshc::api_error;
using tshc::check_count;
using tshc::check_ptr_api;
using tshc::check_stride;
using tshc::device;
using tshc::kMaxBatch;
using tshc::kMaxHeads;
using tshc::launched;
using tshc::overlap;
using tshc::rows_overlap;

// Bytes from the first row's first element to the last row's last.
size_t span(int n, long stride, long width, size_t size) { return ((size_t)(n - 1) * stride + width) * size; }

// Memory that a call reads or writes (n = 0: not given).
struct Part {
    const void *p;
    size_t n;
    const char *name;
};

// What is written apart from all of what is read, and from one another.
template <int W, int R>
ts_status check_apart(const Part (&written)[W], const Part (&read)[R])
{
    for (int i = 0; i < W; ++i) {
        for (const Part &r : read)
            if (written[i].n > 0 && r.n > 0 && overlap(written[i].p, written[i].n, r.p, r.n))
                return api_error(TS_ERR_INVALID_ARG, "%s overlaps %s", written[i].name, r.name);
        for (int j = 0; j < i; ++j)
            if (written[i].n > 0 && written[j].n > 0 && overlap(written[i].p, written[i].n, written[j].p, written[j].n))
                return api_error(TS_ERR_INVALID_ARG, "%s overlaps %s", written[j].name, written[i].name);
    }
    return TS_OK;
}

// The heads of the gated delta rule: D, the key heads and the value heads that share them.
ts_status check_delta_heads(int k_heads, int v_heads, int D)
{
    TS_TRY(check_count(k_heads, "k_heads", 1, kMaxHeads));
    TS_TRY(check_count(v_heads, "v_heads", 1, kMaxHeads));
    if (v_heads % k_heads != 0)
        return api_error(TS_ERR_INVALID_ARG, "v_heads = %d must be a multiple of k_heads = %d", v_heads, k_heads);
    if (D != 64 && D != 128)
        return api_error(TS_ERR_UNSUPPORTED, "D = %d: heads of 64 and 128 are supported", D);
    return TS_OK;
}

ts_status check_delta_rows(const void *q, long q_stride, const void *k, long k_stride, const void *v, long v_stride, const float *decay,
                           const float *beta, const void *out, int n, int k_heads, int v_heads, int D)
{
    const long kw = (long)k_heads * D, vw = (long)v_heads * D;
    TS_TRY(check_ptr_api(q, "q", 16));
    TS_TRY(check_ptr_api(k, "k", 16));
    TS_TRY(check_ptr_api(v, "v", 16));
    TS_TRY(check_stride(q_stride, "q_stride", kw, 8));
    TS_TRY(check_stride(k_stride, "k_stride", kw, 8));
    TS_TRY(check_stride(v_stride, "v_stride", vw, 8));
    TS_TRY(check_ptr_api(decay, "decay", 4));
    TS_TRY(check_ptr_api(beta, "beta", 4));
    TS_TRY(check_ptr_api(out, "out", 16));
    // rows of other heads and tokens are read while a block writes its own
    if (rows_overlap(out, vw, vw, q, q_stride, kw, n))
        return api_error(TS_ERR_INVALID_ARG, "out overlaps q");
    if (rows_overlap(out, vw, vw, k, k_stride, kw, n))
        return api_error(TS_ERR_INVALID_ARG, "out overlaps k");
    if (rows_overlap(out, vw, vw, v, v_stride, vw, n))
        return api_error(TS_ERR_INVALID_ARG, "out overlaps v");
    const size_t bytes = span(n, vw, vw, 2), gates = sizeof(float) * (size_t)n * v_heads;
    if (overlap(out, bytes, decay, gates) || overlap(out, bytes, beta, gates))
        return api_error(TS_ERR_INVALID_ARG, "out overlaps decay or beta");
    return TS_OK;
}

// The states before and after: the same ones or apart, and apart from what is read beside them.
ts_status check_states(const float *state_in, const float *state_out, int n_states, int v_heads, int D, const void *out, size_t out_bytes)
{
    TS_TRY(check_ptr_api(state_in, "state_in", 16));
    TS_TRY(check_ptr_api(state_out, "state_out", 16));
    const size_t bytes = sizeof(float) * (size_t)n_states * v_heads * D * D;
    if (state_in != state_out && overlap(state_in, bytes, state_out, bytes))
        return api_error(TS_ERR_INVALID_ARG, "state_out overlaps state_in");
    if (out_bytes > 0 && (overlap(state_out, bytes, out, out_bytes) || overlap(state_in, bytes, out, out_bytes)))
        return api_error(TS_ERR_INVALID_ARG, "out overlaps the states");
    return TS_OK;
}

ts_status check_scale(float scale, float norm_eps)
{
    if (!std::isfinite(scale))
        return api_error(TS_ERR_INVALID_ARG, "scale = %g must be finite", (double)scale);
    if (!std::isfinite(norm_eps))
        return api_error(TS_ERR_INVALID_ARG, "norm_eps = %g must be finite", (double)norm_eps);
    return TS_OK;
}

}  // namespace

extern "C" {

ts_status ts_hc_qk_norm_rope(const void *q, long q_stride, const void *k, long k_stride, const int32_t *positions, const float *table,
                             int max_pos, const void *q_norm_w, const void *k_norm_w, float eps, void *q_out, long q_out_stride,
                             void *k_out, long k_out_stride, int N, int q_heads, int k_heads, int D, int rot, int interleaved,
                             cudaStream_t stream)
{
    tshc::clear_error();
    TS_TRY(check_count(N, "N", 0, INT_MAX));
    TS_TRY(check_count(q_heads, "q_heads", 1, kMaxHeads));
    TS_TRY(check_count(k_heads, "k_heads", 0, kMaxHeads));
    if (D < 8 || D > 1024 || D % 8 != 0)
        return api_error(TS_ERR_INVALID_ARG, "D = %d must be a multiple of 8 in [8, 1024]", D);
    if (rot < 2 || rot > D || rot % 2 != 0)
        return api_error(TS_ERR_INVALID_ARG, "rot = %d must be even and in [2, D = %d]", rot, D);
    TS_TRY(check_count(max_pos, "max_pos", 1, INT_MAX));
    if (!(eps > 0.f) || !std::isfinite(eps))
        return api_error(TS_ERR_INVALID_ARG, "eps = %g must be > 0", (double)eps);
    if (N == 0)
        return TS_OK;
    const long qw = (long)q_heads * D, kw = (long)k_heads * D;
    TS_TRY(check_ptr_api(q, "q", 16));
    TS_TRY(check_ptr_api(q_out, "q_out", 16));
    TS_TRY(check_ptr_api(q_norm_w, "q_norm_w", 16));
    TS_TRY(check_stride(q_stride, "q_stride", qw, 8));
    TS_TRY(check_stride(q_out_stride, "q_out_stride", qw, 8));
    if (k_heads > 0) {
        TS_TRY(check_ptr_api(k, "k", 16));
        TS_TRY(check_ptr_api(k_out, "k_out", 16));
        TS_TRY(check_ptr_api(k_norm_w, "k_norm_w", 16));
        TS_TRY(check_stride(k_stride, "k_stride", kw, 8));
        TS_TRY(check_stride(k_out_stride, "k_out_stride", kw, 8));
    }
    TS_TRY(check_ptr_api(positions, "positions", 4));
    TS_TRY(check_ptr_api(table, "table", 16));
    if ((long)N * (q_heads + k_heads) * ((D + 15) / 16) > INT_MAX)
        return api_error(TS_ERR_UNSUPPORTED, "%d tokens of %d heads are too many for one call: split them", N, q_heads + k_heads);
    const bool q_in = q_out == q, k_in = k_heads == 0 || k_out == k;
    if (q_in && q_stride != q_out_stride)
        return api_error(TS_ERR_INVALID_ARG, "q_out is q but q_out_stride = %ld is not q_stride = %ld", q_out_stride, q_stride);
    if (k_heads > 0 && k_in && k_stride != k_out_stride)
        return api_error(TS_ERR_INVALID_ARG, "k_out is k but k_out_stride = %ld is not k_stride = %ld", k_out_stride, k_stride);
    if (!q_in && rows_overlap(q, q_stride, qw, q_out, q_out_stride, qw, N))
        return api_error(TS_ERR_INVALID_ARG, "q_out overlaps q");
    if (k_heads > 0) {
        if (!k_in && rows_overlap(k, k_stride, kw, k_out, k_out_stride, kw, N))
            return api_error(TS_ERR_INVALID_ARG, "k_out overlaps k");
        if (rows_overlap(q_out, q_out_stride, qw, k, k_stride, kw, N))
            return api_error(TS_ERR_INVALID_ARG, "q_out overlaps k");
        if (rows_overlap(k_out, k_out_stride, kw, q, q_stride, qw, N))
            return api_error(TS_ERR_INVALID_ARG, "k_out overlaps q");
        if (rows_overlap(q_out, q_out_stride, qw, k_out, k_out_stride, kw, N))
            return api_error(TS_ERR_INVALID_ARG, "q_out overlaps k_out");
    }
    const size_t weights = 2 * (size_t)D, places = sizeof(int32_t) * (size_t)N, q_bytes = span(N, q_out_stride, qw, 2);
    const size_t k_bytes = k_heads > 0 ? span(N, k_out_stride, kw, 2) : 0, angles = sizeof(float) * (size_t)max_pos * rot;
    const auto written = [&](const void *a, size_t n) { return overlap(q_out, q_bytes, a, n) || (k_heads > 0 && overlap(k_out, k_bytes, a, n)); };
    if (written(q_norm_w, weights) || (k_heads > 0 && written(k_norm_w, weights)) || written(positions, places) || written(table, angles))
        return api_error(TS_ERR_INVALID_ARG, "an output overlaps a norm's weights, the positions or the table");
    tshc::LaunchCfg cfg;
    tshc::NormRopeParams p{};
    TS_TRY(device(&cfg, &p.r.status));
    p.r.q = static_cast<const uint16_t *>(q);
    p.r.k = static_cast<const uint16_t *>(k);
    p.r.q_out = static_cast<uint16_t *>(q_out);
    p.r.k_out = static_cast<uint16_t *>(k_out);
    p.r.q_stride = q_stride;
    p.r.k_stride = k_stride;
    p.r.q_out_stride = q_out_stride;
    p.r.k_out_stride = k_out_stride;
    p.r.positions = positions;
    p.r.table = table;
    p.r.max_pos = max_pos;
    p.r.N = N;
    p.r.q_heads = q_heads;
    p.r.k_heads = k_heads;
    p.r.D = D;
    p.r.rot = rot;
    p.r.interleaved = interleaved != 0;
    p.qw = static_cast<const uint16_t *>(q_norm_w);
    p.kw = static_cast<const uint16_t *>(k_norm_w);
    p.eps = eps;
    return launched(tshc::launch_qk_norm_rope(p, cfg, stream), "launching the head norm kernel");
}

ts_status ts_hc_prompt_attention(const void *q, long q_stride, const void *k, long k_stride, const void *v, long v_stride,
                                 const int32_t *starts, void *out, float *lse, int N, int S, int q_heads, int kv_heads, int D, float scale,
                                 cudaStream_t stream)
{
    tshc::clear_error();
    TS_TRY(check_count(N, "N", 0, INT_MAX));
    TS_TRY(check_count(S, "S", 0, kMaxBatch));
    TS_TRY(check_count(q_heads, "q_heads", 1, kMaxHeads));
    TS_TRY(check_count(kv_heads, "kv_heads", 1, kMaxHeads));
    if (q_heads % kv_heads != 0)
        return api_error(TS_ERR_INVALID_ARG, "q_heads = %d must be a multiple of kv_heads = %d", q_heads, kv_heads);
    if (D != 64 && D != 128)
        return api_error(TS_ERR_UNSUPPORTED, "D = %d: heads of 64 and 128 are supported", D);
    if (!(scale > 0.f) || !std::isfinite(scale))
        return api_error(TS_ERR_INVALID_ARG, "scale = %g must be > 0", (double)scale);
    if (N == 0 || S == 0)
        return TS_OK;
    const long qw = (long)q_heads * D, kw = (long)kv_heads * D;
    TS_TRY(check_ptr_api(q, "q", 16));
    TS_TRY(check_ptr_api(k, "k", 16));
    TS_TRY(check_ptr_api(v, "v", 16));
    TS_TRY(check_stride(q_stride, "q_stride", qw, 8));
    TS_TRY(check_stride(k_stride, "k_stride", kw, 8));
    TS_TRY(check_stride(v_stride, "v_stride", kw, 8));
    TS_TRY(check_ptr_api(starts, "starts", 4));
    TS_TRY(check_ptr_api(out, "out", 16));
    if (lse)
        TS_TRY(check_ptr_api(lse, "lse", 4));
    if (rows_overlap(out, qw, qw, q, q_stride, qw, N))
        return api_error(TS_ERR_INVALID_ARG, "out overlaps q");
    if (rows_overlap(out, qw, qw, k, k_stride, kw, N))
        return api_error(TS_ERR_INVALID_ARG, "out overlaps k");
    if (rows_overlap(out, qw, qw, v, v_stride, kw, N))
        return api_error(TS_ERR_INVALID_ARG, "out overlaps v");
    const Part written[] = {{out, span(N, qw, qw, 2), "out"}, {lse, lse ? sizeof(float) * (size_t)N * q_heads : 0, "lse"}};
    const Part rows[] = {{q, span(N, q_stride, qw, 2), "q"}, {k, span(N, k_stride, kw, 2), "k"}, {v, span(N, v_stride, kw, 2), "v"}};
    const Part places[] = {{starts, sizeof(int32_t) * ((size_t)S + 1), "starts"}}, lse_alone[] = {written[1]};
    TS_TRY(check_apart(written, places));
    TS_TRY(check_apart(lse_alone, rows));
    if (tshc::prompt_attn_blocks(N, S, q_heads, kv_heads) > INT_MAX)
        return api_error(TS_ERR_UNSUPPORTED, "%d tokens of %d heads are too many for one call: split them", N, q_heads);
    tshc::LaunchCfg cfg;
    tshc::PromptAttnParams p{};
    TS_TRY(device(&cfg, &p.status));
    p.v = static_cast<const uint16_t *>(v);
    p.v_stride = v_stride;
    p.starts = starts;
    p.out = static_cast<uint16_t *>(out);
    p.lse = lse;
    p.N = N;
    p.S = S;
    p.q_heads = q_heads;
    p.kv_heads = kv_heads;
    p.scale_log2 = scale * 1.4426950408889634f;
    return launched(tshc::launch_prompt_attention(p, static_cast<const uint16_t *>(q), q_stride, static_cast<const uint16_t *>(k), k_stride, D, cfg,
                                                  stream),
                    "launching the prompt attention kernel");
}

ts_status ts_hc_delta_step(const void *q, long q_stride, const void *k, long k_stride, const void *v, long v_stride, const float *decay,
                           const float *beta, const int32_t *counts, const float *state_in, float *state_out, void *out, int B, int T,
                           int k_heads, int v_heads, int D, float scale, float norm_eps, cudaStream_t stream)
{
    tshc::clear_error();
    TS_TRY(check_count(B, "B", 0, kMaxBatch));
    TS_TRY(check_count(T, "T", 0, 4096));
    TS_TRY(check_delta_heads(k_heads, v_heads, D));
    TS_TRY(check_scale(scale, norm_eps));
    if (B == 0 || T == 0)
        return TS_OK;
    TS_TRY(check_delta_rows(q, q_stride, k, k_stride, v, v_stride, decay, beta, out, B * T, k_heads, v_heads, D));
    TS_TRY(check_states(state_in, state_out, B, v_heads, D, out, span(B * T, (long)v_heads * D, (long)v_heads * D, 2)));
    if (counts)
        TS_TRY(check_ptr_api(counts, "counts", 4));
    const long kw = (long)k_heads * D, vw = (long)v_heads * D;
    const size_t gates = sizeof(float) * (size_t)B * T * v_heads;
    const Part written[] = {{state_out, sizeof(float) * (size_t)B * vw * D, "state_out"}}, outs[] = {{out, span(B * T, vw, vw, 2), "out"}};
    const Part read[] = {{q, span(B * T, q_stride, kw, 2), "q"}, {k, span(B * T, k_stride, kw, 2), "k"}, {v, span(B * T, v_stride, vw, 2), "v"},
                         {decay, gates, "decay"}, {beta, gates, "beta"}, {counts, counts ? sizeof(int32_t) * (size_t)B : 0, "counts"}};
    const Part counted[] = {read[5]};
    TS_TRY(check_apart(written, read));
    TS_TRY(check_apart(outs, counted));
    tshc::LaunchCfg cfg;
    tshc::DeltaStepParams p{};
    TS_TRY(device(&cfg, &p.status));
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.decay = decay;
    p.beta = beta;
    p.counts = counts;
    p.state_in = state_in;
    p.state_out = state_out;
    p.out = static_cast<uint16_t *>(out);
    p.B = B;
    p.T = T;
    p.Hk = k_heads;
    p.Hv = v_heads;
    p.D = D;
    p.scale = scale;
    p.norm_eps = norm_eps;
    return launched(tshc::launch_delta_step(p, cfg, stream), "launching the delta rule's step kernel");
}

size_t ts_hc_delta_prompt_workspace_bytes(int N, int S, int k_heads, int v_heads, int D)
{
    if (check_count(N, "N", 0, INT_MAX) != TS_OK || check_count(S, "S", 0, kMaxBatch) != TS_OK || check_delta_heads(k_heads, v_heads, D) != TS_OK)
        return 0;
    return tshc::delta_prompt_bytes(N, S, k_heads, v_heads, D);
}

ts_status ts_hc_delta_prompt(const void *q, long q_stride, const void *k, long k_stride, const void *v, long v_stride, const float *decay,
                             const float *beta, const int32_t *starts, const float *state_in, float *state_out, void *out, int N, int S,
                             int k_heads, int v_heads, int D, float scale, float norm_eps, void *workspace, size_t workspace_bytes,
                             cudaStream_t stream)
{
    tshc::clear_error();
    TS_TRY(check_count(N, "N", 0, INT_MAX));
    TS_TRY(check_count(S, "S", 0, kMaxBatch));
    TS_TRY(check_delta_heads(k_heads, v_heads, D));
    TS_TRY(check_scale(scale, norm_eps));
    if (N == 0 || S == 0)
        return TS_OK;
    TS_TRY(check_delta_rows(q, q_stride, k, k_stride, v, v_stride, decay, beta, out, N, k_heads, v_heads, D));
    TS_TRY(check_states(state_in, state_out, S, v_heads, D, out, span(N, (long)v_heads * D, (long)v_heads * D, 2)));
    TS_TRY(check_ptr_api(starts, "starts", 4));
    if (((long)N / 64 + S) * v_heads > INT_MAX)
        return api_error(TS_ERR_UNSUPPORTED, "%d tokens of %d heads are too many for one call: split them", N, v_heads);
    const size_t need = tshc::delta_prompt_bytes(N, S, k_heads, v_heads, D);
    if (!workspace || workspace_bytes < need)
        return api_error(TS_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", workspace ? workspace_bytes : (size_t)0, need);
    TS_TRY(check_ptr_api(workspace, "workspace", 256));
    const long kw = (long)k_heads * D, vw = (long)v_heads * D;
    const size_t gates = sizeof(float) * (size_t)N * v_heads, states = sizeof(float) * (size_t)S * vw * D;
    const Part written[] = {{state_out, states, "state_out"}, {workspace, need, "workspace"}}, outs[] = {{out, span(N, vw, vw, 2), "out"}};
    const Part read[] = {{q, span(N, q_stride, kw, 2), "q"}, {k, span(N, k_stride, kw, 2), "k"}, {v, span(N, v_stride, vw, 2), "v"},
                         {decay, gates, "decay"}, {beta, gates, "beta"}, {starts, sizeof(int32_t) * ((size_t)S + 1), "starts"}};
    const Part apart[] = {read[5], written[1]}, states_in[] = {{state_in, states, "state_in"}}, work[] = {written[1]};
    TS_TRY(check_apart(written, read));
    TS_TRY(check_apart(outs, apart));
    TS_TRY(check_apart(work, states_in));
    tshc::LaunchCfg cfg;
    tshc::DeltaPromptParams p{};
    TS_TRY(device(&cfg, &p.status));
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.decay = decay;
    p.beta = beta;
    p.starts = starts;
    p.state_in = state_in;
    p.state_out = state_out;
    p.out = static_cast<uint16_t *>(out);
    p.work = static_cast<uint8_t *>(workspace);
    p.N = N;
    p.S = S;
    p.Hk = k_heads;
    p.Hv = v_heads;
    p.D = D;
    p.scale = scale;
    p.norm_eps = norm_eps;
    return launched(tshc::launch_delta_prompt(p, cfg, stream), "launching the delta rule's prompt kernels");
}

ts_status ts_hc_logprobs(const void *logits, int logits_type, long logits_stride, const int32_t *tokens, float *logp, float *entropy,
                         int32_t *top_ids, float *top_logp, int N, int V, int J, int top, cudaStream_t stream)
{
    tshc::clear_error();
    TS_TRY(check_count(N, "N", 0, INT_MAX));
    TS_TRY(check_count(V, "V", 1, (1 << 30) - 1));
    TS_TRY(check_count(J, "J", 0, INT_MAX));
    TS_TRY(check_count(top, "top", 0, V < 32 ? V : 32));
    if (logits_type != TS_LOGITS_FP32 && logits_type != TS_LOGITS_BF16)
        return api_error(TS_ERR_INVALID_ARG, "logits_type = %d is not a ts_logits_type", logits_type);
    if (N == 0)
        return TS_OK;
    const size_t size = logits_type == TS_LOGITS_BF16 ? 2 : 4;
    TS_TRY(check_ptr_api(logits, "logits", size));
    TS_TRY(check_stride(logits_stride, "logits_stride", V, 1));
    if (J > 0) {
        TS_TRY(check_ptr_api(tokens, "tokens", 4));
        TS_TRY(check_ptr_api(logp, "logp", 4));
    }
    if (entropy)
        TS_TRY(check_ptr_api(entropy, "entropy", 4));
    if (top > 0) {
        TS_TRY(check_ptr_api(top_ids, "top_ids", 4));
        TS_TRY(check_ptr_api(top_logp, "top_logp", 4));
    }
    if (J == 0 && !entropy && top == 0)
        return api_error(TS_ERR_INVALID_ARG, "nothing is asked for: no tokens, no entropy and no alternatives");
    const struct { const void *p; size_t n; const char *name; } outs[] = {
        {J > 0 ? logp : nullptr, sizeof(float) * (size_t)N * J, "logp"},
        {entropy, sizeof(float) * (size_t)N, "entropy"},
        {top > 0 ? top_ids : nullptr, sizeof(int32_t) * (size_t)N * top, "top_ids"},
        {top > 0 ? top_logp : nullptr, sizeof(float) * (size_t)N * top, "top_logp"}};
    for (int i = 0; i < 4; ++i) {
        if (!outs[i].p)
            continue;
        if (overlap(outs[i].p, outs[i].n, logits, span(N, logits_stride, V, size)))
            return api_error(TS_ERR_INVALID_ARG, "%s overlaps logits", outs[i].name);
        if (J > 0 && overlap(outs[i].p, outs[i].n, tokens, sizeof(int32_t) * (size_t)N * J))
            return api_error(TS_ERR_INVALID_ARG, "%s overlaps tokens", outs[i].name);
        for (int j = i + 1; j < 4; ++j)
            if (outs[j].p && overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
                return api_error(TS_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, outs[j].name);
    }
    tshc::LaunchCfg cfg;
    tshc::LogprobParams p{};
    TS_TRY(device(&cfg, &p.status));
    p.logits = logits;
    p.stride = logits_stride;
    p.tokens = tokens;
    p.logp = logp;
    p.entropy = entropy;
    p.top_ids = top_ids;
    p.top_logp = top_logp;
    p.N = N;
    p.V = V;
    p.J = J;
    p.top = top;
    return launched(tshc::launch_logprobs(p, logits_type == TS_LOGITS_BF16, cfg, stream), "launching the log probability kernel");
}

}  // extern "C"
