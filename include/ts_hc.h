/*
 * ts_hc.h -- C ABI of the GB300 (sm_103a) hyper-connection residual call.
 *
 * The operations are those of the qwen4_exp decode flow in the
 * turbospark-runtime 0.3.0 source pages:
 *   - families/qwen4/mod.rs, module doc, "## Hyper-connections": one call maps
 *     the C*H-wide residual `raw` to the H-wide `mixed` and the C-wide gate
 *     `inject_w`;
 *   - families/qwen4/mod.rs, decoder-layer pseudocode and "THE INJECTION
 *     TRAP": the inject-add onto the un-normalized residual;
 *   - families/qwen4/mod.rs, the paragraph on the final
 *     `hyper_connection_mixer` (the call without block_inject_weight);
 *   - families/qwen4/hc.rs, `encode_hyper_connection`: step order, weight
 *     shapes (rows = outputs, cols = inputs) and the per-token inject row.
 *
 * Conventions shared by every entry point
 *   - All tensor pointers are DEVICE pointers owned by the caller. The library
 *     allocates nothing and keeps no state beyond per-device attributes it
 *     queries once. Every call is asynchronous on `stream` (0 = legacy default
 *     stream).
 *   - Row-major everywhere. A wide vector has C*H elements; stream c occupies
 *     elements [c*H, (c+1)*H). Linear weights are [out][in] with no bias.
 *   - bf16 tensors are 16-byte aligned; H is a multiple of 8, hc_lowrank (L)
 *     a multiple of 8 (32 for INT4 weights); 1 <= C <= 8; 8 <= L <= 1024.
 *   - M == 0 (no tokens) is a no-op for every entry point: once the shape
 *     arguments are valid it returns TS_OK without examining any pointer.
 *   - Arguments are validated on the host before anything is launched; a bad
 *     argument returns an error status without launching, and
 *     ts_hc_last_error() names it. Launch failures return TS_ERR_CUDA.
 *   - Results of the GPU path are deterministic: the same inputs give the same
 *     bits on every run (fixed-order split-K reductions, no float atomics).
 *   - A kernel that waits on an asynchronous copy gives up after about one
 *     second, records TS_ERR_TIMEOUT in a device-side status word and returns
 *     without hanging; read it with ts_hc_device_status().
 */
#ifndef TS_HC_H
#define TS_HC_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    TS_OK = 0,
    TS_ERR_INVALID_ARG = 1,   /* null / misaligned pointer, bad size or stride */
    TS_ERR_UNSUPPORTED = 2,   /* valid request outside what this build supports */
    TS_ERR_CUDA = 3,          /* a CUDA runtime call or launch failed */
    TS_ERR_WORKSPACE = 4,     /* workspace missing or smaller than ts_hc_workspace_bytes() */
    TS_ERR_TIMEOUT = 5        /* a device-side wait gave up (see ts_hc_device_status) */
} ts_status;

typedef enum {
    TS_W_BF16 = 0,            /* data: bf16 [out][in] */
    TS_W_INT4_AFFINE = 1      /* data: uint8 [out][in/2], element 2i in the low nibble of
                                 byte i; scales, biases: fp16 [out][in/group];
                                 weight = q * scale + bias, q in [0, 15] */
} ts_wtype;

/* A linear weight [out][in] in its storage format (real_forward.rs,
 * RealForwardRunner doc: projections are INT4-affine quantised or dense). */
typedef struct {
    int32_t type;             /* ts_wtype */
    int32_t group;            /* INT4: inputs per (scale, bias) group: 32, 64 or 128 */
    const void *data;
    const void *scales;       /* INT4 only, else NULL */
    const void *biases;       /* INT4 only, else NULL */
} ts_weight;

/*
 * Bytes of device workspace ts_hc_call / ts_hc_mixer need for M tokens
 * (0 for invalid shapes). The workspace is caller-owned scratch: it need not
 * be initialised, is overwritten by every call, and must not be shared by two
 * calls that can run at the same time.
 *
 * After a successful call the workspace holds two fp32 intermediates of the
 * last call, at the byte offsets ts_hc_workspace_layout() reports:
 *   inv_rms [M][C]: 1/sqrt(mean_h raw[m][c*H+h]^2 + eps), per token and stream;
 *   act     [M][L]: silu(input_mix_weight_down(normed) / C).
 */
size_t ts_hc_workspace_bytes(int M, int H, int C, int lowrank);
ts_status ts_hc_workspace_layout(int M, int H, int C, int lowrank,
                                 size_t *inv_rms_offset, size_t *act_offset);

/*
 * One hyper-connection call (attn_hc / mlp_hc) on M independent tokens
 * (families/qwen4/mod.rs "## Hyper-connections"; families/qwen4/hc.rs
 * encode_hyper_connection):
 *
 *   normed  = hc_norm(raw)                 grouped RMS, group = H, eps inside
 *                                          the root, scale applied directly
 *   act     = silu(down(normed) / C)       C*H -> L
 *   w       = sigmoid(up(act))             L -> C*H, no division
 *   mixed   = mean_c(w[c*H+h] * normed[c*H+h])
 *   gate    = 2 * sigmoid(inject(normed) / C)
 *
 *   raw        bf16 [M][C*H], read only (the caller injects separately)
 *   hc_norm_w  bf16 [C*H] (hc_norm.weight)
 *   down       [L][C*H]   (input_mix_weight_down.weight)
 *   up         [C*H][L]   (input_mix_weight_up.weight)
 *   inject     [C][C*H]   (block_inject_weight.weight)
 *   mixed      bf16 [M][H], written (rounded to nearest even)
 *   inject_w   fp32; token t's C gates are written at inject_w + t*inject_stride
 *              (inject_stride >= C; 2*C with a +C base offset for mlp_hc gives
 *              the per-token row t*C*2 of a shared micro-batch gate buffer)
 *   eps        RMS epsilon (the pages use 1e-6)
 *   workspace  >= ts_hc_workspace_bytes(M, H, C, lowrank) bytes, 256-byte aligned
 *
 * M == 0 is a no-op. Returns TS_OK or an error status (nothing launched on
 * argument errors).
 */
ts_status ts_hc_call(const void *raw, const void *hc_norm_w,
                     const ts_weight *down, const ts_weight *up, const ts_weight *inject,
                     void *mixed, float *inject_w, long inject_stride,
                     int M, int H, int C, int lowrank, float eps,
                     void *workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * The inject-add (families/qwen4/mod.rs decoder pseudocode and THE INJECTION
 * TRAP): raw[m][c*H+h] += out[m][h] * inject_w[m*inject_stride + c], in place
 * on the UN-normalized residual, computed in fp32 and rounded to bf16 (nearest
 * even).
 *
 *   raw       bf16 [M][C*H], read and written
 *   out       bf16 [M][H], the sublayer output
 *   inject_w  fp32, token m's gates at inject_w + m*inject_stride (inject_stride >= C)
 */
ts_status ts_hc_inject_add(void *raw, const void *out, const float *inject_w,
                           long inject_stride, int M, int H, int C, cudaStream_t stream);

/*
 * The final hyper_connection_mixer (families/qwen4/mod.rs, paragraph after the
 * hyper-connection pseudocode; families/qwen4/hc.rs, has_inject_gate = false):
 * ts_hc_call without block_inject_weight. Writes `mixed` bf16 [M][H] only.
 */
ts_status ts_hc_mixer(const void *raw, const void *hc_norm_w,
                      const ts_weight *down, const ts_weight *up,
                      void *mixed, int M, int H, int C, int lowrank, float eps,
                      void *workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * Test and debugging aid: ts_hc_call (or, with inject == NULL, ts_hc_mixer)
 * that also writes w, the output of the up projection's sigmoid
 * (families/qwen4/mod.rs, "## Hyper-connections": w = sigmoid(up(act)), the
 * per-element mixing weight that multiplies normed before the mean over the
 * streams). The regular entry points keep w on chip.
 *
 *   w_out  fp32 [M][C*H], written: element m*C*H + c*H + h is token m's
 *          weight for stream c at h (the values the same launch mixes)
 *   inject, inject_w, inject_stride  as for ts_hc_call; inject may be NULL
 *          (the exit mixer), and then inject_w is not used
 * Every other output (mixed, the gates, the workspace intermediates) is bit
 * for bit what ts_hc_call / ts_hc_mixer writes for the same inputs: the same
 * kernels run, with one extra store per element of w.
 */
ts_status ts_hc_call_debug(const void *raw, const void *hc_norm_w,
                           const ts_weight *down, const ts_weight *up, const ts_weight *inject,
                           void *mixed, float *inject_w, long inject_stride,
                           int M, int H, int C, int lowrank, float eps,
                           void *workspace, size_t workspace_bytes, float *w_out,
                           cudaStream_t stream);

/*
 * ts_hc_call for callers that cannot allocate device memory. The pages have
 * no counterpart to this entry point; it exists for this library's users.
 *
 * Some callers cannot call cudaMalloc (or any allocator) at the point where
 * they run the call: real-time loops that must not hit the implicit
 * synchronisation an allocation can cause, and hosts that hand this library a
 * fixed memory budget and no allocator. They pass inputs and outputs
 * as for ts_hc_call but no workspace: the scratch lives in a file-scope device
 * array of TS_HC_STATIC_SCRATCH_BYTES that every GPU which loads this library
 * holds until the process exits.
 *
 *   - Shapes whose ts_hc_workspace_bytes() exceeds TS_HC_STATIC_SCRATCH_BYTES
 *     are refused with TS_ERR_WORKSPACE before anything is launched (at the
 *     full shape H=2560, C=4, lowrank=320 that allows up to 1373 tokens).
 *   - The first call on each device looks up the array's device address (with
 *     that device current); make that first call before any stream capture.
 *   - Every call on a device shares the one array and leaves its contents
 *     behind. Nothing in it needs to start at zero: each call writes every
 *     scratch byte it reads. Calls that can overlap on the GPU (other streams,
 *     other threads) race on it; serialise them.
 *   - Allocates nothing: no cudaMalloc, cudaFree or allocating library call.
 *
 * Arguments and results as for ts_hc_call, without workspace/workspace_bytes.
 */
#define TS_HC_STATIC_SCRATCH_BYTES (64u * 1024u * 1024u)
ts_status ts_hc_call_noalloc(const void *raw, const void *hc_norm_w,
                             const ts_weight *down, const ts_weight *up, const ts_weight *inject,
                             void *mixed, float *inject_w, long inject_stride,
                             int M, int H, int C, int lowrank, float eps, cudaStream_t stream);

/*
 * The previous sublayer's inject-add fused into the next call
 * (families/qwen4/mod.rs, decoder pseudocode: each `hidden = raw + out * inject_w`
 * is immediately followed by the next attn_hc / mlp_hc, or by the exit mixer).
 * Equivalent, bit for bit, to
 *     ts_hc_inject_add(raw, out, prev_inject_w, prev_inject_stride, ...);
 *     ts_hc_call(raw, ...)            (or ts_hc_mixer when inject == NULL)
 * but with one kernel fewer on the dependency chain: the call reads
 * raw + out * prev_gate directly and writes the updated residual back to raw.
 *
 *   raw            bf16 [M][C*H], read and written (in place)
 *   out            bf16 [M][H], the sublayer output
 *   prev_inject_w  fp32, token m's previous gates at prev_inject_w + m*prev_inject_stride
 *   inject         may be NULL: then this is the exit mixer and inject_w is unused
 *   inject_w       must not share an element with prev_inject_w (two slots of a
 *                  [M][2][C] micro-batch buffer are fine); refused otherwise
 * Other arguments as for ts_hc_call.
 */
ts_status ts_hc_inject_call(void *raw, const void *out, const float *prev_inject_w, long prev_inject_stride,
                            const void *hc_norm_w, const ts_weight *down, const ts_weight *up,
                            const ts_weight *inject, void *mixed, float *inject_w, long inject_stride,
                            int M, int H, int C, int lowrank, float eps,
                            void *workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * The decoder's exit (families/qwen4/mod.rs, decoder pseudocode, exit lines:
 * hidden = hyper_connection_mixer(hidden); logits = lm_head(hidden), with no
 * softcap and no separate final norm), with the last sublayer's inject-add
 * fused in front when `out` is given:
 *     raw += out * prev_inject_w                    (only if out != NULL)
 *     mixed = hyper_connection_mixer(raw)           bf16 [M][H]
 *     logits[m][v] = sum_h lm_head[v][h] * mixed[m][h]   (fp32, mixed as stored)
 * lm_head runs on the tensor cores (bf16 operands, fp32 accumulation) in
 * launches of at most 16 tokens; each launches as a programmatic dependent of
 * the kernel before it and streams its first weight tiles before that kernel
 * has finished. With one token the mixer's up kernel also asks L2 to prefetch
 * the first 24 MB of lm_head while the mixer runs.
 *
 *   raw             bf16 [M][C*H]; read, and written with the fused inject-add
 *   out, prev_inject_w, prev_inject_stride   as for ts_hc_inject_call, or
 *                   out == NULL (then the other two are not used)
 *   hc_norm_w, down, up   the exit mixer's module (no inject weight)
 *   lm_head         bf16 [V][H] (lm_head.weight), 16-byte aligned
 *   mixed           bf16 [M][H], written (the lm_head reads it back)
 *   logits          fp32 [M][V], written
 * Other arguments as for ts_hc_mixer; the workspace is ts_hc_workspace_bytes(M, ...).
 * Any V >= 1 is taken; H must be a multiple of 64 (TS_ERR_UNSUPPORTED
 * otherwise), the other shape rules are those of ts_hc_mixer.
 */
ts_status ts_hc_exit_logits(void *raw, const void *out, const float *prev_inject_w, long prev_inject_stride,
                            const void *hc_norm_w, const ts_weight *down, const ts_weight *up,
                            const void *lm_head, int V, void *mixed, float *logits,
                            int M, int H, int C, int lowrank, float eps,
                            void *workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * PLE, the per-layer embedding gate on the wide residual (families/qwen4/mod.rs,
 * "## PLE": added to the residual before layer index 1's attn_hc, and only
 * there). For M consecutive tokens of one sequence:
 *   emb   = concat of the 16 table rows rows[m][0..16), each H/16 wide
 *   key   = norm_key(key_proj(emb))        value = value_proj(emb)
 *   query = norm_query(hidden)
 *   gate  = sigmoid(s * sqrt(max(|d|, 1e-6))), d = sum_h key[c][h] query[c][h] / sqrt(H),
 *           s the sign of d, per stream c
 *   gv    = gate * value                   (value broadcast to every stream)
 *   hidden += gv + silu(conv(norm_conv(gv)))    (rounded to bf16, in place)
 * The norms are grouped RMS norms in the hyper-connection norm's form (groups
 * of H, eps inside the root, a direct scale per element). conv is depthwise and
 * causal along the token axis: channel j of token t is
 * sum_i conv_w[j][i] * x[t - 3*(3 - i)][j], dilation 3, four taps; the inputs
 * of the 9 tokens before the chunk come from conv_state, which is updated to
 * the chunk's last 9 (zero it for a new sequence). The page notes that this
 * formula was not cross-checked upstream; the hash that picks the row ids is
 * not on the pages, so the caller supplies them.
 *
 *   hidden           bf16 [M][C*H], read and written
 *   rows             int32 [M][16], each in [0, n_rows); an id out of range reads
 *                    zeros and records TS_ERR_INVALID_ARG in the device status word
 *   table            bf16 [n_rows][H/16]
 *   key_proj         bf16 [C*H][H];  value_proj  bf16 [H][H]
 *   norm_*_w         bf16 [C*H] each
 *   conv_w           bf16 [C*H][4]
 *   conv_state       fp32 [9][C*H], oldest token first; read and written
 *   H                a multiple of 128
 *   workspace        >= ts_hc_ple_workspace_bytes(M, H, C) bytes, 256-byte
 *                    aligned; after the call it holds value fp32 [M][H], the
 *                    gates fp32 [M][C] and the conv input x fp32 [M][C*H] at the
 *                    offsets ts_hc_ple_workspace_layout() reports
 */
size_t ts_hc_ple_workspace_bytes(int M, int H, int C);
ts_status ts_hc_ple_workspace_layout(int M, int H, int C, size_t *value_offset, size_t *gate_offset,
                                     size_t *x_offset);
ts_status ts_hc_ple(void *hidden, const int32_t *rows, const void *table, long n_rows,
                    const void *key_proj, const void *value_proj, const void *norm_key_w,
                    const void *norm_query_w, const void *norm_conv_w, const void *conv_w,
                    float *conv_state, int M, int H, int C, float eps,
                    void *workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * Entry replication fused into the stack's first call (families/qwen4/mod.rs,
 * decoder pseudocode: the entry line hidden = embed_tokens(ids).repeat(1, 1, C),
 * followed by layer 0's attn_hc). Equivalent, bit for bit, to
 *     ts_hc_replicate_entry(emb, raw, M, H, C, stream);
 *     ts_hc_call(raw, ...)            (or ts_hc_mixer when inject == NULL)
 * with one kernel fewer: the call reads every stream from the embedding row
 * and writes the replicated residual to raw.
 *
 *   emb   bf16 [M][H], read
 *   raw   bf16 [M][C*H], written (must not overlap emb; refused otherwise)
 * Other arguments as for ts_hc_call; inject may be NULL (then inject_w is not used).
 */
ts_status ts_hc_entry_call(const void *emb, void *raw, const void *hc_norm_w,
                           const ts_weight *down, const ts_weight *up, const ts_weight *inject,
                           void *mixed, float *inject_w, long inject_stride,
                           int M, int H, int C, int lowrank, float eps,
                           void *workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * Entry replication (families/qwen4/mod.rs, decoder pseudocode, entry line:
 * the embedding row is repeated C times, not padded):
 * raw[m][c*H + h] = emb[m][h] for every stream c.
 *
 *   emb  bf16 [M][H], read
 *   raw  bf16 [M][C*H], written
 */
ts_status ts_hc_replicate_entry(const void *emb, void *raw, int M, int H, int C, cudaStream_t stream);

/*
 * The decoder stack's hyper-connection path, driven over a prompt in chunks
 * (families/qwen4/mod.rs, decoder-layer pseudocode: entry replication, per
 * layer attn_hc -> sublayer -> inject-add -> mlp_hc -> sublayer -> inject-add,
 * exit hyper_connection_mixer; real_forward.rs, the chunked-prefill driver that
 * runs a prompt through the layers a micro-batch of rows at a time).
 *
 * Tokens do not interact in this path, so the T tokens are processed in
 * chunks of at most max_chunk tokens, one after the other. For each chunk of
 * M tokens starting at token t0:
 *   raw = repeat(emb[t0 .. t0+M), C), fused into layer 0's attn_hc   ts_hc_entry_call
 *   for layer l: attn_hc(attn[l]) -> sublayer(l, 0) -> mlp_hc(mlp[l]) -> sublayer(l, 1),
 *                each inject-add fused into the call after it   ts_hc_inject_call
 *   mixed_out[t0 .. t0+M) = hyper_connection_mixer(final)   (fused with the last inject-add)
 * attn_hc writes token t's gates to slot 0 and mlp_hc to slot 1 of a
 * [M][2][C] gate buffer, i.e. at element t*C*2 and t*C*2 + C (hc.rs,
 * inject_row_offset).
 *
 * The sublayers (GDN / QSA attention, MoE) are the caller's: after every
 * hyper-connection call the driver calls
 *     sublayer(user, layer, which, t0, M, mixed, &out, stream)
 * with `mixed` the call's output (bf16 [M][H], device, valid in stream order
 * until the driver's next launch) and which = 0 after attn_hc, 1 after mlp_hc.
 * The callback may enqueue work on `stream`; it sets `out` to a 16-byte aligned
 * device buffer bf16 [M][H] holding the sublayer output, outside the workspace,
 * which must stay valid until the next hyper-connection call has read it (in
 * stream order). A status other than TS_OK, or a NULL, misaligned or
 * workspace-overlapping `out`, stops the driver, which returns an error; work
 * launched before that point stays queued.
 *
 *   emb        bf16 [T][H], the embedding rows
 *   attn, mlp  n_layers modules each; their inject weights are required
 *   final      the exit mixer's module; its inject is not read
 *   mixed_out  bf16 [T][H], written
 *   max_chunk  >= 1 tokens per chunk
 *   workspace  >= ts_hc_stack_workspace_bytes(max_chunk, H, C, lowrank) bytes,
 *              256-byte aligned; on return it begins with the last chunk's
 *              residual bf16 [M][C*H] after its last inject-add
 * Every module's tensors are validated before anything is launched. The driver
 * allocates nothing and never synchronises, so a caller may capture the whole
 * pass into a CUDA graph when its callback's work is capturable. T == 0 is a
 * no-op.
 */
typedef struct {
    const void *hc_norm_w;    /* bf16 [C*H] */
    ts_weight down;           /* [lowrank][C*H] */
    ts_weight up;             /* [C*H][lowrank] */
    ts_weight inject;         /* [C][C*H]; not read for the exit mixer */
} ts_hc_module;

/*
 * A stack's PLE module (families/qwen4/mod.rs, "## PLE"), the tensors ts_hc_ple
 * takes: table bf16 [n_rows][H/16]; key_proj bf16 [C*H][H]; value_proj bf16
 * [H][H]; norm_key_w, norm_query_w, norm_conv_w bf16 [C*H] each; conv_w bf16
 * [C*H][4]. Every pointer 16-byte aligned.
 */
typedef struct {
    const void *table;
    long n_rows;
    const void *key_proj;
    const void *value_proj;
    const void *norm_key_w;
    const void *norm_query_w;
    const void *norm_conv_w;
    const void *conv_w;
} ts_hc_ple_module;

typedef ts_status (*ts_hc_sublayer_fn)(void *user, int layer, int which, int t0, int M,
                                       const void *mixed, const void **out, cudaStream_t stream);

size_t ts_hc_stack_workspace_bytes(int max_chunk, int H, int C, int lowrank);
ts_status ts_hc_stack(const void *emb, int T, const ts_hc_module *attn, const ts_hc_module *mlp,
                      int n_layers, const ts_hc_module *final_mixer, ts_hc_sublayer_fn sublayer,
                      void *user, void *mixed_out, int max_chunk, int H, int C, int lowrank,
                      float eps, void *workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * ts_hc_stack with the PLE gate at layer index 1 (families/qwen4/mod.rs, decoder
 * pseudocode: `if layer_idx == 1: hidden = hidden + ple(hidden, input_ids)`
 * before that layer's attn_hc). For each chunk, layer 0's last inject-add is
 * applied on its own (ts_hc_inject_add), then ts_hc_ple on the residual, then
 * layer 1's attn_hc (ts_hc_call); every other step is as in ts_hc_stack.
 *
 *   ple             the PLE module (all of it validated before any launch)
 *   ple_rows        int32 [T][16], token t's 16 table row ids
 *   ple_conv_state  fp32 [9][C*H], the conv inputs of the 9 tokens before token 0
 *                   (zero for a new sequence); read and updated chunk by chunk, so
 *                   on return it holds the last 9 tokens' inputs
 *   n_layers        >= 2 (the PLE layer must exist)
 *   H               a multiple of 128
 *   workspace       >= ts_hc_stack_ple_workspace_bytes(max_chunk, H, C, lowrank)
 * Other arguments and results as for ts_hc_stack.
 */
size_t ts_hc_stack_ple_workspace_bytes(int max_chunk, int H, int C, int lowrank);
ts_status ts_hc_stack_ple(const void *emb, int T, const ts_hc_module *attn, const ts_hc_module *mlp,
                          int n_layers, const ts_hc_module *final_mixer, const ts_hc_ple_module *ple,
                          const int32_t *ple_rows, float *ple_conv_state, ts_hc_sublayer_fn sublayer,
                          void *user, void *mixed_out, int max_chunk, int H, int C, int lowrank,
                          float eps, void *workspace, size_t workspace_bytes, cudaStream_t stream);

/* ---- a speculative decoding step: rotary positions, a quantised cache, tree attention, verification ----
 *
 * What a sublayer and the step around the stack need when a model decodes several drafted tokens at a
 * time. A step has B sequences of T tokens each ("nodes"): node 0 is the last committed token, the
 * others are drafts, a chain or a tree in which a node comes after its parent. The nodes' keys and
 * values lie in the cache at positions ctx_len[b] .. ctx_len[b] + T - 1, after the sequence's
 * ctx_len[b] committed ones. A step runs
 *   ts_hc_tree_build   the nodes' masks and positions from their parents       (once)
 *   ts_hc_rope         turns the query and key heads                           (per layer)
 *   ts_hc_kv_write     stores the keys and values                              (per layer)
 *   ts_hc_tree_attention                                                       (per layer)
 *   ts_hc_verify       on ts_hc_exit_logits' logits: which drafts hold         (once)
 *   ts_hc_kv_compact   moves the accepted nodes' rows to the committed ones    (per layer)
 *
 * Lengths, page ids, parents and tokens are device data, so that a step can be captured in a graph
 * and replayed with other contents. What the host cannot check of them the kernels do: an id, a
 * position or a length out of range is not followed (its row reads zeros and is not written) and
 * TS_ERR_INVALID_ARG is recorded in the device status word (ts_hc_device_status).
 * B == 0 or T == 0 (N == 0, n == 0) is a no-op, as M == 0 is above.
 */

typedef enum {
    TS_ROPE_PLAIN = 0,        /* f_i = theta^(-2i/rot) */
    TS_ROPE_LINEAR = 1,       /* f_i / factor: positions interpolated */
    TS_ROPE_NTK = 2,          /* theta replaced by theta * factor^(rot/(rot-2)) */
    TS_ROPE_BY_PARTS = 3      /* f_i / factor where f_i turns fewer than beta_slow times in
                                 original_positions, f_i where more than beta_fast times, a
                                 blend of the two between, linear in the number of turns (not, as
                                 some programs have it, in i between two rounded indices) */
} ts_rope_scaling_type;

typedef struct {
    int32_t type;             /* ts_rope_scaling_type */
    float factor;             /* > 0 */
    float original_positions; /* BY_PARTS: > 0 */
    float beta_fast;          /* BY_PARTS: > beta_slow */
    float beta_slow;          /* BY_PARTS: >= 0 */
    float magnitude;          /* > 0: multiplies cos and sin (1 for none) */
} ts_hc_rope_scaling;

/*
 * The cosines and sines of a rotary embedding: table fp32 [max_pos][rot/2][2] = (cos, sin) of
 * pos * f_i, times magnitude, with the angle formed and reduced in 64 bits.
 *
 *   table    16-byte aligned, written; rot even, in [2, 1024]; theta > 1
 *   scaling  NULL for TS_ROPE_PLAIN
 */
ts_status ts_hc_rope_table(float *table, int max_pos, int rot, double theta,
                           const ts_hc_rope_scaling *scaling, cudaStream_t stream);

/*
 * Rotary positions for the query and key heads of N tokens, one launch:
 *   (y0, y1) = (x0 c - x1 s, x0 s + x1 c),  (c, s) = table[positions[n]][i],  i < rot/2
 * where pair i is (x[i], x[i + rot/2]) of the head, or (x[2i], x[2i+1]) when interleaved != 0.
 * Elements rot .. D-1 of a head are copied. inverse != 0 turns the other way (s -> -s): the
 * gradient of the operator, and what undoes it (up to rounding) for a magnitude of 1.
 * fp32 arithmetic, rounded to bf16 once.
 *
 *   q, k            bf16: head h of token n at q + n*q_stride + h*D; strides in elements, multiples
 *                   of 8, >= heads*D (a slice of a fused projection's output can be passed);
 *                   k may be NULL with k_heads == 0
 *   q_out, k_out    bf16, laid out likewise with their own strides; q_out == q with the same stride
 *                   turns in place (buffers must not overlap otherwise)
 *   positions       int32 [N], in [0, max_pos)
 *   D               a multiple of 8 in [8, 1024]; rot even, 2 <= rot <= D
 */
ts_status ts_hc_rope(const void *q, long q_stride, const void *k, long k_stride, const int32_t *positions,
                     const float *table, int max_pos, void *q_out, long q_out_stride, void *k_out,
                     long k_out_stride, int N, int q_heads, int k_heads, int D, int rot, int interleaved,
                     int inverse, cudaStream_t stream);

typedef enum {
    TS_KV_BF16 = 0,           /* bf16 [D] */
    TS_KV_FP8 = 1,            /* e4m3 [D] and one scale 2^(byte - 127) a row: the smallest power of two
                                 with max|x| <= 448 * scale, at least 2^-117. Elements beyond +-240 * 2^120,
                                 whose nearest code would be 2^128, are stored as that. Byte 255 marks a row
                                 that held an infinity or a NaN; it reads back as NaN. No code is a NaN, and
                                 code * scale is a finite bf16 */
    TS_KV_INT4 = 2            /* uint8 [D/2], element 2i in the low nibble of byte i, and fp16 scale and
                                 bias per group, as TS_W_INT4_AFFINE: x = q * scale + bias with
                                 scale = (max - min) / 15, bias = min (rounded to fp16; values beyond
                                 +-57344 saturate there), q = round((x - bias) / scale), ties to
                                 even, in [0, 15]. A group that held an infinity or a NaN reads back as NaN */
} ts_kvtype;

/*
 * A paged cache of one layer's keys and values. Position p of sequence b lies in page
 * page_table[b][p / page_size] at place p % page_size. "Row" is one token's vector of one head.
 * Codes are [n_pages][n_kv_heads][page_size][row], scales likewise: FP8 uint8
 * [n_pages][n_kv_heads][page_size], INT4 fp16 [n_pages][n_kv_heads][page_size][head_dim/group].
 */
typedef struct {
    int32_t type;             /* ts_kvtype */
    int32_t group;            /* INT4: 32, 64 or 128, at most head_dim */
    int32_t page_size;        /* a power of two in [16, 1024] */
    int32_t n_kv_heads;       /* [1, 1024] */
    int32_t head_dim;         /* 64, 128 or 256 */
    int32_t max_pages;        /* entries per sequence of page_table */
    long n_pages;
    void *k, *v;              /* 16-byte aligned, as are the scales and biases */
    void *k_scales, *v_scales; /* FP8, INT4; else NULL */
    void *k_biases, *v_biases; /* INT4; else NULL */
    const int32_t *page_table; /* int32 [B][max_pages] */
} ts_hc_kv_cache;

/*
 * Stores T tokens' keys and values of B sequences at positions ctx_len[b] .. ctx_len[b] + T - 1,
 * quantised to the cache's type.
 *   k, v      bf16: head h of token t of sequence b at k + (b*T + t)*k_stride + h*D; strides in
 *             elements, multiples of 8, >= n_kv_heads*D; 16-byte aligned
 *   ctx_len   int32 [B]
 * Two nodes never share a place unless two page-table entries are the same page.
 */
ts_status ts_hc_kv_write(const void *k, long k_stride, const void *v, long v_stride, const ts_hc_kv_cache *cache,
                         const int32_t *ctx_len, int B, int T, cudaStream_t stream);

/*
 * Reads positions start[b] .. start[b] + n - 1 of each sequence back as bf16 [B][n][n_kv_heads][D]
 * (FP8 rows are exact in bf16; INT4's q * scale + bias is formed in fp32 and rounded once).
 */
ts_status ts_hc_kv_read(const ts_hc_kv_cache *cache, const int32_t *start, void *k_out, void *v_out, int B, int n,
                        cudaStream_t stream);

/*
 * After a verification: the rows of the accepted nodes, at ctx_len[b] + path[b][i], move to
 * ctx_len[b] + i for i = 1 .. n_accepted[b] (codes and scales as they are), and new_len[b] =
 * ctx_len[b] + n_accepted[b] + 1. A path ascends, so that no row is overwritten before it is read.
 * A step that does not ascend or has no place ends its path there (recorded): the steps before it are
 * moved, and new_len counts those. With a length or a count out of range nothing is, and new_len = ctx_len.
 *   path         int32 [B][T] and n_accepted int32 [B], as ts_hc_verify writes them
 *   new_len      int32 [B] or NULL; must not overlap ctx_len, n_accepted or path (other blocks still read them)
 */
ts_status ts_hc_kv_compact(const ts_hc_kv_cache *cache, const int32_t *ctx_len, const int32_t *path,
                           const int32_t *n_accepted, int32_t *new_len, int B, int T, cudaStream_t stream);

/*
 * The masks and positions of B trees of T nodes. parents[b*parents_stride + i] is node i's parent,
 * less than i; node 0 is the root (its entry is not read). parents_stride 0 shares one tree. A node
 * i > 0 whose parent is negative is absent: no node sees it and it sees none of them.
 *   mask       uint32 [B][T][(T+31)/32] or NULL: bit j%32 of word j/32 of row i is set where node i
 *              sees node j (itself and its ancestors)
 *   positions  int32 [B][T] or NULL: ctx_len[b] + the node's depth (ctx_len NULL: the depth)
 */
ts_status ts_hc_tree_build(const int32_t *parents, long parents_stride, const int32_t *ctx_len, uint32_t *mask,
                           int32_t *positions, int B, int T, cudaStream_t stream);

/*
 * Attention of B*T nodes over the cache. Head h's keys and values are head h / (q_heads/n_kv_heads)
 * of the cache. Row (b, t, h) sees the positions j < ctx_len[b], and ctx_len[b] + i for the nodes i
 * that its mask row has (mask NULL: i <= t, a chain):
 *   out = softmax_j(scale * q . k_j) v,   lse = log sum_j exp(scale * q . k_j)
 * A row that sees nothing gets zeros and an lse of -infinity. What a row does not see does not
 * reach it, whatever it holds: an infinity or a NaN in an unseen node's key or value (or in a page
 * past the end) changes nothing.
 *   q          bf16: head h of node t of sequence b at q + (b*T + t)*q_stride + h*D (a multiple of 8,
 *              >= q_heads*D), 16-byte aligned
 *   mask       uint32, sequence b's [T][(T+31)/32] at mask + b*mask_stride (words; 0 shares one)
 *   out        bf16 [B][T][q_heads][D], 16-byte aligned; lse fp32 [B][T][q_heads] or NULL
 *   workspace  >= ts_hc_tree_attention_workspace_bytes(...) bytes, 256-byte aligned; it need not be
 *              initialised and must not be shared by calls that can run at the same time
 * The products run on the tensor cores in bf16 (an INT4 row's values, and their weights, in fp16: a weight is
 * off by 2^-11 of itself or 2^-31 of the row's largest) with fp32 sums; the softmax's maximum and sum are fp32. Over FP8 rows of 128 elements, 33 to 64 rows a key head
 * (T * q_heads/n_kv_heads) meet the keys as two e4m3 parts each, which leaves an element of q off by at
 * most 2^-17.8 of its row's largest. Weights times values are added up in fp32 before they are divided by the
 * weights' sum, a weight being up to 2^8 times the one that a row's sum is kept relative to: values beyond
 * 2^119 / (the keys that a row sees) can overflow to an infinity, and below 2^-100 they lose bits. A length
 * out of the page table's range is taken as the nearest one in it (recorded).
 * T <= 4096, T * q_heads/n_kv_heads <= 32768.
 */
size_t ts_hc_tree_attention_workspace_bytes(int B, int T, int q_heads, const ts_hc_kv_cache *cache);
ts_status ts_hc_tree_attention(const void *q, long q_stride, const ts_hc_kv_cache *cache, const int32_t *ctx_len,
                               const uint32_t *mask, long mask_stride, void *out, float *lse, int B, int T,
                               int q_heads, float scale, void *workspace, size_t workspace_bytes,
                               cudaStream_t stream);

/*
 * Which drafted tokens hold, and the token after them. Per sequence, from the root: p is the target's
 * distribution at the node reached, softmax(logits / temperature), q the draft's, from which the
 * node's children were drawn independently. With R = p and S = 1, for each child in node order, with
 * x its token:
 *     u * S * q[x] < R[x]:  the child is accepted; the walk goes on at it
 *     otherwise:            R = max(R - S q, 0), S = sum R       (kept as max(p - c q, 0), c += S)
 * and at the node where no child is left the next token is argmax_v R[v] / noise[v] over exponential
 * variates (p in R's place where nothing is left of it), which draws from R. So the tokens are distributed as the
 * target's own samples. A sequence with temperature <= 0 is greedy: a child holds where it is the argmax of
 * the logits, and the next token is the argmax. Ties go to the lowest index.
 *   logits       fp32 [B][T][V]: row i is the target's at node i (its successor's distribution)
 *   draft_probs  fp32 [B][T][V]: row i is the draft's at node i; rows of nodes without children are
 *                not read. NULL (with u and noise NULL): every sequence is greedy, temperature is not read
 *   tokens       int32 [B][T]; parents as in ts_hc_tree_build (NULL: a chain)
 *   temperature  fp32 [B]
 *   u            fp32 [B][T], in [0, 1): node i's at u[b][i] (the root's is not read)
 *   noise        fp32 [B][V], > 0
 *   n_accepted   int32 [B]; path int32 [B][T]: 0 and the accepted nodes, then -1; next_token int32 [B]
 * Only the rows that a walk reaches are read. A walk ends at a row that is no distribution -- a NaN in it,
 * or, not greedy, a +infinity or nothing but -infinity -- with 0 as the next token, and TS_ERR_INVALID_ARG
 * is recorded. T <= 4096, V < 2^30.
 */
ts_status ts_hc_verify(const float *logits, const float *draft_probs, const int32_t *tokens,
                       const int32_t *parents, long parents_stride, const float *temperature, const float *u,
                       const float *noise, int32_t *n_accepted, int32_t *path, int32_t *next_token, int B, int T,
                       int V, cudaStream_t stream);

/*
 * Self-test of the failure path. Launches one thread that waits, with the same
 * bounded wait the kernels use for their asynchronous copies, on a
 * shared-memory barrier that nothing arrives at. After about one second it
 * gives up and records TS_ERR_TIMEOUT in the device status word, as a kernel
 * whose copy never completed would; ts_hc_device_status() then reports it and
 * clears it. Nothing else is read or written, and the context stays usable.
 * Returns TS_OK once launched (asynchronous on `stream`).
 */
ts_status ts_hc_selftest_timeout(cudaStream_t stream);

/* The last error message of the calling thread ("" if none). */
const char *ts_hc_last_error(void);

/*
 * Reads the device-side status word of the current device (synchronising
 * `stream`) into *status (TS_OK or TS_ERR_TIMEOUT) and clears it. Returns
 * TS_ERR_CUDA if the read itself fails.
 */
ts_status ts_hc_device_status(cudaStream_t stream, int *status);

#ifdef __cplusplus
}
#endif

#endif /* TS_HC_H */
