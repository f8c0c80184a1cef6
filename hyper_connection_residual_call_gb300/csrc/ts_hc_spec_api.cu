// ts_hc_spec_api.cu -- the C ABI of the speculative decoding step in
// include/ts_hc.h (rotary positions, the paged cache, tree attention, the
// verification): argument validation on the host, then the launches.
#include <climits>
#include <cmath>

#include "hc_spec.h"
#include "ts_hc.h"
#include "ts_hc_internal.h"

namespace {

using tshc::api_error;
using tshc::check_ptr_api;

#define TS_TRY(expr)                      \
    do {                                  \
        const ts_status st_ = (expr);     \
        if (st_ != TS_OK)                 \
            return st_;                   \
    } while (0)

constexpr int kMaxNodes = 4096;
constexpr int kMaxHeads = 1024;
constexpr int kMaxBatch = 65535;

ts_status check_count(int v, const char *name, int lo, int hi)
{
    if (v < lo || v > hi)
        return api_error(TS_ERR_INVALID_ARG, "%s = %d must be in [%d, %d]", name, v, lo, hi);
    return TS_OK;
}

ts_status check_batch(int B, int T)
{
    TS_TRY(check_count(B, "B", 0, kMaxBatch));
    return check_count(T, "T", 0, kMaxNodes);
}

ts_status check_stride(long stride, const char *name, long least, long multiple)
{
    if (stride < least || stride % multiple != 0)
        return api_error(TS_ERR_INVALID_ARG, "%s = %ld must be a multiple of %ld and >= %ld", name, stride, multiple, least);
    return TS_OK;
}

ts_status check_tree_stride(long stride, int T)
{
    if (stride != 0 && stride < T)
        return api_error(TS_ERR_INVALID_ARG, "parents_stride = %ld must be 0 or >= T = %d", stride, T);
    return TS_OK;
}

// The cache's format; `tensors`: its pointers too.
ts_status check_cache(const ts_hc_kv_cache *c, bool tensors)
{
    if (!c)
        return api_error(TS_ERR_INVALID_ARG, "cache is NULL");
    if (c->type != TS_KV_BF16 && c->type != TS_KV_FP8 && c->type != TS_KV_INT4)
        return api_error(TS_ERR_INVALID_ARG, "cache.type = %d is not a ts_kvtype", (int)c->type);
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
        return api_error(TS_ERR_UNSUPPORTED, "cache.head_dim = %d: 64, 128 and 256 are supported", (int)c->head_dim);
    if (c->type == TS_KV_INT4 &&
        ((c->group != 32 && c->group != 64 && c->group != 128) || c->group > c->head_dim))
        return api_error(TS_ERR_UNSUPPORTED, "cache.group = %d: INT4 groups of 32, 64 or 128 and at most head_dim = %d are supported",
                         (int)c->group, (int)c->head_dim);
    if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)) != 0)
        return api_error(TS_ERR_INVALID_ARG, "cache.page_size = %d must be a power of two in [16, 1024]", (int)c->page_size);
    TS_TRY(check_count(c->n_kv_heads, "cache.n_kv_heads", 1, kMaxHeads));
    TS_TRY(check_count(c->max_pages, "cache.max_pages", 1, (1 << 30) / c->page_size));
    if (c->n_pages < 1 || c->n_pages > INT_MAX)
        return api_error(TS_ERR_INVALID_ARG, "cache.n_pages = %ld must be in [1, %d]", c->n_pages, INT_MAX);
    if (!tensors)
        return TS_OK;
    TS_TRY(check_ptr_api(c->k, "cache.k", 16));
    TS_TRY(check_ptr_api(c->v, "cache.v", 16));
    TS_TRY(check_ptr_api(c->page_table, "cache.page_table", 4));
    if (c->type != TS_KV_BF16) {
        TS_TRY(check_ptr_api(c->k_scales, "cache.k_scales", 16));
        TS_TRY(check_ptr_api(c->v_scales, "cache.v_scales", 16));
    }
    if (c->type == TS_KV_INT4) {
        TS_TRY(check_ptr_api(c->k_biases, "cache.k_biases", 16));
        TS_TRY(check_ptr_api(c->v_biases, "cache.v_biases", 16));
    }
    return TS_OK;
}

tshc::KvView view(const ts_hc_kv_cache *c)
{
    tshc::KvView v{};
    v.type = c->type;
    v.group = c->type == TS_KV_INT4 ? c->group : 0;
    while ((1 << v.page_shift) < c->page_size)
        ++v.page_shift;
    v.heads = c->n_kv_heads;
    v.D = c->head_dim;
    v.max_pages = c->max_pages;
    v.n_pages = c->n_pages;
    v.k = static_cast<uint8_t *>(c->k);
    v.v = static_cast<uint8_t *>(c->v);
    v.ks = static_cast<uint8_t *>(c->k_scales);
    v.vs = static_cast<uint8_t *>(c->v_scales);
    v.kb = static_cast<uint8_t *>(c->k_biases);
    v.vb = static_cast<uint8_t *>(c->v_biases);
    v.pages = c->page_table;
    return v;
}

ts_status device(tshc::LaunchCfg *cfg, unsigned **status)
{
    cfg->pdl = true;
    return tshc::device_api(&cfg->sm_count, status);
}

ts_status launched(cudaError_t e, const char *what) { return e == cudaSuccess ? TS_OK : tshc::cuda_error(e, what); }

// Rows of the cache that one call moves, one thread for 16 elements: 32-bit indices.
ts_status check_rows(long B, long T, const ts_hc_kv_cache *c)
{
    if (2 * B * (T + 31) * c->n_kv_heads * (c->head_dim / 16) > INT_MAX)  // (runs of 32 tokens)
        return api_error(TS_ERR_UNSUPPORTED, "%ld tokens of %d heads are too many for one call: split them", B * T,
                         (int)c->n_kv_heads);
    return TS_OK;
}

// Whether [a, a + na) and [b, b + nb) (bytes) share one.
bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// Whether n rows of wa 16-bit elements at a + i*sa and n rows of wb at b + i*sb
// share one. Exact for equal strides (slices of one projection's output are
// disjoint), by the address ranges otherwise.
bool rows_overlap(const void *a, long sa, long wa, const void *b, long sb, long wb, int n)
{
    if (!overlap(a, 2 * ((size_t)(n - 1) * sa + wa), b, 2 * ((size_t)(n - 1) * sb + wb)))
        return false;
    const intptr_t bytes = reinterpret_cast<intptr_t>(b) - reinterpret_cast<intptr_t>(a);
    if (sa != sb || bytes % 2 != 0)
        return true;
    const long m = ((long)(bytes / 2) % sa + sa) % sa;
    return !(m >= wa && m + wb <= sa);
}

}  // namespace

extern "C" {

ts_status ts_hc_rope_table(float *table, int max_pos, int rot, double theta, const ts_hc_rope_scaling *scaling,
                           cudaStream_t stream)
{
    tshc::clear_error();
    TS_TRY(check_count(max_pos, "max_pos", 0, INT_MAX));
    if (rot < 2 || rot > 1024 || rot % 2 != 0)
        return api_error(TS_ERR_INVALID_ARG, "rot = %d must be even and in [2, 1024]", rot);
    if (!(theta > 1.0) || !std::isfinite(theta))
        return api_error(TS_ERR_INVALID_ARG, "theta = %g must be > 1", theta);
    tshc::RopeTableParams p{};
    p.magnitude = 1.0;
    p.factor = 1.0;
    p.log_theta = std::log(theta);
    if (scaling) {
        const ts_hc_rope_scaling &s = *scaling;
        if (s.type < TS_ROPE_PLAIN || s.type > TS_ROPE_BY_PARTS)
            return api_error(TS_ERR_INVALID_ARG, "scaling.type = %d is not a ts_rope_scaling_type", (int)s.type);
        if (!(s.magnitude > 0.f) || !std::isfinite(s.magnitude))
            return api_error(TS_ERR_INVALID_ARG, "scaling.magnitude = %g must be > 0", (double)s.magnitude);
        if (s.type != TS_ROPE_PLAIN && (!(s.factor > 0.f) || !std::isfinite(s.factor)))
            return api_error(TS_ERR_INVALID_ARG, "scaling.factor = %g must be > 0", (double)s.factor);
        if (s.type == TS_ROPE_NTK && rot == 2)
            return api_error(TS_ERR_INVALID_ARG, "rot = 2 has no TS_ROPE_NTK scaling");
        if (s.type == TS_ROPE_BY_PARTS) {
            if (!(s.original_positions > 0.f) || !std::isfinite(s.original_positions))
                return api_error(TS_ERR_INVALID_ARG, "scaling.original_positions = %g must be > 0", (double)s.original_positions);
            if (!(s.beta_slow >= 0.f) || !(s.beta_fast > s.beta_slow) || !std::isfinite(s.beta_fast))
                return api_error(TS_ERR_INVALID_ARG, "scaling.beta_fast = %g must be > scaling.beta_slow = %g >= 0",
                                 (double)s.beta_fast, (double)s.beta_slow);
        }
        p.type = s.type;
        p.magnitude = s.magnitude;
        p.factor = s.factor;
        p.original = s.original_positions;
        p.beta_fast = s.beta_fast;
        p.beta_slow = s.beta_slow;
        if (s.type == TS_ROPE_NTK)
            p.log_theta += std::log((double)s.factor) * rot / (rot - 2);
    }
    if (max_pos == 0)
        return TS_OK;
    TS_TRY(check_ptr_api(table, "table", 16));
    p.table = table;
    p.max_pos = max_pos;
    p.half = rot / 2;
    return launched(tshc::launch_rope_table(p, stream), "launching the rotary table kernel");
}

ts_status ts_hc_rope(const void *q, long q_stride, const void *k, long k_stride, const int32_t *positions,
                     const float *table, int max_pos, void *q_out, long q_out_stride, void *k_out, long k_out_stride,
                     int N, int q_heads, int k_heads, int D, int rot, int interleaved, int inverse,
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
    if (N == 0)
        return TS_OK;
    const long qw = (long)q_heads * D, kw = (long)k_heads * D;
    TS_TRY(check_ptr_api(q, "q", 16));
    TS_TRY(check_ptr_api(q_out, "q_out", 16));
    TS_TRY(check_stride(q_stride, "q_stride", qw, 8));
    TS_TRY(check_stride(q_out_stride, "q_out_stride", qw, 8));
    if (k_heads > 0) {
        TS_TRY(check_ptr_api(k, "k", 16));
        TS_TRY(check_ptr_api(k_out, "k_out", 16));
        TS_TRY(check_stride(k_stride, "k_stride", kw, 8));
        TS_TRY(check_stride(k_out_stride, "k_out_stride", kw, 8));
    }
    TS_TRY(check_ptr_api(positions, "positions", 4));
    TS_TRY(check_ptr_api(table, "table", 16));
    if ((long)N * (q_heads + k_heads) * ((D + 15) / 16) > INT_MAX)
        return api_error(TS_ERR_UNSUPPORTED, "%d tokens of %d heads are too many for one call: split them", N,
                         q_heads + k_heads);
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
    tshc::LaunchCfg cfg;
    tshc::RopeParams p{};
    TS_TRY(device(&cfg, &p.status));
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.q_out = static_cast<uint16_t *>(q_out);
    p.k_out = static_cast<uint16_t *>(k_out);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.q_out_stride = q_out_stride;
    p.k_out_stride = k_out_stride;
    p.positions = positions;
    p.table = table;
    p.max_pos = max_pos;
    p.N = N;
    p.q_heads = q_heads;
    p.k_heads = k_heads;
    p.D = D;
    p.rot = rot;
    p.interleaved = interleaved != 0;
    p.inverse = inverse != 0;
    p.copy_rest = rot < D && !(q_in && k_in);
    return launched(tshc::launch_rope(p, cfg, stream), "launching the rotary kernel");
}

ts_status ts_hc_kv_write(const void *k, long k_stride, const void *v, long v_stride, const ts_hc_kv_cache *cache,
                         const int32_t *ctx_len, int B, int T, cudaStream_t stream)
{
    tshc::clear_error();
    TS_TRY(check_count(B, "B", 0, kMaxBatch));
    TS_TRY(check_count(T, "T", 0, INT_MAX));
    TS_TRY(check_cache(cache, B > 0 && T > 0));
    if (B == 0 || T == 0)
        return TS_OK;
    const long w = (long)cache->n_kv_heads * cache->head_dim;
    TS_TRY(check_ptr_api(k, "k", 16));
    TS_TRY(check_ptr_api(v, "v", 16));
    TS_TRY(check_stride(k_stride, "k_stride", w, 8));
    TS_TRY(check_stride(v_stride, "v_stride", w, 8));
    TS_TRY(check_ptr_api(ctx_len, "ctx_len", 4));
    TS_TRY(check_rows(B, T, cache));
    tshc::LaunchCfg cfg;
    tshc::KvParams p{};
    TS_TRY(device(&cfg, &p.status));
    p.c = view(cache);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.start = ctx_len;
    p.B = B;
    p.T = T;
    return launched(tshc::launch_kv_write(p, cfg, stream), "launching the cache write kernel");
}

ts_status ts_hc_kv_read(const ts_hc_kv_cache *cache, const int32_t *start, void *k_out, void *v_out, int B, int n,
                        cudaStream_t stream)
{
    tshc::clear_error();
    TS_TRY(check_count(B, "B", 0, kMaxBatch));
    TS_TRY(check_count(n, "n", 0, INT_MAX));
    TS_TRY(check_cache(cache, B > 0 && n > 0));
    if (B == 0 || n == 0)
        return TS_OK;
    TS_TRY(check_ptr_api(start, "start", 4));
    TS_TRY(check_ptr_api(k_out, "k_out", 16));
    TS_TRY(check_ptr_api(v_out, "v_out", 16));
    TS_TRY(check_rows(B, n, cache));
    tshc::LaunchCfg cfg;
    tshc::KvParams p{};
    TS_TRY(device(&cfg, &p.status));
    p.c = view(cache);
    p.k_out = static_cast<uint16_t *>(k_out);
    p.v_out = static_cast<uint16_t *>(v_out);
    p.start = start;
    p.B = B;
    p.T = n;
    return launched(tshc::launch_kv_read(p, cfg, stream), "launching the cache read kernel");
}

ts_status ts_hc_kv_compact(const ts_hc_kv_cache *cache, const int32_t *ctx_len, const int32_t *path,
                           const int32_t *n_accepted, int32_t *new_len, int B, int T, cudaStream_t stream)
{
    tshc::clear_error();
    TS_TRY(check_batch(B, T));
    TS_TRY(check_cache(cache, B > 0 && T > 0));
    if (B == 0 || T == 0)
        return TS_OK;
    TS_TRY(check_ptr_api(ctx_len, "ctx_len", 4));
    TS_TRY(check_ptr_api(path, "path", 4));
    TS_TRY(check_ptr_api(n_accepted, "n_accepted", 4));
    if (new_len) {
        TS_TRY(check_ptr_api(new_len, "new_len", 4));
        if (overlap(new_len, sizeof(int32_t) * (size_t)B, ctx_len, sizeof(int32_t) * (size_t)B))
            return api_error(TS_ERR_INVALID_ARG, "new_len overlaps ctx_len");
        if (overlap(new_len, sizeof(int32_t) * (size_t)B, n_accepted, sizeof(int32_t) * (size_t)B))
            return api_error(TS_ERR_INVALID_ARG, "new_len overlaps n_accepted");
        if (overlap(new_len, sizeof(int32_t) * (size_t)B, path, sizeof(int32_t) * (size_t)B * T))
            return api_error(TS_ERR_INVALID_ARG, "new_len overlaps path");
    }
    tshc::LaunchCfg cfg;
    tshc::KvCompactParams p{};
    TS_TRY(device(&cfg, &p.status));
    p.c = view(cache);
    p.ctx_len = ctx_len;
    p.path = path;
    p.n_accepted = n_accepted;
    p.new_len = new_len;
    p.B = B;
    p.T = T;
    return launched(tshc::launch_kv_compact(p, cfg, stream), "launching the cache compaction kernel");
}

ts_status ts_hc_tree_build(const int32_t *parents, long parents_stride, const int32_t *ctx_len, uint32_t *mask,
                           int32_t *positions, int B, int T, cudaStream_t stream)
{
    tshc::clear_error();
    TS_TRY(check_batch(B, T));
    TS_TRY(check_tree_stride(parents_stride, T));
    if (B == 0 || T == 0)
        return TS_OK;
    TS_TRY(check_ptr_api(parents, "parents", 4));
    if (!mask && !positions)
        return api_error(TS_ERR_INVALID_ARG, "mask and positions are both NULL");
    if (mask)
        TS_TRY(check_ptr_api(mask, "mask", 4));
    if (positions)
        TS_TRY(check_ptr_api(positions, "positions", 4));
    if (ctx_len)
        TS_TRY(check_ptr_api(ctx_len, "ctx_len", 4));
    tshc::LaunchCfg cfg;
    tshc::TreeBuildParams p{};
    TS_TRY(device(&cfg, &p.status));
    p.parents = parents;
    p.parents_stride = parents_stride;
    p.ctx_len = ctx_len;
    p.mask = mask;
    p.positions = positions;
    p.B = B;
    p.T = T;
    return launched(tshc::launch_tree_build(p, cfg, stream), "launching the tree mask kernel");
}

}  // extern "C"

namespace {

ts_status check_attention(const ts_hc_kv_cache *cache, int B, int T, int q_heads, bool tensors)
{
    TS_TRY(check_batch(B, T));
    TS_TRY(check_cache(cache, tensors));
    if (q_heads < 1 || q_heads % cache->n_kv_heads != 0)
        return api_error(TS_ERR_INVALID_ARG, "q_heads = %d must be a positive multiple of cache.n_kv_heads = %d", q_heads,
                         (int)cache->n_kv_heads);
    if ((long)T * (q_heads / cache->n_kv_heads) > 32768)
        return api_error(TS_ERR_UNSUPPORTED, "T = %d nodes of %d query heads a key head are more than 32768 rows: split the nodes", T,
                         q_heads / cache->n_kv_heads);
    return TS_OK;
}

}  // namespace

extern "C" {

size_t ts_hc_tree_attention_workspace_bytes(int B, int T, int q_heads, const ts_hc_kv_cache *cache)
{
    if (check_attention(cache, B, T, q_heads, false) != TS_OK)
        return 0;
    return tshc::attn_part_bytes(B, T, q_heads, view(cache));
}

ts_status ts_hc_tree_attention(const void *q, long q_stride, const ts_hc_kv_cache *cache, const int32_t *ctx_len,
                               const uint32_t *mask, long mask_stride, void *out, float *lse, int B, int T, int q_heads,
                               float scale, void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    tshc::clear_error();
    const bool some = B > 0 && T > 0;
    TS_TRY(check_attention(cache, B, T, q_heads, some));
    if (!some)
        return TS_OK;
    const int words = (T + 31) / 32;
    TS_TRY(check_ptr_api(q, "q", 16));
    TS_TRY(check_stride(q_stride, "q_stride", (long)q_heads * cache->head_dim, 8));
    TS_TRY(check_ptr_api(ctx_len, "ctx_len", 4));
    if (mask) {
        TS_TRY(check_ptr_api(mask, "mask", 4));
        if (mask_stride != 0 && mask_stride < (long)T * words)
            return api_error(TS_ERR_INVALID_ARG, "mask_stride = %ld must be 0 or >= %ld words", mask_stride, (long)T * words);
    }
    TS_TRY(check_ptr_api(out, "out", 16));
    if (lse)
        TS_TRY(check_ptr_api(lse, "lse", 4));
    if (!std::isfinite(scale))
        return api_error(TS_ERR_INVALID_ARG, "scale = %g must be finite", (double)scale);
    tshc::LaunchCfg cfg;
    tshc::AttnParams p{};
    p.c = view(cache);
    const size_t need = tshc::attn_part_bytes(B, T, q_heads, p.c);
    if (!workspace || workspace_bytes < need)
        return api_error(TS_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", workspace ? workspace_bytes : (size_t)0, need);
    TS_TRY(check_ptr_api(workspace, "workspace", 256));
    TS_TRY(device(&cfg, &p.status));
    p.q = static_cast<const uint16_t *>(q);
    p.q_stride = q_stride;
    p.ctx_len = ctx_len;
    p.mask = mask;
    p.mask_stride = mask_stride;
    p.mask_words = words;
    p.out = static_cast<uint16_t *>(out);
    p.lse = lse;
    p.B = B;
    p.T = T;
    p.q_heads = q_heads;
    p.G = q_heads / cache->n_kv_heads;
    p.rows = T * p.G;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.part = static_cast<float *>(workspace);
    return launched(tshc::launch_tree_attention(p, cfg, stream), "launching the tree attention kernels");
}

ts_status ts_hc_verify(const float *logits, const float *draft_probs, const int32_t *tokens, const int32_t *parents,
                       long parents_stride, const float *temperature, const float *u, const float *noise,
                       int32_t *n_accepted, int32_t *path, int32_t *next_token, int B, int T, int V, cudaStream_t stream)
{
    tshc::clear_error();
    TS_TRY(check_batch(B, T));
    TS_TRY(check_count(V, "V", 1, (1 << 30) - 1));
    TS_TRY(check_tree_stride(parents_stride, T));
    if (B == 0 || T == 0)
        return TS_OK;
    TS_TRY(check_ptr_api(logits, "logits", 4));
    TS_TRY(check_ptr_api(tokens, "tokens", 4));
    if ((draft_probs != nullptr) != (u != nullptr) || (draft_probs != nullptr) != (noise != nullptr))
        return api_error(TS_ERR_INVALID_ARG, "draft_probs, u and noise are given together, or none of them (greedy)");
    if (draft_probs) {
        TS_TRY(check_ptr_api(draft_probs, "draft_probs", 4));
        TS_TRY(check_ptr_api(u, "u", 4));
        TS_TRY(check_ptr_api(noise, "noise", 4));
        TS_TRY(check_ptr_api(temperature, "temperature", 4));
    }
    if (parents)
        TS_TRY(check_ptr_api(parents, "parents", 4));
    TS_TRY(check_ptr_api(n_accepted, "n_accepted", 4));
    TS_TRY(check_ptr_api(path, "path", 4));
    TS_TRY(check_ptr_api(next_token, "next_token", 4));
    tshc::LaunchCfg cfg;
    tshc::VerifyParams p{};
    TS_TRY(device(&cfg, &p.status));
    p.logits = logits;
    p.draft = draft_probs;
    p.temperature = temperature;
    p.u = u;
    p.noise = noise;
    p.tokens = tokens;
    p.parents = parents;
    p.parents_stride = parents_stride;
    p.n_accepted = n_accepted;
    p.path = path;
    p.next_token = next_token;
    p.B = B;
    p.T = T;
    p.V = V;
    return launched(tshc::launch_verify(p, cfg, stream), "launching the verification kernel");
}

}  // extern "C"
