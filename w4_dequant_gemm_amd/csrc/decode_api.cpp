// C ABI of the decoding calls (paged cache, attention over it, token choice):
// argument checks, then the launches on the caller's stream.  As for the
// products: no allocation, no state, nothing launched on a refused argument.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "checks.hpp"
#include "decode_kernels.hpp"

namespace {
using w4::aligned16;
using w4::fail;
using w4::hip_status;

constexpr int64_t kInt32Most = 0x7FFFFFFF;
constexpr int64_t kMaxLength = int64_t{1} << 29;   // tokens of one sequence
constexpr int64_t kMaxVocab = int64_t{1} << 20;

long long ll(int64_t v) { return static_cast<long long>(v); }

int check_cache(const char* fn, const w4_kv_cache* c, bool one_layer, w4::KvCache* out) {
    if (!c) return fail(W4_EINVAL, "%s: cache is NULL", fn);
    if (c->dtype != W4_KV_BF16 && c->dtype != W4_KV_E4M3)
        return fail(W4_EINVAL, "%s: cache dtype %d is neither W4_KV_BF16 nor W4_KV_E4M3", fn, c->dtype);
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
        return fail(W4_EUNSUPPORTED, "%s: head_dim %d is not one of 64, 128, 256", fn, c->head_dim);
    if (c->page_size <= 0 || c->page_size % 16 != 0 || c->page_size > 1024)
        return fail(W4_EUNSUPPORTED, "%s: page_size %d is not a multiple of 16 up to 1024", fn, c->page_size);
    if (c->kv_heads <= 0 || c->kv_heads > 65535) return fail(W4_EINVAL, "%s: kv_heads = %d must be in 1..65535", fn, c->kv_heads);
    if (c->layers <= 0 || c->layers > 65535) return fail(W4_EINVAL, "%s: layers = %d must be in 1..65535", fn, c->layers);
    if (one_layer && c->layers != 1) return fail(W4_EINVAL, "%s: takes one layer of the cache, not %d", fn, c->layers);
    if (c->pages <= 0 || c->pages > kInt32Most / c->page_size)
        return fail(W4_EINVAL, "%s: pages = %lld outside 1..(2^31 - 1) / page_size", fn, ll(c->pages));
    W4_REQUIRE_PTR(fn, c->k);
    W4_REQUIRE_PTR(fn, c->v);
    // (moving copies codes and needs no scales)
    if (one_layer && c->dtype == W4_KV_E4M3 && (!c->k_scale || !c->v_scale))
        return fail(W4_EINVAL, "%s: an E4M3 cache needs k_scale and v_scale", fn);
    if (c->dtype == W4_KV_BF16 && (c->k_scale || c->v_scale))
        return fail(W4_EINVAL, "%s: k_scale and v_scale must be NULL for a bf16 cache", fn);
    *out = w4::KvCache{c->k, c->v, c->k_scale, c->v_scale, c->pages, c->layers, c->kv_heads, c->head_dim,
                       c->page_size / 16, c->dtype == W4_KV_E4M3};
    return W4_OK;
}

// rows [T, heads, dim] of bf16, `stride` elements apart
int check_rows(const char* fn, const char* name, const uint16_t* x, int64_t stride, int64_t heads, int dim) {
    if (!x) return fail(W4_EINVAL, "%s: %s is NULL", fn, name);
    if (!aligned16(x)) return fail(W4_EINVAL, "%s: %s is not 16-byte aligned", fn, name);
    if (stride < heads * dim || stride % 8 != 0)
        return fail(W4_EINVAL, "%s: rows of %s are %lld elements apart; a multiple of 8 of at least %lld is needed", fn, name,
                    ll(stride), ll(heads * dim));
    return W4_OK;
}

int check_table(const char* fn, const int32_t* page_table, int64_t table_pages, int page_size) {
    if (!page_table) return fail(W4_EINVAL, "%s: page_table is NULL", fn);
    if (table_pages <= 0 || table_pages > kMaxLength / page_size)
        return fail(W4_EINVAL, "%s: table_pages = %lld outside 1..2^29 / page_size", fn, ll(table_pages));
    return W4_OK;
}

bool attention_sizes_ok(int64_t T, int64_t B, int hq, int hk, int64_t max_q, int64_t max_kv, int64_t window) {
    return T > 0 && B > 0 && B <= 65535 && hq > 0 && hk > 0 && hq % hk == 0 && hq <= 65535 && T <= kInt32Most / hq && max_q > 0 &&
           max_q <= T && max_kv > 0 && max_kv <= kMaxLength && window >= 0 && window <= kMaxLength;
}
}  // namespace

extern "C" {

int w4_kv_append(const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                 int64_t v_stride, int64_t T, int Hq, const w4_kv_cache* cache, const int32_t* slots,
                 const float* rope, int64_t rope_rows, int rot, int interleaved, const int32_t* positions,
                 const float* q_norm, const float* k_norm, float eps, uint16_t* Q, hipStream_t stream) {
    const char* fn = "w4_kv_append";
    w4::KvAppendParams p{};
    W4_TRY(check_cache(fn, cache, true, &p.cache));
    const int hk = p.cache.heads, dim = p.cache.dim;
    if (!q != !Q) return fail(W4_EINVAL, "%s: q and Q must both be given or both be NULL", fn);
    if (q && (Hq <= 0 || Hq > 65535)) return fail(W4_EINVAL, "%s: Hq = %d must be in 1..65535", fn, Hq);
    const int hq = q ? Hq : 0;
    if (T < 0 || T > kInt32Most / (hq + 2 * hk) / (dim / 8) - 16)   // (a thread each 8 dims)
        return fail(W4_EINVAL, "%s: T = %lld outside 0..2^31 / (heads * head_dim / 8)", fn, ll(T));
    if (T == 0) return W4_OK;
    if (q) W4_TRY(check_rows(fn, "q", q, q_stride, hq, dim));
    W4_TRY(check_rows(fn, "k", k, k_stride, hk, dim));
    W4_TRY(check_rows(fn, "v", v, v_stride, hk, dim));
    if (Q && !aligned16(Q)) return fail(W4_EINVAL, "%s: Q is not 16-byte aligned", fn);
    if (!slots) return fail(W4_EINVAL, "%s: slots is NULL", fn);
    if (!rope != !positions) return fail(W4_EINVAL, "%s: rope and positions must both be given or both be NULL", fn);
    if (rope) {
        if (!aligned16(rope)) return fail(W4_EINVAL, "%s: rope is not 16-byte aligned", fn);
        if (rope_rows <= 0) return fail(W4_EINVAL, "%s: rope_rows = %lld must be > 0", fn, ll(rope_rows));
        if (rot <= 0 || rot > dim) return fail(W4_EINVAL, "%s: rot = %d outside 1..head_dim", fn, rot);
        if (rot % 16 != 0) return fail(W4_EUNSUPPORTED, "%s: rot = %d is not a multiple of 16", fn, rot);
    }
    if ((q_norm && !aligned16(q_norm)) || (k_norm && !aligned16(k_norm)))
        return fail(W4_EINVAL, "%s: q_norm or k_norm is not 16-byte aligned", fn);
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(W4_EINVAL, "%s: eps = %g must be finite and >= 0", fn, static_cast<double>(eps));
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.T = static_cast<int>(T);
    p.hq = hq;
    p.slots = slots;
    p.rope = rope;
    p.rope_rows = rope_rows;
    p.rot = rot;
    p.interleaved = interleaved != 0;
    p.positions = positions;
    p.q_norm = q_norm;
    p.k_norm = k_norm;
    p.eps = eps;
    p.Q = Q;
    return hip_status(w4::launch_kv_append(p, stream), fn);
}

size_t w4_tree_attention_workspace_bytes(int64_t T, int64_t B, int Hq, int kv_heads, int head_dim, int dtype,
                                         int64_t max_q, int64_t max_kv, int64_t window) {
    if (!attention_sizes_ok(T, B, Hq, kv_heads, max_q, max_kv, window)) return 0;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
    if (dtype != W4_KV_BF16 && dtype != W4_KV_E4M3) return 0;
    return w4::attention_workspace_bytes(T, B, Hq, kv_heads, head_dim, dtype == W4_KV_E4M3, max_q, max_kv, window);
}

int w4_tree_attention(const uint16_t* q, int64_t q_stride, int64_t T, int Hq, const w4_kv_cache* cache,
                      const int32_t* page_table, int64_t table_pages, const int32_t* kv_len, const int32_t* q_start,
                      int64_t B, int64_t max_q, int64_t max_kv, const uint64_t* tree, int tree_words,
                      const int32_t* positions, int64_t window, float scale, uint16_t* O, void* workspace,
                      size_t workspace_bytes, hipStream_t stream) {
    const char* fn = "w4_tree_attention";
    w4::AttentionParams p{};
    W4_TRY(check_cache(fn, cache, true, &p.cache));
    const int hk = p.cache.heads, dim = p.cache.dim, page_size = 16 * p.cache.page_blocks;
    if (T < 0 || B < 0) return fail(W4_EINVAL, "%s: T = %lld and B = %lld must be >= 0", fn, ll(T), ll(B));
    if (Hq <= 0 || Hq % hk != 0)
        return fail(W4_EINVAL, "%s: Hq = %d must be a positive multiple of kv_heads = %d", fn, Hq, hk);
    if (T == 0 || B == 0) return W4_OK;
    if (max_q < 0 || max_q > T) return fail(W4_EINVAL, "%s: max_q = %lld outside 0..T", fn, ll(max_q));
    if (max_kv < 0 || max_kv > kMaxLength) return fail(W4_EINVAL, "%s: max_kv = %lld outside 0..2^29", fn, ll(max_kv));
    if (window < 0 || window > kMaxLength) return fail(W4_EINVAL, "%s: window = %lld outside 0..2^29", fn, ll(window));
    if (max_q == 0) return W4_OK;
    const int64_t plan_kv = max_kv > 0 ? max_kv : 1;   // 0: every row is empty, zeros
    if (!attention_sizes_ok(T, B, Hq, hk, max_q, plan_kv, window))
        return fail(W4_EUNSUPPORTED, "%s: T = %lld, B = %lld, Hq = %d: T Hq is limited to 2^31 - 1, B and Hq to 65535", fn, ll(T), ll(B), Hq);
    W4_TRY(check_rows(fn, "q", q, q_stride, Hq, dim));
    W4_REQUIRE_PTR(fn, O);
    W4_TRY(check_table(fn, page_table, table_pages, page_size));
    if (max_kv > table_pages * page_size)
        return fail(W4_EINVAL, "%s: max_kv = %lld tokens do not fit %lld pages of %d", fn, ll(max_kv), ll(table_pages), page_size);
    if (!kv_len || !q_start) return fail(W4_EINVAL, "%s: kv_len or q_start is NULL", fn);
    if (tree && (tree_words <= 0 || (max_q + 63) / 64 > tree_words))
        return fail(W4_EINVAL, "%s: tree_words = %d hold fewer than max_q = %lld nodes", fn, tree_words, ll(max_q));
    if (tree && window > 0 && !positions) return fail(W4_EINVAL, "%s: a window over a tree needs positions", fn);
    if (!std::isfinite(scale)) return fail(W4_EINVAL, "%s: scale is not finite", fn);
    if (workspace && !aligned16(workspace)) return fail(W4_EINVAL, "%s: workspace is not 16-byte aligned", fn);
    const size_t need = w4::attention_workspace_bytes(T, B, Hq, hk, dim, p.cache.e4m3, max_q, plan_kv, window);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(W4_EINVAL, "%s: workspace of %zu bytes, these sizes need %zu (w4_tree_attention_workspace_bytes)", fn,
                    workspace ? workspace_bytes : size_t{0}, need);
    p.q = q;
    p.q_stride = q_stride;
    p.T = T;
    p.hq = Hq;
    p.page_table = page_table;
    p.table_pages = table_pages;
    p.kv_len = kv_len;
    p.q_start = q_start;
    p.B = static_cast<int>(B);
    p.max_q = static_cast<int>(max_q);
    p.max_kv = static_cast<int>(max_kv);
    p.tree = tree;
    p.tree_words = tree_words;
    p.positions = window > 0 ? positions : nullptr;
    p.window = static_cast<int>(window);
    p.scale = scale;
    p.O = O;
    p.ws = need > 0 ? static_cast<float*>(workspace) : nullptr;
    return hip_status(w4::launch_attention(p, stream), fn);
}

int w4_sample(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride, const float* u,
              const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
              int32_t* tokens, float* probs, hipStream_t stream) {
    const char* fn = "w4_sample";
    if (dtype != W4_LOGITS_BF16 && dtype != W4_LOGITS_F32)
        return fail(W4_EINVAL, "%s: dtype %d is neither W4_LOGITS_BF16 nor W4_LOGITS_F32", fn, dtype);
    if (B < 0 || B > 65535) return fail(W4_EINVAL, "%s: B = %lld outside 0..65535", fn, ll(B));
    if (V <= 0) return fail(W4_EINVAL, "%s: V = %lld must be > 0", fn, ll(V));
    if (V > kMaxVocab) return fail(W4_EUNSUPPORTED, "%s: V = %lld above 2^20", fn, ll(V));
    if (row_stride != 0 && row_stride < V)
        return fail(W4_EINVAL, "%s: row_stride = %lld is neither 0 (one row for all) nor at least V = %lld", fn, ll(row_stride), ll(V));
    if (B == 0) return W4_OK;
    if (!logits) return fail(W4_EINVAL, "%s: logits is NULL", fn);
    if (reinterpret_cast<uintptr_t>(logits) % (dtype == W4_LOGITS_F32 ? 4 : 2) != 0)
        return fail(W4_EINVAL, "%s: logits is not aligned to its elements", fn);
    if (!u) return fail(W4_EINVAL, "%s: u is NULL", fn);
    if (!tokens) return fail(W4_EINVAL, "%s: tokens is NULL", fn);
    const w4::SampleParams p{logits, dtype == W4_LOGITS_F32, static_cast<int>(B), static_cast<int>(V), row_stride, u,
                             temperature, top_k, top_p, min_p, tokens, probs};
    return hip_status(w4::launch_sample(p, stream), fn);
}

int w4_kv_move(const w4_kv_cache* cache, const int32_t* page_table, int64_t table_pages, const int32_t* base,
               const int32_t* path, int64_t path_len, const int32_t* count, int64_t B, hipStream_t stream) {
    const char* fn = "w4_kv_move";
    w4::KvMoveParams p{};
    W4_TRY(check_cache(fn, cache, false, &p.cache));
    if (B < 0 || B > 65535) return fail(W4_EINVAL, "%s: B = %lld outside 0..65535", fn, ll(B));
    if (path_len < 0 || path_len > kMaxLength) return fail(W4_EINVAL, "%s: path_len = %lld outside 0..2^29", fn, ll(path_len));
    if (B == 0 || path_len == 0) return W4_OK;
    W4_TRY(check_table(fn, page_table, table_pages, 16 * p.cache.page_blocks));
    if (!base || !path || !count) return fail(W4_EINVAL, "%s: base, path or count is NULL", fn);
    p.page_table = page_table;
    p.table_pages = table_pages;
    p.base = base;
    p.path = path;
    p.path_len = path_len;
    p.count = count;
    p.B = static_cast<int>(B);
    return hip_status(w4::launch_kv_move(p, stream), fn);
}

}  // extern "C"
