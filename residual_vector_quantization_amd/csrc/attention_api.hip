// C ABI of the streaming-attention operators: argument checks, then the
// launches on the caller's stream. Declarations and contract are in
// include/rvq_attention.h. No allocation, no global state.
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "rvq_attention.h"
#include "attention_internal.h"
#include "cache_index.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

rvq_status from_hip(hipError_t e)
{
    return e == hipSuccess ? RVQ_OK : e == hipErrorNotSupported ? RVQ_ERR_UNSUPPORTED : RVQ_ERR_DEVICE;
}

int element_bytes(int32_t dtype) { return dtype == RVQ_F32 ? 4 : 2; }

// 64 rows span less than 2^31 bytes
constexpr int64_t kMaxTokenStride = (1 << 23) - 16;

bool known_dtype(int32_t dtype) { return dtype == RVQ_F32 || dtype == RVQ_F16 || dtype == RVQ_BF16; }

bool good_heads(const rvq_heads *h, int32_t dtype)
{
    const int64_t row = 16 / element_bytes(dtype);
    return h && h->data && aligned(h->data, 16) && h->token_stride >= 0 && h->head_stride >= 0 &&
           h->token_stride <= kMaxTokenStride &&
           h->token_stride % row == 0 && h->head_stride % row == 0;
}

// Rows that the kernels write must lie apart: one of the strides spans the other's rows.
bool good_output(const rvq_heads *h, int32_t dtype, int32_t heads, int32_t dim, int64_t tokens)
{
    if (!good_heads(h, dtype)) return false;
    const __int128 token = h->token_stride, head = h->head_stride;
    const bool heads_inside = (heads == 1 || head >= dim) && (tokens <= 1 || token >= (heads - 1) * head + dim);
    const bool tokens_inside = (tokens <= 1 || token >= dim) && (heads == 1 || head >= (tokens - 1) * token + dim);
    return heads_inside || tokens_inside;
}

rvq::Heads heads(const rvq_heads *h) { return rvq::Heads{h->data, h->token_stride, h->head_stride}; }

int clamp_window(int64_t window) { return window < 0 || window > INT_MAX ? INT_MAX : static_cast<int>(window); }

bool good_scale(float scale) { return isfinite(scale) && scale >= 0.0f; }

rvq_status check_attention(const rvq_attention_shape *s)
{
    if (!s || s->n_clips < 0 || s->q_heads <= 0 || s->kv_heads <= 0 || s->dim <= 0 || s->sinks < 0 ||
        s->q_tokens < 0 || s->k_tokens < 0 || !good_scale(s->scale))
        return RVQ_ERR_INVALID_ARG;
    if (s->q_heads % s->kv_heads != 0 || !known_dtype(s->dtype)) return RVQ_ERR_INVALID_ARG;
    // row offsets are int32, and one grid dimension holds the heads
    if ((s->dim != 64 && s->dim != 128) || s->q_tokens > INT_MAX - 1024 || s->k_tokens > INT_MAX - 1024 ||
        s->n_clips > (1 << 20) || s->q_heads > 65535)
        return RVQ_ERR_UNSUPPORTED;
    return RVQ_OK;
}

rvq::AttentionArgs attention_args(const rvq_attention_shape *s)
{
    rvq::AttentionArgs a = {};
    a.dtype = s->dtype;
    a.dim = s->dim;
    a.n_clips = s->n_clips;
    a.q_heads = s->q_heads;
    a.kv_heads = s->kv_heads;
    a.window = clamp_window(s->window);
    a.sinks = s->sinks;
    a.q_tokens = s->q_tokens;
    a.k_tokens = s->k_tokens;
    a.cu_q = s->cu_q;
    a.cu_k = s->cu_k;
    a.scale = s->scale;
    return a;
}

rvq_status check_cache(const rvq_cache_shape *s)
{
    if (!s || s->n_clips < 0 || s->kv_heads <= 0 || s->dim <= 0 || s->page_size <= 0 || s->n_pages < 0 ||
        s->table_ld < 0 || !known_dtype(s->dtype))
        return RVQ_ERR_INVALID_ARG;
    if ((s->dim != 64 && s->dim != 128) || s->kv_heads > 65535 ||
        static_cast<int64_t>(s->table_ld) * s->page_size > INT_MAX - 1024 ||
        static_cast<__int128>(s->n_pages) * s->page_size * s->kv_heads > rvq::kMaxRows)
        return RVQ_ERR_UNSUPPORTED;
    return RVQ_OK;
}

rvq_status check_upkeep(int32_t n_clips, int32_t table_ld, int32_t page_size, int32_t n_pages)
{
    if (n_clips < 0 || table_ld < 0 || page_size <= 0 || n_pages < 0) return RVQ_ERR_INVALID_ARG;
    if (static_cast<int64_t>(table_ld) * page_size > INT_MAX - 1024 ||
        static_cast<int64_t>(table_ld) * n_clips > INT_MAX - 1024 || n_pages > INT_MAX - (1 << 20) ||
        n_clips > (1 << 20))
        return RVQ_ERR_UNSUPPORTED;
    return RVQ_OK;
}

int64_t page_bytes(const rvq_cache_shape *s)
{
    return static_cast<int64_t>(s->kv_heads) * s->page_size * s->dim * element_bytes(s->dtype);
}

bool ints(const void *p) { return p && aligned(p, 4); }

bool scratch(const void *p, int64_t given, int64_t wanted)
{
    return wanted == 0 || (p && aligned(p, 16) && given >= wanted);
}

}  // namespace

extern "C" {

RVQ_API rvq_status rvq_window_attention(const rvq_attention_shape *shape, const rvq_heads *q, const rvq_heads *k,
                                        const rvq_heads *v, const rvq_heads *out, float *lse, void *stream)
{
    const rvq_status st = check_attention(shape);
    if (st != RVQ_OK) return st;
    if (shape->n_clips == 0 || shape->q_tokens == 0) return RVQ_OK;
    if (!ints(shape->cu_q) || !ints(shape->cu_k) || !good_heads(q, shape->dtype) ||
        !good_output(out, shape->dtype, shape->q_heads, shape->dim, shape->q_tokens) || (lse && !aligned(lse, 4)))
        return RVQ_ERR_INVALID_ARG;
    rvq::AttentionArgs a = attention_args(shape);
    if (a.k_tokens > 0) {
        if (!good_heads(k, shape->dtype) || !good_heads(v, shape->dtype)) return RVQ_ERR_INVALID_ARG;
        a.k = heads(k);
        a.v = heads(v);
    }
    a.q = heads(q);
    a.out = heads(out);
    a.lse = lse;
    return from_hip(rvq::launch_window_attention(a, static_cast<hipStream_t>(stream)));
}

RVQ_API int64_t rvq_window_attention_backward_bytes(const rvq_attention_shape *shape)
{
    const rvq_status st = check_attention(shape);
    if (st != RVQ_OK) return st;
    return rvq::window_attention_backward_bytes(attention_args(shape));
}

RVQ_API rvq_status rvq_window_attention_backward(const rvq_attention_shape *shape, const rvq_heads *dout,
                                                 const rvq_heads *q, const rvq_heads *k, const rvq_heads *v,
                                                 const rvq_heads *out, const float *lse,
                                                 const rvq_heads *dq, const rvq_heads *dk, const rvq_heads *dv,
                                                 void *workspace, int64_t workspace_bytes, void *stream)
{
    const int64_t wanted = rvq_window_attention_backward_bytes(shape);
    if (wanted < 0) return static_cast<rvq_status>(wanted);
    if (shape->n_clips == 0 || (shape->q_tokens == 0 && shape->k_tokens == 0)) return RVQ_OK;
    if (!ints(shape->cu_q) || !ints(shape->cu_k) || !scratch(workspace, workspace_bytes, wanted))
        return RVQ_ERR_INVALID_ARG;
    rvq::AttentionArgs a = attention_args(shape);
    if (a.q_tokens > 0) {
        if (!good_heads(q, a.dtype) || !good_heads(dout, a.dtype) || !good_heads(out, a.dtype) || !lse ||
            !aligned(lse, 4) || !good_output(dq, a.dtype, a.q_heads, a.dim, a.q_tokens))
            return RVQ_ERR_INVALID_ARG;
        a.q = heads(q);
        a.dout = heads(dout);
        a.out = heads(out);
        a.dq = heads(dq);
        a.lse = const_cast<float *>(lse);   // read only in the backward pass
    }
    if (a.k_tokens > 0) {
        if (!good_heads(k, a.dtype) || !good_heads(v, a.dtype) ||
            !good_output(dk, a.dtype, a.kv_heads, a.dim, a.k_tokens) ||
            !good_output(dv, a.dtype, a.kv_heads, a.dim, a.k_tokens))
            return RVQ_ERR_INVALID_ARG;
        a.k = heads(k);
        a.v = heads(v);
        a.dk = heads(dk);
        a.dv = heads(dv);
    }
    a.workspace = workspace;
    return from_hip(rvq::launch_window_attention_backward(a, static_cast<hipStream_t>(stream)));
}

RVQ_API int64_t rvq_cache_attention_bytes(const rvq_cache_shape *shape, int32_t q_heads)
{
    const rvq_status st = check_cache(shape);
    if (st != RVQ_OK) return st;
    if (q_heads <= 0 || q_heads % shape->kv_heads != 0) return RVQ_ERR_INVALID_ARG;
    return rvq::cache_attention_bytes(shape->n_clips, q_heads, shape->kv_heads, shape->dim,
                                      static_cast<int64_t>(shape->table_ld) * shape->page_size);
}

RVQ_API rvq_status rvq_cache_attention(const rvq_cache_shape *shape, int32_t q_heads, const rvq_heads *q,
                                       const void *k_pool, const void *v_pool, const int32_t *table,
                                       const int32_t *lens, int64_t window, int32_t sinks, float scale,
                                       const rvq_heads *out, void *workspace, int64_t workspace_bytes, void *stream)
{
    const int64_t wanted = rvq_cache_attention_bytes(shape, q_heads);
    if (wanted < 0) return static_cast<rvq_status>(wanted);
    if (sinks < 0 || !good_scale(scale)) return RVQ_ERR_INVALID_ARG;
    if (q_heads > 65535 || shape->n_clips > (1 << 20)) return RVQ_ERR_UNSUPPORTED;
    if (shape->n_clips == 0) return RVQ_OK;
    if (!good_heads(q, shape->dtype) || !good_output(out, shape->dtype, q_heads, shape->dim, shape->n_clips) ||
        !ints(lens) || !scratch(workspace, workspace_bytes, wanted))
        return RVQ_ERR_INVALID_ARG;
    if (shape->table_ld > 0 && !ints(table)) return RVQ_ERR_INVALID_ARG;
    if (shape->n_pages > 0 && (!k_pool || !v_pool || !aligned(k_pool, 16) || !aligned(v_pool, 16)))
        return RVQ_ERR_INVALID_ARG;
    rvq::CacheAttentionArgs a = {};
    a.dtype = shape->dtype;
    a.dim = shape->dim;
    a.n_clips = shape->n_clips;
    a.q_heads = q_heads;
    a.kv_heads = shape->kv_heads;
    a.page_size = shape->page_size;
    a.n_pages = shape->n_pages;
    a.table_ld = shape->table_ld;
    a.window = clamp_window(window);
    a.sinks = sinks;
    a.scale = scale;
    a.q = heads(q);
    a.out = heads(out);
    a.k_pool = k_pool;
    a.v_pool = v_pool;
    a.table = table;
    a.lens = lens;
    a.workspace = workspace;
    return from_hip(rvq::launch_cache_attention(a, static_cast<hipStream_t>(stream)));
}

RVQ_API rvq_status rvq_cache_append(const rvq_cache_shape *shape, const rvq_heads *k, const rvq_heads *v,
                                    int64_t n_tokens, const int32_t *cu, const int32_t *table, const int32_t *lens,
                                    void *k_pool, void *v_pool, void *stream)
{
    const rvq_status st = check_cache(shape);
    if (st != RVQ_OK) return st;
    if (n_tokens < 0 || (!cu && n_tokens != shape->n_clips)) return RVQ_ERR_INVALID_ARG;
    if (n_tokens > INT_MAX - 1024) return RVQ_ERR_UNSUPPORTED;
    if (n_tokens == 0 || shape->n_clips == 0 || shape->n_pages == 0 || shape->table_ld == 0) return RVQ_OK;
    if (!good_heads(k, shape->dtype) || !good_heads(v, shape->dtype) || !ints(table) || !ints(lens) ||
        (cu && !aligned(cu, 4)) || !k_pool || !v_pool || !aligned(k_pool, 16) || !aligned(v_pool, 16))
        return RVQ_ERR_INVALID_ARG;
    return from_hip(rvq::launch_cache_append(heads(k), heads(v), n_tokens, cu, shape->n_clips, shape->kv_heads,
                                             shape->dim, element_bytes(shape->dtype), shape->page_size,
                                             shape->n_pages, shape->table_ld, table, lens, k_pool, v_pool,
                                             static_cast<hipStream_t>(stream)));
}

RVQ_API int64_t rvq_cache_scratch_bytes(int32_t n_clips, int32_t n_pages)
{
    const rvq_status st = check_upkeep(n_clips, 0, 1, n_pages);
    return st != RVQ_OK ? st : rvq::cache_scratch_bytes(n_clips, n_pages);
}

RVQ_API rvq_status rvq_cache_reserve(const int32_t *table, const int32_t *lens, const int32_t *new_lens,
                                     const int32_t *refs, int32_t n_clips, int32_t table_ld, int32_t page_size,
                                     int32_t n_pages, int32_t *table_out, int32_t *refs_out, int32_t *missing,
                                     void *workspace, int64_t workspace_bytes, void *stream)
{
    const rvq_status st = check_upkeep(n_clips, table_ld, page_size, n_pages);
    if (st != RVQ_OK) return st;
    if (!ints(missing) || (n_pages > 0 && (!ints(refs) || !ints(refs_out))) ||
        (n_clips > 0 && (!ints(lens) || !ints(new_lens))) ||
        (n_clips > 0 && table_ld > 0 && (!ints(table) || !ints(table_out))) ||
        !scratch(workspace, workspace_bytes, rvq::cache_scratch_bytes(n_clips, n_pages)))
        return RVQ_ERR_INVALID_ARG;
    return from_hip(rvq::launch_cache_reserve(table, lens, new_lens, refs, n_clips, table_ld, page_size, n_pages,
                                              table_out, refs_out, missing, workspace,
                                              static_cast<hipStream_t>(stream)));
}

RVQ_API rvq_status rvq_cache_fork(const rvq_cache_shape *shape, int32_t n_layers, const int32_t *table,
                                  const int32_t *lens, const int32_t *refs, const int32_t *parents,
                                  const int32_t *children, int32_t n_children, void *k_pool, void *v_pool,
                                  int32_t *table_out, int32_t *lens_out, int32_t *refs_out, int32_t *missing,
                                  void *workspace, int64_t workspace_bytes, void *stream)
{
    rvq_status st = check_cache(shape);
    if (st == RVQ_OK) st = check_upkeep(shape->n_clips, shape->table_ld, shape->page_size, shape->n_pages);
    if (st != RVQ_OK) return st;
    if (n_layers <= 0 || n_children < 0 || n_children > shape->n_clips) return RVQ_ERR_INVALID_ARG;
    const bool clips = shape->n_clips > 0, pages = shape->n_pages > 0, entries = clips && shape->table_ld > 0;
    if (!ints(missing) || (clips && (!ints(lens) || !ints(lens_out))) ||
        (entries && (!ints(table) || !ints(table_out))) ||
        (pages && (!ints(refs) || !ints(refs_out) || !k_pool || !v_pool || !aligned(k_pool, 16) ||
                   !aligned(v_pool, 16))) ||
        (n_children > 0 && (!ints(parents) || !ints(children))) ||
        !scratch(workspace, workspace_bytes, rvq::cache_scratch_bytes(shape->n_clips, shape->n_pages)))
        return RVQ_ERR_INVALID_ARG;
    return from_hip(rvq::launch_cache_fork(table, lens, refs, parents, children, n_children, shape->n_clips,
                                           shape->table_ld, shape->page_size, shape->n_pages, n_layers,
                                           page_bytes(shape), k_pool, v_pool, table_out, lens_out, refs_out,
                                           missing, workspace, static_cast<hipStream_t>(stream)));
}

RVQ_API rvq_status rvq_cache_free(const int32_t *table, const int32_t *lens, const int32_t *refs,
                                  const int32_t *drop, int32_t n_clips, int32_t table_ld, int32_t page_size,
                                  int32_t n_pages, int64_t window, int32_t sinks, int32_t *table_out,
                                  int32_t *lens_out, int32_t *refs_out, void *stream)
{
    const rvq_status st = check_upkeep(n_clips, table_ld, page_size, n_pages);
    if (st != RVQ_OK) return st;
    if (sinks < 0 || (n_clips > 0 && (!ints(lens) || !ints(lens_out))) || (drop && !aligned(drop, 4)) ||
        (n_clips > 0 && table_ld > 0 && (!ints(table) || !ints(table_out))) ||
        (n_pages > 0 && (!ints(refs) || !ints(refs_out))))
        return RVQ_ERR_INVALID_ARG;
    return from_hip(rvq::launch_cache_free(table, lens, refs, drop, n_clips, table_ld, page_size, n_pages, window,
                                           sinks, table_out, lens_out, refs_out,
                                           static_cast<hipStream_t>(stream)));
}

RVQ_API rvq_status rvq_cache_compact(const rvq_cache_shape *shape, int32_t n_layers, const int32_t *table,
                                     const int32_t *refs, void *k_pool, void *v_pool, int32_t *table_out,
                                     int32_t *refs_out, int32_t *live, void *workspace, int64_t workspace_bytes,
                                     void *stream)
{
    rvq_status st = check_cache(shape);
    if (st == RVQ_OK) st = check_upkeep(shape->n_clips, shape->table_ld, shape->page_size, shape->n_pages);
    if (st != RVQ_OK) return st;
    if (n_layers <= 0) return RVQ_ERR_INVALID_ARG;
    if (!ints(live) || (shape->n_clips > 0 && shape->table_ld > 0 && (!ints(table) || !ints(table_out))) ||
        (shape->n_pages > 0 && (!ints(refs) || !ints(refs_out) || !k_pool || !v_pool || !aligned(k_pool, 16) ||
                                !aligned(v_pool, 16))) ||
        !scratch(workspace, workspace_bytes, rvq::cache_scratch_bytes(shape->n_clips, shape->n_pages)))
        return RVQ_ERR_INVALID_ARG;
    return from_hip(rvq::launch_cache_compact(table, refs, shape->n_clips, shape->table_ld, shape->n_pages, n_layers,
                                              page_bytes(shape), k_pool, v_pool, table_out, refs_out, live,
                                              workspace, static_cast<hipStream_t>(stream)));
}

RVQ_API rvq_status rvq_cache_copy(const rvq_cache_shape *shape, int32_t n_layers, const int32_t *src,
                                  const int32_t *dst, int32_t n_copies, void *k_pool, void *v_pool, void *stream)
{
    const rvq_status st = check_cache(shape);
    if (st != RVQ_OK) return st;
    if (n_layers <= 0 || n_copies < 0) return RVQ_ERR_INVALID_ARG;
    if (n_copies == 0 || shape->n_pages == 0) return RVQ_OK;
    if (!ints(src) || !ints(dst) || !k_pool || !v_pool || !aligned(k_pool, 16) || !aligned(v_pool, 16))
        return RVQ_ERR_INVALID_ARG;
    return from_hip(rvq::launch_cache_copy(src, dst, n_copies, shape->n_pages, n_layers, page_bytes(shape), k_pool,
                                           v_pool, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
