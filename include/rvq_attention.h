/*
 * rvq_attention.h -- C ABI of the streaming-attention operators of librvq:
 * windowed and cross attention with their gradients, attention of one new frame over a
 * paged key-value cache and of a chunk of new frames over it, rotary positions,
 * and the upkeep of the cache's pages.
 *
 * These are the operators of the transformers that stand around a residual
 * quantizer and of the models that generate its codes: both run over frames
 * (25 or 12.5 a second), with a bounded view into the past.
 *
 * Conventions are those of rvq.h: plain C99, caller-owned DEVICE memory, no
 * allocation and no state between calls, work enqueued on `stream` (a
 * hipStream_t cast to void*), argument errors reported synchronously before
 * anything is enqueued, status codes of rvq_status. Shapes that take 2^24
 * workgroups or more are refused (RVQ_ERR_UNSUPPORTED). A workgroup is a head
 * of 128 frames or of a clip's rest in the windowed attention, 16 query heads
 * of a key head and clip in the cache attention, 128 queries and heads of a key
 * head, or a clip's few ones, in chunk and cross attention (times the splits of
 * their keys), 8 new frames in an append, 256 times 32 bytes in rotary positions.
 *
 * Which frames a frame sees. A frame at position p of its clip sees the
 * frames j <= p with p - j < window, and of those further back the first
 * `sinks` frames of the clip (j < sinks). A negative window is unbounded;
 * window 0 leaves only the sinks. A frame that sees nothing has output 0,
 * log-sum-exp -inf and gradient 0; so has a frame whose scores are all -inf.
 *
 * Arithmetic. Products run on the matrix cores in the inputs' type with
 * float32 accumulation (float32 inputs: as three bfloat16 parts a value, six
 * products, off by 2^-22 of a product of two values at most and 2^-25 in the
 * mean square, or as float32); scores, softmax statistics and accumulators
 * are float32. Attention weights and score gradients are rounded once to the
 * inputs' type where they enter a matrix product of it (in float16 times a
 * power of two that keeps them within its range; weights of chunk and cross
 * attention as two parts where a clip has few queries), outputs once at the end. No
 * sum's order depends on timing: the same call gives the same bits.
 */
#ifndef RVQ_ATTENTION_H
#define RVQ_ATTENTION_H

#include "rvq.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum rvq_dtype {
    RVQ_F32 = 0,
    RVQ_F16 = 1,
    RVQ_BF16 = 2
} rvq_dtype;

/*
 * A packed array of heads: element (t, h, d) is at
 * data[t * token_stride + h * head_stride + d], strides in elements. data and
 * both strides must be multiples of 16 bytes, token_stride below 2^23 - 16
 * elements; rows may be slices of a wider
 * array (a fused projection's output). Output rows must not overlap each
 * other or an input.
 */
typedef struct rvq_heads {
    void *data;
    int64_t token_stride;
    int64_t head_stride;
} rvq_heads;

/*
 * Shapes shared by the windowed attention and its gradient. Clips are packed:
 * clip b has the queries cu_q[b] .. cu_q[b+1]-1 and the keys cu_k[b] ..
 * cu_k[b+1]-1 (device int32 [n_clips + 1], non-decreasing, within
 * 0..q_tokens / 0..k_tokens). Its queries are the last ones of its keys'
 * positions: query i of n_q is at position i + n_k - n_q. Rows outside every
 * clip have no influence and are not written. Offsets that break these rules
 * give unspecified results, but no access outside the arrays.
 *
 * dim must be 64 or 128, q_heads a multiple of kv_heads (query head h reads
 * key head h / (q_heads / kv_heads)); scale >= 0 and finite.
 */
typedef struct rvq_attention_shape {
    int32_t dtype;      /* rvq_dtype of q, k, v, out and the gradients */
    int32_t n_clips;
    int32_t q_heads;
    int32_t kv_heads;
    int32_t dim;
    int32_t sinks;
    int64_t window;
    int64_t q_tokens;
    int64_t k_tokens;
    const int32_t *cu_q;
    const int32_t *cu_k;
    float scale;
} rvq_attention_shape;

/*
 * rvq_window_attention -- out = softmax(scale q k^T over the frames seen) v.
 *
 *   q, out  [q_tokens, q_heads, dim]
 *   k, v    [k_tokens, kv_heads, dim]
 *   lse     [q_heads, q_tokens] float32, the log of each softmax's sum of
 *           exponentials (natural log); NULL to skip it
 *
 * A value that a frame does not see has no influence on its output, not even
 * where it is infinite or NaN. A seen one that is infinite makes the output
 * infinite there, with its sign; NaN or infinities of both signs make it NaN.
 */
RVQ_API rvq_status rvq_window_attention(const rvq_attention_shape *shape, const rvq_heads *q, const rvq_heads *k,
                                        const rvq_heads *v, const rvq_heads *out, float *lse, void *stream);

/*
 * rvq_window_attention_backward -- gradients of the above.
 *
 *   dout, q, k, v   as in the forward pass, dout laid out like out
 *   out, lse        what the forward pass gave
 *   dq, dk, dv      outputs, laid out like q, k, v; keys and values shared
 *                   by several query heads get the sum over them. A value of q, k, v or
 *                   dout that is not finite reaches the gradients of the
 *                   queries that see it and of the keys they see, no others
 *   workspace       device memory of at least
 *                   rvq_window_attention_backward_bytes(shape) bytes,
 *                   16-byte aligned (the size is a negative rvq_status for
 *                   shapes that are refused)
 */
RVQ_API int64_t rvq_window_attention_backward_bytes(const rvq_attention_shape *shape);
RVQ_API rvq_status rvq_window_attention_backward(const rvq_attention_shape *shape, const rvq_heads *dout,
                                                 const rvq_heads *q, const rvq_heads *k, const rvq_heads *v,
                                                 const rvq_heads *out, const float *lse,
                                                 const rvq_heads *dq, const rvq_heads *dk, const rvq_heads *dv,
                                                 void *workspace, int64_t workspace_bytes, void *stream);

/*
 * rvq_cross_attention -- every query sees all keys of its clip: attention to
 * an encoder's states, or without a mask within clips. The shape as above, but
 * that window and sinks are not read and that queries and keys of a clip have
 * no common positions; cu_q may be NULL: one query a clip, q_tokens ==
 * n_clips (the next frame of every clip). A clip without keys has output 0,
 * lse -inf and gradient 0. k_tokens may be 0.
 *
 *   workspace       device memory of at least rvq_cross_attention_bytes(shape)
 *                   bytes, 16-byte aligned (NULL where that is 0)
 *
 * A value that is not finite reaches the results of its own clip alone: as
 * above an infinite one makes the output infinite there, with its sign, NaN or
 * infinities of both signs make it NaN.
 * Padded batches: a clip's rows have to follow one another, so rows of padding
 * may stand behind the last clip or before the first only.
 *
 * rvq_cross_attention_backward -- its gradients, as rvq_window_attention_backward;
 * cu_q must be given.
 */
RVQ_API int64_t rvq_cross_attention_bytes(const rvq_attention_shape *shape);
RVQ_API rvq_status rvq_cross_attention(const rvq_attention_shape *shape, const rvq_heads *q, const rvq_heads *k,
                                       const rvq_heads *v, const rvq_heads *out, float *lse, void *workspace,
                                       int64_t workspace_bytes, void *stream);
RVQ_API int64_t rvq_cross_attention_backward_bytes(const rvq_attention_shape *shape);
RVQ_API rvq_status rvq_cross_attention_backward(const rvq_attention_shape *shape, const rvq_heads *dout,
                                                const rvq_heads *q, const rvq_heads *k, const rvq_heads *v,
                                                const rvq_heads *out, const float *lse,
                                                const rvq_heads *dq, const rvq_heads *dk, const rvq_heads *dv,
                                                void *workspace, int64_t workspace_bytes, void *stream);

/*
 * A paged key-value cache. Pools hold pages [n_pages, kv_heads, page_size,
 * dim], dense and 16-byte aligned; a deep stack keeps one pool of each kind,
 * [n_layers, n_pages, kv_heads, page_size, dim], and one table for all
 * layers. table [n_clips, table_ld] int32 names the page that holds a clip's
 * frames e * page_size .. (e + 1) * page_size - 1 in column e, -1 for none.
 * lens [n_clips] int32 counts a clip's frames in the cache.
 *
 * refs [n_pages] int32 counts the table entries that name a page; a page
 * with count 0 is free. Pages are handed out lowest number first, so every
 * operation's result is determined by its inputs. A page that is still being
 * written (its clip's last, not full) is never shared.
 *
 * Page numbers outside [0, n_pages) are never followed.
 */
typedef struct rvq_cache_shape {
    int32_t dtype;      /* rvq_dtype of the pools and of q, k, v, out */
    int32_t n_clips;
    int32_t kv_heads;
    int32_t dim;        /* 64 or 128 */
    int32_t page_size;  /* frames a page, 1 or more */
    int32_t n_pages;
    int32_t table_ld;   /* columns of table */
} rvq_cache_shape;

/*
 * rvq_cache_append -- writes new frames' keys and values into their pages.
 *
 *   k, v    [n_tokens, kv_heads, dim], packed by clip
 *   cu      [n_clips + 1] int32: clip b's new frames are cu[b] .. cu[b+1]-1;
 *           NULL: one new frame each, n_tokens == n_clips
 *   lens    counts before the append: new frame i of clip b goes to position
 *           lens[b] + i; the caller adds the new counts to lens itself
 *
 * A frame whose position has no page in the table is dropped.
 */
RVQ_API rvq_status rvq_cache_append(const rvq_cache_shape *shape, const rvq_heads *k, const rvq_heads *v,
                                    int64_t n_tokens, const int32_t *cu, const int32_t *table, const int32_t *lens,
                                    void *k_pool, void *v_pool, void *stream);

/*
 * rvq_cache_attention -- attention of every clip's newest frame.
 *
 *   q, out     [n_clips, q_heads, dim] (token = clip); q_heads a multiple of
 *              kv_heads
 *   lens       counts with the newest frame, whose key and value are in the
 *              cache: the query's position is lens[b] - 1; a clip with count
 *              0 gets output 0
 *   window, sinks, scale   as in rvq_window_attention
 *   workspace  device memory of at least rvq_cache_attention_bytes(shape,
 *              q_heads) bytes, 16-byte aligned (NULL where that is 0)
 *
 * Only pages with frames that are seen are read; the table may hold -1 for
 * the others. A clip that sees a frame without a valid page (a table entry
 * outside [0, n_pages), a count beyond the table) gets all quiet NaN.
 */
RVQ_API int64_t rvq_cache_attention_bytes(const rvq_cache_shape *shape, int32_t q_heads);
RVQ_API rvq_status rvq_cache_attention(const rvq_cache_shape *shape, int32_t q_heads, const rvq_heads *q,
                                       const void *k_pool, const void *v_pool, const int32_t *table,
                                       const int32_t *lens, int64_t window, int32_t sinks, float scale,
                                       const rvq_heads *out, void *workspace, int64_t workspace_bytes, void *stream);

/*
 * rvq_cache_chunk_attention -- attention of every clip's newest frames, as
 * many as each has: drafted frames that are looked at together, the next
 * piece of a long recording, single frames of some clips beside whole chunks of
 * others.
 *
 *   q, out     [n_tokens, q_heads, dim], packed by clip
 *   cu         [n_clips + 1] int32: clip b's queries are cu[b] .. cu[b+1]-1
 *              (non-decreasing, within 0..n_tokens; rows outside every clip
 *              are not written); NULL: one query each, n_tokens == n_clips
 *              (what rvq_cache_attention does, as fast, with lse and with weights
 *              in two parts)
 *   lens       counts with the new frames, whose keys and values are in the
 *              cache: query i of n is at position lens[b] - n + i. Queries at
 *              negative positions see nothing
 *   lse        [q_heads, n_tokens] float32 as in rvq_window_attention, or NULL
 *   window, sinks, scale   as in rvq_window_attention
 *   workspace  device memory of at least rvq_cache_chunk_attention_bytes(shape,
 *              q_heads, n_tokens) bytes, 16-byte aligned (NULL where that is 0)
 *
 * Only pages with frames that are seen need to be there. A query that sees a
 * frame without a valid page gets quiet NaN, and so do all queries of a clip
 * whose count is beyond the table. A value that a query does not see has no
 * influence on its output, not even where it is infinite or NaN; a seen one
 * that is infinite makes the output infinite there, with its sign, NaN or
 * infinities of both signs make it NaN (a key with score -inf is not seen).
 */
RVQ_API int64_t rvq_cache_chunk_attention_bytes(const rvq_cache_shape *shape, int32_t q_heads, int64_t n_tokens);
RVQ_API rvq_status rvq_cache_chunk_attention(const rvq_cache_shape *shape, int32_t q_heads, int64_t n_tokens,
                                             const int32_t *cu, const rvq_heads *q, const void *k_pool,
                                             const void *v_pool, const int32_t *table, const int32_t *lens,
                                             int64_t window, int32_t sinks, float scale, const rvq_heads *out,
                                             float *lse, void *workspace, int64_t workspace_bytes, void *stream);

/*
 * Rotary positions. Of every head's first rot_dim values (even, 2..dim) pair
 * i turns by the angle position * frequencies[i]: (a, b) becomes amplitude *
 * (a cos - b sin, b cos + a sin). The pairs are the values i and rot_dim / 2
 * + i, or 2 i and 2 i + 1 where interleaved != 0; the values behind rot_dim
 * stay as they are. With inverse != 0 the angles are negative: the gradient of
 * the same call without it. frequencies [rot_dim / 2] are radians a position,
 * device float64; angles are taken in two float64 parts, known to 2^-50 of a
 * turn, so far positions lose nothing.
 */
typedef struct rvq_rotation {
    const double *frequencies;
    int32_t rot_dim;
    int32_t interleaved;
    int32_t inverse;
    float amplitude;    /* finite */
} rvq_rotation;

/*
 * rvq_rotary_frequencies -- base^(-2 i / rot_dim) for i < rot_dim / 2, scaled
 * for clips longer than a model was trained on. HOST memory, no GPU involved.
 *
 *   RVQ_ROTARY_PLAIN   as they are
 *   RVQ_ROTARY_LINEAR  all divided by factor (positions are)
 *   RVQ_ROTARY_BASE    base times factor^(rot_dim / (rot_dim - 2)): the last
 *                      pair's frequency is divided by factor, the first stays
 *   RVQ_ROTARY_RAMP    pairs that turn at least `fast` times within `context`
 *                      positions stay, those that turn at most `slow` times
 *                      are divided by factor, between them in proportion to
 *                      the turns
 *
 * base and factor must be positive; slow < fast and context > 0 (RAMP only,
 * else not read).
 */
typedef enum rvq_rotary_scaling {
    RVQ_ROTARY_PLAIN = 0,
    RVQ_ROTARY_LINEAR = 1,
    RVQ_ROTARY_BASE = 2,
    RVQ_ROTARY_RAMP = 3
} rvq_rotary_scaling;

RVQ_API rvq_status rvq_rotary_frequencies(int32_t rot_dim, double base, int32_t scaling, double factor,
                                          double context, double slow, double fast, double *frequencies);

/*
 * rvq_rotary -- turns packed queries and keys, in one launch.
 *
 *   q, q_out   [n_tokens, q_heads, dim]; q_heads 0: none (NULL)
 *   k, k_out   [n_tokens, kv_heads, dim]; kv_heads 0: none (NULL)
 *   positions  [n_tokens] int32, or NULL: frame i of clip b (rows cu[b] ..
 *              cu[b+1]-1) is at position first[b] + i (first [n_clips] int32,
 *              NULL: 0). Rows outside every clip are not written.
 *
 * dim must be 64 or 128. An output may be its input (the same data and
 * strides); otherwise outputs must not overlap inputs.
 */
RVQ_API rvq_status rvq_rotary(const rvq_rotation *rotation, int32_t dtype, int64_t n_tokens, int32_t q_heads,
                              int32_t kv_heads, int32_t dim, int32_t n_clips, const int32_t *cu, const int32_t *first,
                              const int32_t *positions, const rvq_heads *q, const rvq_heads *k,
                              const rvq_heads *q_out, const rvq_heads *k_out, void *stream);

/*
 * rvq_rotary_append -- rvq_cache_append with rotary positions: new frame i of
 * clip b is at position lens[b] + i. Its queries are turned into q_out (which
 * may be q), its keys on their way into the pages; values go there as they
 * are. q_heads 0: keys and values alone. Frames whose position has no page
 * are dropped, but their queries are turned. rotation->inverse must be 0.
 */
RVQ_API rvq_status rvq_rotary_append(const rvq_cache_shape *shape, const rvq_rotation *rotation, int32_t q_heads,
                                     const rvq_heads *q, const rvq_heads *k, const rvq_heads *v, int64_t n_tokens,
                                     const int32_t *cu, const int32_t *table, const int32_t *lens,
                                     const rvq_heads *q_out, void *k_pool, void *v_pool, void *stream);

/*
 * Upkeep of the pages. Each operation reads its inputs and writes new table,
 * lens and refs (`*_out`, the same shapes). No output may overlap an input
 * or another output. workspace: at least rvq_cache_scratch_bytes(n_clips,
 * n_pages) bytes, 16-byte aligned.
 *
 * rvq_cache_reserve gives every clip pages for positions lens[b] ..
 * new_lens[b] - 1, in order of clips and positions, in the columns behind
 * that of position lens[b] - 1. Columns that name a page keep it, so pages
 * may be reserved ahead, and a call that found too few may be made again with
 * its results. missing [1] int32 counts the pages that were wanted and not
 * there (none free, or a position beyond the table); their entries stay as
 * they were.
 *
 * rvq_cache_fork lets clip children[c] go on from clip parents[c], for all c
 * at once (the step of a beam search when children are all clips). The child
 * lets go of its own pages, shares the parent's full pages and gets a copy
 * of the parent's partial page in a page that is free beforehand, in all
 * n_layers of both pools. Parents are read as they were before the call;
 * children must be distinct. A pair with a clip outside [0, n_clips) is
 * skipped. missing [1] counts the children whose partial page found no room
 * (entry -1). Where the parent itself has no partial page the child has none
 * either (entry -1, not counted). Pages that the parent has reserved ahead
 * stay its own: the child's columns behind its frames are -1.
 *
 * rvq_cache_free lets go of all pages of the clips with drop[b] != 0 (NULL:
 * none), whose count becomes 0, and, with window >= 0, of the pages that no
 * later frame of the other clips will see (window, sinks as above).
 *
 * rvq_cache_compact moves the pages in use to the numbers 0 .. live - 1, in
 * all layers: only pages with a number of live or more move, the k-th of
 * them into the k-th free page. live [1] is the count of pages in use.
 *
 * rvq_cache_copy copies page src[i] to page dst[i] for i < n_copies, in all
 * layers; pairs with a number outside [0, n_pages) are skipped, and a page
 * must not be both a source and a target or a target twice.
 */
RVQ_API int64_t rvq_cache_scratch_bytes(int32_t n_clips, int32_t n_pages);
RVQ_API rvq_status rvq_cache_reserve(const int32_t *table, const int32_t *lens, const int32_t *new_lens,
                                     const int32_t *refs, int32_t n_clips, int32_t table_ld, int32_t page_size,
                                     int32_t n_pages, int32_t *table_out, int32_t *refs_out, int32_t *missing,
                                     void *workspace, int64_t workspace_bytes, void *stream);
RVQ_API rvq_status rvq_cache_fork(const rvq_cache_shape *shape, int32_t n_layers, const int32_t *table,
                                  const int32_t *lens, const int32_t *refs, const int32_t *parents,
                                  const int32_t *children, int32_t n_children, void *k_pool, void *v_pool,
                                  int32_t *table_out, int32_t *lens_out, int32_t *refs_out, int32_t *missing,
                                  void *workspace, int64_t workspace_bytes, void *stream);
RVQ_API rvq_status rvq_cache_free(const int32_t *table, const int32_t *lens, const int32_t *refs,
                                  const int32_t *drop, int32_t n_clips, int32_t table_ld, int32_t page_size,
                                  int32_t n_pages, int64_t window, int32_t sinks, int32_t *table_out,
                                  int32_t *lens_out, int32_t *refs_out, void *stream);
RVQ_API rvq_status rvq_cache_compact(const rvq_cache_shape *shape, int32_t n_layers, const int32_t *table,
                                     const int32_t *refs, void *k_pool, void *v_pool, int32_t *table_out,
                                     int32_t *refs_out, int32_t *live, void *workspace, int64_t workspace_bytes,
                                     void *stream);
RVQ_API rvq_status rvq_cache_copy(const rvq_cache_shape *shape, int32_t n_layers, const int32_t *src,
                                  const int32_t *dst, int32_t n_copies, void *k_pool, void *v_pool, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* RVQ_ATTENTION_H */
