// Launch interface between the C ABI layer (attention_api.hip) and the
// streaming-attention kernels. Not installed, not exported.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rvq_attention.h"

namespace rvq {

// A packed array of heads on the device: element (t, h, d) at data + t * token + h * head + d.
struct Heads {
    void *data;
    int64_t token;
    int64_t head;
};

struct AttentionArgs {
    int dtype, dim, n_clips, q_heads, kv_heads;
    int window, sinks;            // window INT32_MAX: unbounded
    int64_t q_tokens, k_tokens;   // below 2^31
    const int32_t *cu_q, *cu_k;
    float scale;
    Heads q, k, v, out;
    float *lse;                   // nullable in the forward pass
    Heads dout, dq, dk, dv;       // backward only
    void *workspace;
};

struct CacheAttentionArgs {
    int dtype, dim, n_clips, q_heads, kv_heads;
    int page_size, n_pages, table_ld;
    int window, sinks;
    float scale;
    Heads q, out;
    const void *k_pool, *v_pool;
    const int32_t *table, *lens;
    void *workspace;
};

// A launch holds fewer than 2^32 threads. Launches that need more are refused with hipErrorNotSupported before any other.
inline bool fits(int64_t groups, int threads) { return groups <= 0xffffffffll / threads; }

hipError_t launch_window_attention(const AttentionArgs &a, hipStream_t stream);
int64_t window_attention_backward_bytes(const AttentionArgs &a);     // of the shape alone
hipError_t launch_window_attention_backward(const AttentionArgs &a, hipStream_t stream);

int64_t cache_attention_bytes(int n_clips, int q_heads, int kv_heads, int dim, int64_t capacity);
hipError_t launch_cache_attention(const CacheAttentionArgs &a, hipStream_t stream);

// element_bytes: size of one cache value; rows of dim values are copied whole.
hipError_t launch_cache_append(const Heads &k, const Heads &v, int64_t n_tokens, const int32_t *cu, int n_clips,
                               int kv_heads, int dim, int element_bytes, int page_size, int n_pages, int table_ld,
                               const int32_t *table, const int32_t *lens, void *k_pool, void *v_pool,
                               hipStream_t stream);

int64_t cache_scratch_bytes(int n_clips, int n_pages);
hipError_t launch_cache_reserve(const int32_t *table, const int32_t *lens, const int32_t *new_lens,
                                const int32_t *refs, int n_clips, int table_ld, int page_size, int n_pages,
                                int32_t *table_out, int32_t *refs_out, int32_t *missing, void *workspace,
                                hipStream_t stream);
hipError_t launch_cache_fork(const int32_t *table, const int32_t *lens, const int32_t *refs, const int32_t *parents,
                             const int32_t *children, int n_children, int n_clips, int table_ld, int page_size,
                             int n_pages, int n_layers, int64_t page_bytes, void *k_pool, void *v_pool,
                             int32_t *table_out, int32_t *lens_out, int32_t *refs_out, int32_t *missing,
                             void *workspace, hipStream_t stream);
hipError_t launch_cache_free(const int32_t *table, const int32_t *lens, const int32_t *refs, const int32_t *drop,
                             int n_clips, int table_ld, int page_size, int n_pages, int64_t window, int sinks,
                             int32_t *table_out, int32_t *lens_out, int32_t *refs_out, hipStream_t stream);
hipError_t launch_cache_compact(const int32_t *table, const int32_t *refs, int n_clips, int table_ld, int n_pages,
                                int n_layers, int64_t page_bytes, void *k_pool, void *v_pool, int32_t *table_out,
                                int32_t *refs_out, int32_t *live, void *workspace, hipStream_t stream);
hipError_t launch_cache_copy(const int32_t *src, const int32_t *dst, int n_copies, int n_pages, int n_layers,
                             int64_t page_bytes, void *k_pool, void *v_pool, hipStream_t stream);

}  // namespace rvq
