// Attention of every clip's newest frame over its paged key-value cache.
//
// One wavefront a clip and query head, lanes over the head dim, the frames
// seen one after another with a running softmax.
#include <limits.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "attention_device.h"
#include "attention_internal.h"

namespace rvq {
namespace {

template <typename T, int kD>
__global__ __launch_bounds__(64)
void newest_frame(CacheAttentionArgs a)
{
    const int lane = threadIdx.x, clip = blockIdx.x, head = blockIdx.y;
    const int kv = head / (a.q_heads / a.kv_heads), len = a.lens[clip];
    const int64_t first = static_cast<int64_t>(len) - a.window;
    const T *q = static_cast<const T *>(a.q.data) + clip * a.q.token + head * a.q.head;
    float x[kD / 64], o[kD / 64] = {};
#pragma unroll
    for (int i = 0; i < kD / 64; ++i) x[i] = to_float(q[lane + 64 * i]);
    float m = -INFINITY, l = 0.0f;
    bool bad = false;
    for (int j = 0; j < len; ++j) {
        if (j < first && j >= a.sinks) {
            j = static_cast<int>(first) - 1;
            continue;
        }
        const int e = j / a.page_size;
        const int page = e < a.table_ld ? a.table[static_cast<int64_t>(clip) * a.table_ld + e] : -1;
        if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.n_pages)) {
            bad = true;
            break;
        }
        const int64_t at = ((static_cast<int64_t>(page) * a.kv_heads + kv) * a.page_size + j % a.page_size) * kD;
        const T *k = static_cast<const T *>(a.k_pool) + at, *v = static_cast<const T *>(a.v_pool) + at;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kD / 64; ++i) s += x[i] * to_float(k[lane + 64 * i]);
        s = wave_sum(s) * a.scale;
        const float top = fmaxf(m, s);
        const float safe = top == -INFINITY ? 0.0f : top;
        const float keep = exp2f((m - safe) * kLog2e), w = exp2f((s - safe) * kLog2e);
        l = l * keep + w;
#pragma unroll
        for (int i = 0; i < kD / 64; ++i) o[i] = o[i] * keep + w * to_float(v[lane + 64 * i]);
        m = top;
    }
    T *out = static_cast<T *>(a.out.data) + clip * a.out.token + head * a.out.head;
#pragma unroll
    for (int i = 0; i < kD / 64; ++i)
        out[lane + 64 * i] = static_cast<T>(bad ? __builtin_nanf("") : l == 0.0f ? 0.0f : o[i] / l);
}

template <typename T, int kD>
hipError_t run(const CacheAttentionArgs &a, hipStream_t stream)
{
    newest_frame<T, kD><<<dim3(a.n_clips, a.q_heads), 64, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

int64_t cache_attention_bytes(int n_clips, int q_heads, int kv_heads, int dim, int64_t capacity) { return 0; }

hipError_t launch_cache_attention(const CacheAttentionArgs &a, hipStream_t stream)
{
    if (a.dtype == RVQ_F32) return a.dim == 64 ? run<float, 64>(a, stream) : run<float, 128>(a, stream);
    if (a.dtype == RVQ_F16) return a.dim == 64 ? run<f16_t, 64>(a, stream) : run<f16_t, 128>(a, stream);
    return a.dim == 64 ? run<bf16_t, 64>(a, stream) : run<bf16_t, 128>(a, stream);
}

}  // namespace rvq
