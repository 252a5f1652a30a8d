// Gradient of the windowed attention with sinks.
//
//   x_ij = scale q_i . k_j over the keys j that query i sees,
//   w = softmax(x), out_i = sum_j w_ij v_j, lse_i = log sum_j exp(x_ij)
//   delta_i = dout_i . out_i,  dw_ij = dout_i . v_j,  dx_ij = w_ij (dw_ij - delta_i)
//   dq_i = scale sum_j dx_ij k_j,  dk_j = scale sum_i dx_ij q_i,  dv_j = sum_i w_ij dout_i
//
// One wavefront a row: a query with its keys one after another (dq)
// or a key with the queries that see it (dk, dv), lanes over the head dim.
#include <limits.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "attention_device.h"
#include "attention_internal.h"

namespace rvq {
namespace {

constexpr int kRowsPerBlock = 4;

template <typename T, int kD>
__device__ inline void load_row(const Heads &h, int64_t row, int head, int lane, float (&x)[kD / 64])
{
    const T *p = static_cast<const T *>(h.data) + row * h.token + head * h.head;
#pragma unroll
    for (int i = 0; i < kD / 64; ++i) x[i] = to_float(p[lane + 64 * i]);
}

template <typename T, int kD>
__device__ inline void store_row(const Heads &h, int64_t row, int head, int lane, const float (&x)[kD / 64])
{
    T *p = static_cast<T *>(h.data) + row * h.token + head * h.head;
#pragma unroll
    for (int i = 0; i < kD / 64; ++i) p[lane + 64 * i] = static_cast<T>(x[i]);
}

template <int kN>
__device__ inline float dot(const float (&x)[kN], const float (&y)[kN])
{
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kN; ++i) s += x[i] * y[i];
    return wave_sum(s);
}

__device__ inline bool find_row(const int32_t *cu, int n_clips, int64_t tokens, int row, int &clip)
{
    int first, count;
    clip = clip_of_row(cu, n_clips, row);
    clip_range(cu, clip, tokens, first, count);
    return row >= first && row < first + count;
}

// delta[head, row] = dout . out
template <typename T, int kD>
__global__ __launch_bounds__(64 * kRowsPerBlock)
void delta_rows(AttentionArgs a)
{
    const int lane = threadIdx.x & 63;
    const int row = blockIdx.x * kRowsPerBlock + (threadIdx.x >> 6), head = blockIdx.y;
    int clip;
    if (row >= a.q_tokens || !find_row(a.cu_q, a.n_clips, a.q_tokens, row, clip)) return;
    float g[kD / 64], o[kD / 64];
    load_row<T, kD>(a.dout, row, head, lane, g);
    load_row<T, kD>(a.out, row, head, lane, o);
    const float s = dot(g, o);
    if (lane == 0) static_cast<float *>(a.workspace)[static_cast<int64_t>(head) * a.q_tokens + row] = s;
}

template <typename T, int kD>
__global__ __launch_bounds__(64 * kRowsPerBlock)
void dq_rows(AttentionArgs a)
{
    const int lane = threadIdx.x & 63;
    const int row = blockIdx.x * kRowsPerBlock + (threadIdx.x >> 6), head = blockIdx.y;
    if (row >= a.q_tokens) return;
    int clip, q0, nq, k0, nk;
    if (!find_row(a.cu_q, a.n_clips, a.q_tokens, row, clip)) return;
    clip_range(a.cu_q, clip, a.q_tokens, q0, nq);
    clip_range(a.cu_k, clip, a.k_tokens, k0, nk);
    const int kv = head / (a.q_heads / a.kv_heads);
    const int p = row - q0 + nk - nq;
    const int64_t first = static_cast<int64_t>(p) - a.window + 1;
    const int64_t at = static_cast<int64_t>(head) * a.q_tokens + row;
    const float lse = a.lse[at], delta = static_cast<const float *>(a.workspace)[at];
    float q[kD / 64], k[kD / 64], v[kD / 64], g[kD / 64], dq[kD / 64] = {};
    load_row<T, kD>(a.q, row, head, lane, q);
    load_row<T, kD>(a.dout, row, head, lane, g);
    if (lse != -INFINITY) {
        for (int j = 0; j <= p; ++j) {
            if (j < first && j >= a.sinks) {
                j = static_cast<int>(first) - 1;
                continue;
            }
            load_row<T, kD>(a.k, k0 + j, kv, lane, k);
            load_row<T, kD>(a.v, k0 + j, kv, lane, v);
            const float w = exp2f((dot(q, k) * a.scale - lse) * kLog2e);
            const float dx = w * (dot(g, v) - delta) * a.scale;
#pragma unroll
            for (int i = 0; i < kD / 64; ++i) dq[i] += dx * k[i];
        }
    }
    store_row<T, kD>(a.dq, row, head, lane, dq);
}

template <typename T, int kD>
__global__ __launch_bounds__(64 * kRowsPerBlock)
void dkv_rows(AttentionArgs a)
{
    const int lane = threadIdx.x & 63;
    const int row = blockIdx.x * kRowsPerBlock + (threadIdx.x >> 6), kv = blockIdx.y;
    if (row >= a.k_tokens) return;
    int clip, q0, nq, k0, nk;
    if (!find_row(a.cu_k, a.n_clips, a.k_tokens, row, clip)) return;
    clip_range(a.cu_q, clip, a.q_tokens, q0, nq);
    clip_range(a.cu_k, clip, a.k_tokens, k0, nk);
    const int j = row - k0, group = a.q_heads / a.kv_heads;
    const int64_t last = j < a.sinks ? nk : static_cast<int64_t>(j) + a.window;   // positions below it see j
    float q[kD / 64], k[kD / 64], v[kD / 64], g[kD / 64], dk[kD / 64] = {}, dv[kD / 64] = {};
    load_row<T, kD>(a.k, row, kv, lane, k);
    load_row<T, kD>(a.v, row, kv, lane, v);
    for (int h = kv * group; h < (kv + 1) * group; ++h) {
        for (int64_t p = max(j, nk - nq); p < min(static_cast<int64_t>(nk), last); ++p) {
            const int64_t qr = q0 + p - (nk - nq), at = h * a.q_tokens + qr;
            const float lse = a.lse[at], delta = static_cast<const float *>(a.workspace)[at];
            if (lse == -INFINITY) continue;
            load_row<T, kD>(a.q, qr, h, lane, q);
            load_row<T, kD>(a.dout, qr, h, lane, g);
            const float w = exp2f((dot(q, k) * a.scale - lse) * kLog2e);
            const float dx = w * (dot(g, v) - delta) * a.scale;
#pragma unroll
            for (int i = 0; i < kD / 64; ++i) {
                dk[i] += dx * q[i];
                dv[i] += w * g[i];
            }
        }
    }
    store_row<T, kD>(a.dk, row, kv, lane, dk);
    store_row<T, kD>(a.dv, row, kv, lane, dv);
}

unsigned blocks(int64_t rows) { return static_cast<unsigned>((rows + kRowsPerBlock - 1) / kRowsPerBlock); }

template <typename T, int kD>
hipError_t backward(const AttentionArgs &a, hipStream_t stream)
{
    if (a.q_tokens > 0) {
        delta_rows<T, kD><<<dim3(blocks(a.q_tokens), a.q_heads), 64 * kRowsPerBlock, 0, stream>>>(a);
        dq_rows<T, kD><<<dim3(blocks(a.q_tokens), a.q_heads), 64 * kRowsPerBlock, 0, stream>>>(a);
    }
    if (a.k_tokens > 0)
        dkv_rows<T, kD><<<dim3(blocks(a.k_tokens), a.kv_heads), 64 * kRowsPerBlock, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

int64_t window_attention_backward_bytes(int64_t q_tokens, int64_t k_tokens, int n_clips, int q_heads, int kv_heads,
                                        int dim, int sinks)
{
    return q_tokens * q_heads * 4;
}

hipError_t launch_window_attention_backward(const AttentionArgs &a, hipStream_t stream)
{
    if (a.dtype == RVQ_F32) return a.dim == 64 ? backward<float, 64>(a, stream) : backward<float, 128>(a, stream);
    if (a.dtype == RVQ_F16) return a.dim == 64 ? backward<f16_t, 64>(a, stream) : backward<f16_t, 128>(a, stream);
    return a.dim == 64 ? backward<bf16_t, 64>(a, stream) : backward<bf16_t, 128>(a, stream);
}

}  // namespace rvq
