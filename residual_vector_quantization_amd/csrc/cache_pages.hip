// Upkeep of a paged key-value cache: append, reserve, fork, free, compact, copy.
//
// Page numbers are handed out lowest first, so free pages are ranked by a
// prefix count over refs: every chunk of kChunk pages is counted by its own
// workgroup, then each workgroup adds up the counts before its chunk and
// ranks its pages. Only integer atomics (reference counts) are used, whose
// order changes nothing. Page contents move in 16-byte pieces, one read and
// one write of every byte.
#include <limits.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "attention_device.h"
#include "attention_internal.h"

namespace rvq {
namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 8;
constexpr int kChunk = kThreads * kPerThread;      // pages a ranking workgroup
constexpr int kCopyBlocks = 2048;                  // workgroups that copy pages (8 a CU)

int64_t chunks(int n) { return (static_cast<int64_t>(n) + kChunk - 1) / kChunk; }

unsigned ceil_div(int64_t n, int64_t per) { return static_cast<unsigned>((n + per - 1) / per); }

// Scratch: counts a chunk, totals, first wanted rank a clip, two page lists and a rank a page.
struct Scratch {
    int32_t *counts;     // [chunks]
    int32_t *totals;     // [4]
    int32_t *base;       // [n_clips + 1]
    int32_t *sources;    // [n_pages + n_clips]
    int32_t *targets;    // [n_pages + n_clips]
    int32_t *rank;       // [n_pages]
};

int64_t rounded(int64_t n) { return (n + 3) / 4 * 4; }

int64_t scratch_ints(int n_clips, int n_pages)
{
    return rounded(chunks(n_pages)) + 4 + rounded(n_clips + 1) + 2 * rounded(static_cast<int64_t>(n_pages) + n_clips) +
           rounded(n_pages);
}

Scratch scratch(void *workspace, int n_clips, int n_pages)
{
    Scratch s;
    s.counts = static_cast<int32_t *>(workspace);
    s.totals = s.counts + rounded(chunks(n_pages));
    s.base = s.totals + 4;
    s.sources = s.base + rounded(n_clips + 1);
    s.targets = s.sources + rounded(static_cast<int64_t>(n_pages) + n_clips);
    s.rank = s.targets + rounded(static_cast<int64_t>(n_pages) + n_clips);
    return s;
}

__device__ inline int wave_inclusive(int x, int lane)
{
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const int y = __shfl_up(x, m);
        if (lane >= m) x += y;
    }
    return x;
}

// Exclusive prefix of x over the workgroup's threads; total gets the sum. Every thread calls it.
__device__ inline int block_exclusive(int x, int &total, int *s_wave)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int inclusive = wave_inclusive(x, lane);
    __syncthreads();
    if (lane == 63) s_wave[wave] = inclusive;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
        before += w < wave ? s_wave[w] : 0;
        total += s_wave[w];
    }
    return before + inclusive - x;
}

// Sum of counts[0 .. n) by the whole workgroup.
__device__ inline int block_total(const int32_t *counts, int n, int *s_wave)
{
    int sum = 0, total;
    for (int i = threadIdx.x; i < n; i += kThreads) sum += counts[i];
    block_exclusive(sum, total, s_wave);
    return total;
}

__device__ inline int pages_for(int len, int page_size) { return len <= 0 ? 0 : (len - 1) / page_size + 1; }

// counts[c] = pages in use in chunk c.
__global__ __launch_bounds__(kThreads)
void count_used(const int32_t *__restrict__ refs, int n_pages, int32_t *__restrict__ counts)
{
    __shared__ int s_wave[kThreads / 64];
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kChunk;
    int used = 0, total;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int64_t p = first + i * kThreads + threadIdx.x;
        used += p < n_pages && refs[p] > 0;
    }
    block_exclusive(used, total, s_wave);
    if (threadIdx.x == 0) counts[blockIdx.x] = total;
}

// base[b] = pages wanted by the clips before b, base[n_clips] their sum, *beyond = pages wanted past the table's
// last column; one workgroup.
__global__ __launch_bounds__(kThreads)
void wanted_before(const int32_t *__restrict__ lens, const int32_t *__restrict__ new_lens, int n_clips,
                   int page_size, int table_ld, int32_t *__restrict__ base, int32_t *__restrict__ beyond)
{
    __shared__ int s_wave[kThreads / 64];
    int before = 0, past = 0, total;
    for (int b0 = 0; b0 < n_clips; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        int want = 0;
        if (b < n_clips) {
            const int had = pages_for(lens[b], page_size), wanted = pages_for(new_lens[b], page_size);
            want = max(0, min(wanted, table_ld) - had);
            past += max(0, wanted - max(had, table_ld));
        }
        const int rank = block_exclusive(want, total, s_wave);
        if (b < n_clips) base[b] = before + rank;
        before += total;
    }
    block_exclusive(past, total, s_wave);
    if (threadIdx.x == 0) {
        base[n_clips] = before;
        *beyond = total;
    }
}

// This thread's kPerThread neighbouring pages of chunk blockIdx.x: how many pages in use precede them.
__device__ inline int used_before(const int32_t *refs, int n_pages, const int32_t *counts, int64_t first,
                                  int (&ref)[kPerThread], int *s_wave)
{
    const int before = block_total(counts, blockIdx.x, s_wave);
    int used = 0, total;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        ref[i] = first + i < n_pages ? refs[first + i] : 0;
        used += ref[i] > 0;
    }
    return before + block_exclusive(used, total, s_wave);
}

// Free pages in order -> list (their first `most`), and refs_out with the first `wanted` of them taken.
__global__ __launch_bounds__(kThreads)
void take_free(const int32_t *__restrict__ refs, int n_pages, const int32_t *__restrict__ counts,
               const int32_t *__restrict__ wanted, int32_t *__restrict__ list, int32_t *__restrict__ refs_out)
{
    __shared__ int s_wave[kThreads / 64];
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kChunk + threadIdx.x * kPerThread;
    int ref[kPerThread];
    int used = used_before(refs, n_pages, counts, first, ref, s_wave);
    const int take = *wanted;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int64_t p = first + i;
        if (p >= n_pages) break;
        const int64_t rank = p - used;
        const bool mine = ref[i] <= 0 && rank < take;
        if (mine) list[rank] = static_cast<int32_t>(p);
        refs_out[p] = mine ? 1 : ref[i];
        used += ref[i] > 0;
    }
}

__device__ inline int free_pages(const int32_t *counts, int n_chunks, int n_pages, int *s_wave)
{
    return n_pages - block_total(counts, n_chunks, s_wave);
}

// table_out = table with the wanted entries filled from the list of free pages; one thread an entry.
__global__ __launch_bounds__(kThreads)
void fill_table(const int32_t *__restrict__ table, const int32_t *__restrict__ lens,
                const int32_t *__restrict__ new_lens, int n_clips, int table_ld, int page_size, int n_pages,
                const int32_t *__restrict__ counts, int n_chunks, const int32_t *__restrict__ base,
                const int32_t *__restrict__ list, int32_t *__restrict__ table_out)
{
    __shared__ int s_wave[kThreads / 64];
    const int n_free = free_pages(counts, n_chunks, n_pages, s_wave);
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (at >= static_cast<int64_t>(n_clips) * table_ld) return;
    const int b = static_cast<int>(at / table_ld), e = static_cast<int>(at - static_cast<int64_t>(b) * table_ld);
    const int had = pages_for(lens[b], page_size), want = pages_for(new_lens[b], page_size);
    int page = table[at];
    if (e >= had && e < want) {
        const int rank = base[b] + e - had;
        if (rank < n_free) page = list[rank];
    }
    table_out[at] = page;
}

// missing = wanted pages that there are not (and those past the table), one workgroup.
__global__ __launch_bounds__(kThreads)
void count_missing(const int32_t *__restrict__ counts, int n_chunks, int n_pages,
                   const int32_t *__restrict__ wanted, const int32_t *__restrict__ beyond,
                   int32_t *__restrict__ missing)
{
    __shared__ int s_wave[kThreads / 64];
    const int n_free = free_pages(counts, n_chunks, n_pages, s_wave);
    if (threadIdx.x == 0) *missing = max(0, *wanted - n_free) + (beyond ? *beyond : 0);
}

// fork, first step: which children want a page of their own for a partial page, in order; one workgroup.
__device__ inline bool wants_part(const int32_t *lens, int parent, int child, int n_clips, int table_ld, int page_size)
{
    if (static_cast<unsigned>(parent) >= static_cast<unsigned>(n_clips) ||
        static_cast<unsigned>(child) >= static_cast<unsigned>(n_clips))
        return false;
    const int n = max(lens[parent], 0);
    return n % page_size != 0 && n / page_size < table_ld;
}

__global__ __launch_bounds__(kThreads)
void wanted_parts(const int32_t *__restrict__ lens, const int32_t *__restrict__ parents,
                  const int32_t *__restrict__ children, int n_children, int n_clips, int table_ld, int page_size,
                  int32_t *__restrict__ base)
{
    __shared__ int s_wave[kThreads / 64];
    int before = 0;
    for (int c0 = 0; c0 < n_children; c0 += kThreads) {
        const int c = c0 + threadIdx.x;
        int total;
        const int want = c < n_children && wants_part(lens, parents[c], children[c], n_clips, table_ld, page_size);
        const int rank = block_exclusive(want, total, s_wave);
        if (c < n_children) base[c] = before + rank;
        before += total;
    }
    if (threadIdx.x == 0) base[n_clips] = before;
}

__global__ __launch_bounds__(kThreads)
void copy_ints(const int32_t *__restrict__ from, int32_t *__restrict__ to, int64_t n)
{
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (i < n) to[i] = from[i];
}

// fork, second step: one wavefront a child rewrites its row, counts references and lists its page copy.
__global__ __launch_bounds__(64)
void fork_rows(const int32_t *__restrict__ table, const int32_t *__restrict__ lens,
               const int32_t *__restrict__ parents, const int32_t *__restrict__ children, int n_clips, int table_ld,
               int page_size, int n_pages, const int32_t *__restrict__ counts, int n_chunks,
               const int32_t *__restrict__ base, const int32_t *__restrict__ list, int32_t *__restrict__ table_out,
               int32_t *__restrict__ lens_out, int32_t *__restrict__ refs_out, int32_t *__restrict__ sources,
               int32_t *__restrict__ targets)
{
    const int c = blockIdx.x, lane = threadIdx.x;
    const int parent = parents[c], child = children[c];
    int free_count = 0;
    for (int i = lane; i < n_chunks; i += 64) free_count += counts[i];
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) free_count += __shfl_xor(free_count, m);
    free_count = n_pages - free_count;
    int source = -1, target = -1;
    if (static_cast<unsigned>(parent) < static_cast<unsigned>(n_clips) &&
        static_cast<unsigned>(child) < static_cast<unsigned>(n_clips)) {
        const bool part = wants_part(lens, parent, child, n_clips, table_ld, page_size);
        const int n = lens[parent], own = part ? n / page_size : -1;
        const int fresh = part && base[c] < free_count ? list[base[c]] : -1;
        const int32_t *from = table + static_cast<int64_t>(parent) * table_ld;
        const int32_t *was = table + static_cast<int64_t>(child) * table_ld;
        int32_t *to = table_out + static_cast<int64_t>(child) * table_ld;
        for (int e = lane; e < table_ld; e += 64) {
            const int left = was[e];
            int page = from[e];
            if (static_cast<unsigned>(left) < static_cast<unsigned>(n_pages)) atomicSub(&refs_out[left], 1);
            if (e == own) page = fresh;
            else if (static_cast<unsigned>(page) < static_cast<unsigned>(n_pages)) atomicAdd(&refs_out[page], 1);
            to[e] = page;
        }
        if (lane == 0) lens_out[child] = n;
        if (fresh >= 0) {
            source = from[own];
            target = fresh;
        }
    }
    if (lane == 0) {
        sources[c] = source;
        targets[c] = target;
    }
}

// Copies page sources[i] to targets[i] for i < *count (or n), every layer of both pools; pairs with a number
// outside the pool are skipped. A workgroup takes whole (pair, layer, pool) pages in turn.
__global__ __launch_bounds__(kThreads)
void copy_pages(const int32_t *__restrict__ sources, const int32_t *__restrict__ targets, int n,
                const int32_t *__restrict__ count, int n_pages, int n_layers, int64_t page_bytes, char *k_pool,
                char *v_pool)
{
    if (count) n = min(n, *count);
    const int64_t jobs = static_cast<int64_t>(n) * n_layers * 2;
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const int64_t pair = job / (2 * n_layers);
        const int rest = static_cast<int>(job - pair * 2 * n_layers), layer = rest >> 1;
        const int s = sources[pair], d = targets[pair];
        if (static_cast<unsigned>(s) >= static_cast<unsigned>(n_pages) ||
            static_cast<unsigned>(d) >= static_cast<unsigned>(n_pages))
            continue;
        char *pool = ((rest & 1) ? v_pool : k_pool) + static_cast<int64_t>(layer) * n_pages * page_bytes;
        const u32x4 *from = reinterpret_cast<const u32x4 *>(pool + s * page_bytes);
        u32x4 *to = reinterpret_cast<u32x4 *>(pool + d * page_bytes);
        for (int64_t i = threadIdx.x; i < page_bytes / 16; i += kThreads) to[i] = from[i];
    }
}

// free: what leaves the table, reference counts go down.
__global__ __launch_bounds__(kThreads)
void free_entries(const int32_t *__restrict__ table, const int32_t *__restrict__ lens,
                  const int32_t *__restrict__ drop, int n_clips, int table_ld, int page_size, int n_pages,
                  int64_t window, int sinks, int32_t *__restrict__ table_out, int32_t *__restrict__ lens_out,
                  int32_t *__restrict__ refs_out)
{
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (at < n_clips) lens_out[at] = drop && drop[at] ? 0 : lens[at];
    if (at >= static_cast<int64_t>(n_clips) * table_ld) return;
    const int b = static_cast<int>(at / table_ld), e = static_cast<int>(at - static_cast<int64_t>(b) * table_ld);
    const int64_t low = static_cast<int64_t>(e) * page_size;
    int page = table[at];
    // the next frame stands at position lens[b] and sees the positions above lens[b] - window
    const bool behind = window >= 0 && low >= sinks && low + page_size <= static_cast<int64_t>(lens[b]) - window + 1;
    if ((drop && drop[b]) || behind) {
        if (static_cast<unsigned>(page) < static_cast<unsigned>(n_pages)) atomicSub(&refs_out[page], 1);
        page = -1;
    }
    table_out[at] = page;
}

// compact: pages in use numbered live and more are sources, free pages below live are targets, both in order.
__global__ __launch_bounds__(kThreads)
void list_moves(const int32_t *__restrict__ refs, int n_pages, const int32_t *__restrict__ counts, int n_chunks,
                int32_t *__restrict__ totals, int32_t *__restrict__ sources, int32_t *__restrict__ targets,
                int32_t *__restrict__ rank, int32_t *__restrict__ live_out)
{
    __shared__ int s_wave[kThreads / 64];
    const int live = block_total(counts, n_chunks, s_wave);
    // pages in use below number live
    const int border = live / kChunk;
    int below = block_total(counts, border, s_wave);
    int more = 0, total;
    for (int64_t p = static_cast<int64_t>(border) * kChunk + threadIdx.x; p < live; p += kThreads) more += refs[p] > 0;
    block_exclusive(more, total, s_wave);
    below += total;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kChunk + threadIdx.x * kPerThread;
    int ref[kPerThread];
    int used = used_before(refs, n_pages, counts, first, ref, s_wave);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int64_t p = first + i;
        if (p >= n_pages) break;
        if (p < live && ref[i] <= 0) targets[p - used] = static_cast<int32_t>(p);
        if (p >= live && ref[i] > 0) {
            sources[used - below] = static_cast<int32_t>(p);
            rank[p] = used - below;
        }
        used += ref[i] > 0;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *live_out = live;
        totals[0] = live;
        totals[1] = live - below;    // moves
    }
}

// compact: new numbers in the table, reference counts at the new numbers.
__global__ __launch_bounds__(kThreads)
void renumber(const int32_t *__restrict__ table, int64_t entries, const int32_t *__restrict__ refs, int n_pages,
              const int32_t *__restrict__ totals, const int32_t *__restrict__ sources,
              const int32_t *__restrict__ targets, const int32_t *__restrict__ rank, int32_t *__restrict__ table_out,
              int32_t *__restrict__ refs_out)
{
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int live = totals[0], moves = totals[1];
    if (at < entries) {
        int page = table[at];
        if (page >= live && page < n_pages) page = refs[page] > 0 ? targets[rank[page]] : -1;
        table_out[at] = page;
    }
    if (at < n_pages) {
        const int ref = refs[at];
        if (at >= live) refs_out[at] = 0;
        else if (ref > 0) refs_out[at] = ref;
    }
    if (at < moves) refs_out[targets[at]] = refs[sources[at]];
}

// append: a thread a 16-byte piece of a new frame's key and value rows.
__global__ __launch_bounds__(kThreads)
void append_rows(Heads k, Heads v, int64_t n_tokens, const int32_t *__restrict__ cu, int n_clips, int kv_heads,
                 int pieces, int element_bytes, int page_size, int n_pages, int table_ld,
                 const int32_t *__restrict__ table, const int32_t *__restrict__ lens, char *__restrict__ k_pool,
                 char *__restrict__ v_pool)
{
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int piece = static_cast<int>(at % pieces);
    const int64_t row = at / pieces;
    const int head = static_cast<int>(row % kv_heads);
    const int64_t token = row / kv_heads;
    if (token >= n_tokens) return;
    int clip = static_cast<int>(token), nth = 0;
    if (cu) {
        clip = clip_of_row(cu, n_clips, static_cast<int>(token));
        nth = static_cast<int>(token) - cu[clip];
        if (nth < 0 || token >= cu[clip + 1]) return;    // outside every clip
    }
    const int64_t position = static_cast<int64_t>(lens[clip]) + nth;
    if (position < 0 || position >= static_cast<int64_t>(table_ld) * page_size) return;
    const int e = static_cast<int>(position) / page_size, slot = static_cast<int>(position) - e * page_size;
    const int page = table[static_cast<int64_t>(clip) * table_ld + e];
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(n_pages)) return;
    const int64_t to = (((static_cast<int64_t>(page) * kv_heads + head) * page_size + slot) * pieces + piece) * 16;
    const char *from_k = static_cast<const char *>(k.data) + (token * k.token + head * k.head) * element_bytes;
    const char *from_v = static_cast<const char *>(v.data) + (token * v.token + head * v.head) * element_bytes;
    *reinterpret_cast<u32x4 *>(k_pool + to) = *reinterpret_cast<const u32x4 *>(from_k + piece * 16);
    *reinterpret_cast<u32x4 *>(v_pool + to) = *reinterpret_cast<const u32x4 *>(from_v + piece * 16);
}

hipError_t launch_copy(const int32_t *sources, const int32_t *targets, int64_t most, const int32_t *count, int n_pages,
                       int n_layers, int64_t page_bytes, void *k_pool, void *v_pool, hipStream_t stream)
{
    const int64_t jobs = most * n_layers * 2;
    if (jobs == 0) return hipSuccess;
    copy_pages<<<static_cast<unsigned>(jobs < kCopyBlocks ? jobs : kCopyBlocks), kThreads, 0, stream>>>(
        sources, targets, static_cast<int>(most), count, n_pages, n_layers, page_bytes, static_cast<char *>(k_pool),
        static_cast<char *>(v_pool));
    return hipGetLastError();
}

void launch_copy_ints(const int32_t *from, int32_t *to, int64_t n, hipStream_t stream)
{
    if (n > 0) copy_ints<<<ceil_div(n, kThreads), kThreads, 0, stream>>>(from, to, n);
}

}  // namespace

int64_t cache_scratch_bytes(int n_clips, int n_pages) { return scratch_ints(n_clips, n_pages) * 4; }

hipError_t launch_cache_append(const Heads &k, const Heads &v, int64_t n_tokens, const int32_t *cu, int n_clips,
                               int kv_heads, int dim, int element_bytes, int page_size, int n_pages, int table_ld,
                               const int32_t *table, const int32_t *lens, void *k_pool, void *v_pool,
                               hipStream_t stream)
{
    const int pieces = dim * element_bytes / 16;
    append_rows<<<ceil_div(n_tokens * kv_heads * pieces, kThreads), kThreads, 0, stream>>>(
        k, v, n_tokens, cu, n_clips, kv_heads, pieces, element_bytes, page_size, n_pages, table_ld, table, lens,
        static_cast<char *>(k_pool), static_cast<char *>(v_pool));
    return hipGetLastError();
}

hipError_t launch_cache_reserve(const int32_t *table, const int32_t *lens, const int32_t *new_lens,
                                const int32_t *refs, int n_clips, int table_ld, int page_size, int n_pages,
                                int32_t *table_out, int32_t *refs_out, int32_t *missing, void *workspace,
                                hipStream_t stream)
{
    const Scratch s = scratch(workspace, n_clips, n_pages);
    const int n_chunks = static_cast<int>(chunks(n_pages));
    if (n_chunks) count_used<<<n_chunks, kThreads, 0, stream>>>(refs, n_pages, s.counts);
    wanted_before<<<1, kThreads, 0, stream>>>(lens, new_lens, n_clips, page_size, table_ld, s.base,
                                             s.totals);
    if (n_chunks)
        take_free<<<n_chunks, kThreads, 0, stream>>>(refs, n_pages, s.counts, s.base + n_clips, s.sources, refs_out);
    const int64_t entries = static_cast<int64_t>(n_clips) * table_ld;
    if (entries)
        fill_table<<<ceil_div(entries, kThreads), kThreads, 0, stream>>>(table, lens, new_lens, n_clips, table_ld,
                                                                         page_size, n_pages, s.counts, n_chunks,
                                                                         s.base, s.sources, table_out);
    count_missing<<<1, kThreads, 0, stream>>>(s.counts, n_chunks, n_pages, s.base + n_clips, s.totals, missing);
    return hipGetLastError();
}

hipError_t launch_cache_fork(const int32_t *table, const int32_t *lens, const int32_t *refs, const int32_t *parents,
                             const int32_t *children, int n_children, int n_clips, int table_ld, int page_size,
                             int n_pages, int n_layers, int64_t page_bytes, void *k_pool, void *v_pool,
                             int32_t *table_out, int32_t *lens_out, int32_t *refs_out, int32_t *missing,
                             void *workspace, hipStream_t stream)
{
    const Scratch s = scratch(workspace, n_clips, n_pages);
    const int n_chunks = static_cast<int>(chunks(n_pages));
    if (n_chunks) count_used<<<n_chunks, kThreads, 0, stream>>>(refs, n_pages, s.counts);
    wanted_parts<<<1, kThreads, 0, stream>>>(lens, parents, children, n_children, n_clips, table_ld, page_size, s.base);
    launch_copy_ints(table, table_out, static_cast<int64_t>(n_clips) * table_ld, stream);
    launch_copy_ints(lens, lens_out, n_clips, stream);
    if (n_chunks)
        take_free<<<n_chunks, kThreads, 0, stream>>>(refs, n_pages, s.counts, s.base + n_clips, s.rank, refs_out);
    if (n_children)
        fork_rows<<<n_children, 64, 0, stream>>>(table, lens, parents, children, n_clips, table_ld, page_size, n_pages,
                                                 s.counts, n_chunks, s.base, s.rank, table_out, lens_out, refs_out,
                                                 s.sources, s.targets);
    count_missing<<<1, kThreads, 0, stream>>>(s.counts, n_chunks, n_pages, s.base + n_clips, nullptr, missing);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || n_pages == 0) return e;
    return launch_copy(s.sources, s.targets, n_children, nullptr, n_pages, n_layers, page_bytes, k_pool, v_pool, stream);
}

hipError_t launch_cache_free(const int32_t *table, const int32_t *lens, const int32_t *refs, const int32_t *drop,
                             int n_clips, int table_ld, int page_size, int n_pages, int64_t window, int sinks,
                             int32_t *table_out, int32_t *lens_out, int32_t *refs_out, hipStream_t stream)
{
    launch_copy_ints(refs, refs_out, n_pages, stream);
    const int64_t entries = static_cast<int64_t>(n_clips) * (table_ld > 0 ? table_ld : 1);
    if (entries)
        free_entries<<<ceil_div(entries, kThreads), kThreads, 0, stream>>>(table, lens, drop, n_clips, table_ld,
                                                                           page_size, n_pages, window, sinks,
                                                                           table_out, lens_out, refs_out);
    return hipGetLastError();
}

hipError_t launch_cache_compact(const int32_t *table, const int32_t *refs, int n_clips, int table_ld, int n_pages,
                                int n_layers, int64_t page_bytes, void *k_pool, void *v_pool, int32_t *table_out,
                                int32_t *refs_out, int32_t *live, void *workspace, hipStream_t stream)
{
    const Scratch s = scratch(workspace, n_clips, n_pages);
    const int n_chunks = static_cast<int>(chunks(n_pages));
    if (n_chunks) count_used<<<n_chunks, kThreads, 0, stream>>>(refs, n_pages, s.counts);
    list_moves<<<n_chunks ? n_chunks : 1, kThreads, 0, stream>>>(refs, n_pages, s.counts, n_chunks, s.totals,
                                                                 s.sources, s.targets, s.rank, live);
    const int64_t entries = static_cast<int64_t>(n_clips) * table_ld, most = entries > n_pages ? entries : n_pages;
    if (most)
        renumber<<<ceil_div(most, kThreads), kThreads, 0, stream>>>(table, entries, refs, n_pages, s.totals, s.sources,
                                                                    s.targets, s.rank, table_out, refs_out);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || n_pages == 0) return e;
    return launch_copy(s.sources, s.targets, n_pages / 2, s.totals + 1, n_pages, n_layers, page_bytes, k_pool, v_pool,
                       stream);
}

hipError_t launch_cache_copy(const int32_t *src, const int32_t *dst, int n_copies, int n_pages, int n_layers,
                             int64_t page_bytes, void *k_pool, void *v_pool, hipStream_t stream)
{
    return launch_copy(src, dst, n_copies, nullptr, n_pages, n_layers, page_bytes, k_pool, v_pool, stream);
}

}  // namespace rvq
