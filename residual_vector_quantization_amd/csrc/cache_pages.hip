// Upkeep of a paged key-value cache: append, reserve, fork, free, compact, copy.
//
// Page numbers are handed out lowest first, so free pages are ranked by a
// prefix count over refs. A workgroup ranks the kChunk pages of its chunk; what
// precedes them it counts itself in pools of up to kSelfCounted pages (reading
// them again from the L2 costs less than the launch that would count them), or
// finds as counts of the chunks in larger ones. One workgroup ranks what is
// wanted: the columns asked for that name no page yet, or the partial pages of a
// fork's parents. Table entries, pages and the counts of those taken are then
// written by a second launch. Only integer atomics
// (reference counts) are used, whose order changes nothing. Page contents move
// in 16-byte pieces, one read and one write of every byte: bound by HBM.
// Measured: 0.91 GB moved by a compaction in 183 us (5.0 TB/s), 0.54 GB copied by
// a fork of 256 clips in 98 us (5.5 TB/s), 0.22 GB appended in 46 us (4.8 TB/s);
// the ranking launches take 3 to 9 us, a call from Python 10 us at least.
#include <limits.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "attention_device.h"
#include "attention_internal.h"

namespace rvq {
namespace {

typedef int32_t s32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kPerThread = 8;
constexpr int kChunk = kThreads * kPerThread;      // pages a ranking workgroup
constexpr int kCopyBlocks = 2048;                  // workgroups that copy pages (8 a CU)
constexpr int kSoonRead = 2048;                    // table entries up to which a free takes one launch (8 a thread: 4 us)
constexpr int kSelfCounted = 1 << 16;              // pages (and clips) up to which a workgroup counts for itself

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

// Pages in use below number `end`, by the whole workgroup; counts of the chunks, or null to count the pages.
__device__ inline int used_below(const int32_t *refs, const int32_t *counts, int end, int *s_wave)
{
    const int whole = counts ? end / kChunk : 0;
    int sum = 0, total;
    for (int i = threadIdx.x; i < whole; i += kThreads) sum += counts[i];
    const int first = whole * kChunk, fours = reinterpret_cast<uintptr_t>(refs) % 16 == 0 ? (end - first) / 4 : 0;
    const s32x4 *four = reinterpret_cast<const s32x4 *>(refs + first);
#pragma unroll 8
    for (int i = threadIdx.x; i < fours; i += kThreads) {
        const s32x4 x = four[i];
        sum += (x[0] > 0) + (x[1] > 0) + (x[2] > 0) + (x[3] > 0);
    }
    for (int p = first + 4 * fours + threadIdx.x; p < end; p += kThreads) sum += refs[p] > 0;
    block_exclusive(sum, total, s_wave);
    return total;
}

// This thread's kPerThread neighbouring pages from `first` on, and how many pages in use precede them.
__device__ inline int used_before(const int32_t *refs, int n_pages, const int32_t *counts, int chunk, int64_t first,
                                  int (&ref)[kPerThread], int *s_wave)
{
    const int before = used_below(refs, counts, chunk * kChunk, s_wave);
    int used = 0, total;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        ref[i] = first + i < n_pages ? refs[first + i] : 0;
        used += ref[i] > 0;
    }
    return before + block_exclusive(used, total, s_wave);
}

// What a fork or a reserve wants of the free pages.
struct Wanted {
    const int32_t *table, *lens, *new_lens;     // reserve (table and lens: fork too)
    const int32_t *parents, *children;          // fork (new_lens null)
    int n, n_clips, table_ld, page_size;        // n: clips (reserve) or children (fork)
    int n_pages;

    __device__ bool is_page(int page) const { return static_cast<unsigned>(page) < static_cast<unsigned>(n_pages); }

    // reserve: the columns first .. first + count - 1 of clip i hold the positions asked for, `past` more lie beyond the
    // table. Those of them that name a page already want none.
    __device__ int columns(int i, int &first, int &past) const
    {
        const int want = pages_for(new_lens[i], page_size);
        first = pages_for(lens[i], page_size);
        past = max(0, want - max(first, table_ld));
        return max(0, min(want, table_ld) - first);
    }

    // fork: the partial page of item i's parent, to be copied, or -1 for none (full pages only, or none where it should
    // be); full: the number of columns with full pages
    __device__ int partial(int i, int &full) const
    {
        const int parent = parents[i], child = children[i];
        full = 0;
        if (static_cast<unsigned>(parent) >= static_cast<unsigned>(n_clips) ||
            static_cast<unsigned>(child) >= static_cast<unsigned>(n_clips))
            return -1;
        const int len = max(lens[parent], 0), column = len / page_size;
        full = min(column, table_ld);
        if (len % page_size == 0 || column >= table_ld) return -1;
        const int page = table[static_cast<int64_t>(parent) * table_ld + column];
        return is_page(page) ? page : -1;
    }
};

// Scratch totals: pages wanted in the table, wanted beyond it, free; compact: pages in use, moves.
enum Total { kInTable = 0, kBeyond = 1, kFree = 2, kLive = 0, kMoves = 1 };

// base[i] = pages wanted before item i, i <= w.n, and the totals; one workgroup. A reserve's threads share out the
// columns asked for, of kThreads clips at a time: one clip may ask for one column or thousands.
__device__ inline void rank_wanted(const Wanted &w, int32_t *base, int32_t *totals, int *s_wave)
{
    __shared__ int s_before[kThreads], s_column[kThreads], s_there[kThreads];
    int before = 0, past = 0, total;
    for (int i0 = 0; i0 < w.n; i0 += kThreads) {
        const int i = i0 + threadIdx.x;
        int wants = 0;
        if (w.new_lens) {
            int first = 0, beyond = 0, all;
            if (i < w.n) wants = w.columns(i, first, beyond);
            past += beyond;
            s_before[threadIdx.x] = block_exclusive(wants, all, s_wave);
            s_column[threadIdx.x] = first;
            s_there[threadIdx.x] = 0;
            __syncthreads();
            // a thread takes neighbouring columns, starting in the last clip with s_before <= at
            const int clips = min(kThreads, w.n - i0), each = (all + kThreads - 1) / kThreads;
            int at = min(static_cast<int>(threadIdx.x) * each, all), lo = 0, hi = clips;
            const int end = at + min(each, all - at);
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_before[mid] <= at) lo = mid;
                else hi = mid;
            }
#pragma unroll 4
            for (; at < end; ++at) {
                while (lo + 1 < clips && s_before[lo + 1] <= at) ++lo;
                if (w.is_page(w.table[static_cast<int64_t>(i0 + lo) * w.table_ld + s_column[lo] + at - s_before[lo]]))
                    atomicAdd(&s_there[lo], 1);
            }
            __syncthreads();
            wants -= s_there[threadIdx.x];
        } else if (i < w.n) {
            int full;
            wants = w.partial(i, full) >= 0;
        }
        const int rank = block_exclusive(wants, total, s_wave);
        if (i < w.n) base[i] = before + rank;
        before += total;
    }
    block_exclusive(past, total, s_wave);
    if (threadIdx.x == 0) {
        base[w.n] = before;
        totals[kInTable] = before;
        totals[kBeyond] = total;
    }
}

__global__ __launch_bounds__(kThreads)
void rank_wanted_alone(Wanted w, int32_t *__restrict__ base, int32_t *__restrict__ totals)
{
    __shared__ int s_wave[kThreads / 64];
    rank_wanted(w, base, totals, s_wave);
}

// First launch of reserve and fork. Workgroups 0 .. n_chunks - 1: free pages in order -> list, and refs_out = refs (the
// second launch enters the pages that it takes). The next one ranks what is wanted, unless that has been done (counted).
// Those that are left copy the pairs of arrays for fork.
struct IntCopy {
    const int32_t *from;
    int32_t *to;
    int64_t n;
};

__global__ __launch_bounds__(kThreads)
void take_free(const int32_t *__restrict__ refs, int n_pages, int n_chunks, const int32_t *__restrict__ counts,
               Wanted w, int32_t *__restrict__ base, int32_t *__restrict__ totals, int32_t *__restrict__ list,
               int32_t *__restrict__ refs_out, IntCopy one, IntCopy two)
{
    __shared__ int s_wave[kThreads / 64];
    const int chunk = blockIdx.x;
    if (chunk > n_chunks) {
        int64_t i = (chunk - n_chunks - 1) * static_cast<int64_t>(kThreads) + threadIdx.x;
        if (i < one.n) one.to[i] = one.from[i];
        else if ((i -= one.n) < two.n) two.to[i] = two.from[i];
        return;
    }
    if (chunk == n_chunks) {
        if (!counts) rank_wanted(w, base, totals, s_wave);
        if (n_chunks == 0 && threadIdx.x == 0) totals[kFree] = 0;
        return;
    }
    const int64_t first = static_cast<int64_t>(chunk) * kChunk + threadIdx.x * kPerThread;
    int ref[kPerThread];
    int used = used_before(refs, n_pages, counts, chunk, first, ref, s_wave);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int64_t p = first + i;
        if (p >= n_pages) break;
        if (ref[i] <= 0) list[p - used] = static_cast<int32_t>(p);
        refs_out[p] = ref[i];
        used += ref[i] > 0;
    }
    if (chunk == n_chunks - 1 && threadIdx.x == kThreads - 1) totals[kFree] = n_pages - used;
}

__device__ inline void write_missing(const int32_t *totals, int32_t *missing)
{
    *missing = max(0, totals[kInTable] - totals[kFree]) + totals[kBeyond];
}

// reserve, second launch: table_out = table with the wanted entries filled from the list of free pages as far as it goes;
// one thread an entry.
__global__ __launch_bounds__(kThreads)
void fill_table(Wanted w, const int32_t *__restrict__ totals, const int32_t *__restrict__ base,
                const int32_t *__restrict__ list, int32_t *__restrict__ table_out, int32_t *__restrict__ refs_out,
                int32_t *__restrict__ missing)
{
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (at == 0) write_missing(totals, missing);
    if (at >= static_cast<int64_t>(w.n) * w.table_ld) return;
    const int b = static_cast<int>(at / w.table_ld), e = static_cast<int>(at - static_cast<int64_t>(b) * w.table_ld);
    int first, past, page = w.table[at];
    const int count = w.columns(b, first, past);
    if (e >= first && e < first + count && !w.is_page(page)) {
        int rank = base[b] + e - first;
        if (base[b + 1] - base[b] < count)      // less those before it that are there
            for (int64_t i = at - (e - first); i < at; ++i) rank -= w.is_page(w.table[i]);
        if (rank < totals[kFree]) {
            page = list[rank];
            refs_out[page] = 1;
        }
    }
    table_out[at] = page;
}

// Copies one page of one layer of one pool; the whole workgroup.
__device__ inline void copy_page(char *pool, int source, int target, int64_t page_bytes)
{
    const u32x4 *from = reinterpret_cast<const u32x4 *>(pool + source * page_bytes);
    u32x4 *to = reinterpret_cast<u32x4 *>(pool + target * page_bytes);
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < page_bytes / 16; i += kThreads) to[i] = from[i];
}

struct Pools {
    char *k, *v;
    int n_pages, n_layers;
    int64_t page_bytes;

    // job = (pair * n_layers + layer) * 2 + pool
    __device__ void copy(int64_t job, int64_t pair, int source, int target) const
    {
        if (static_cast<unsigned>(source) >= static_cast<unsigned>(n_pages) ||
            static_cast<unsigned>(target) >= static_cast<unsigned>(n_pages))
            return;
        const int rest = static_cast<int>(job - pair * 2 * n_layers), layer = rest >> 1;
        copy_page(((rest & 1) ? v : k) + static_cast<int64_t>(layer) * n_pages * page_bytes, source, target, page_bytes);
    }
};

// fork, second launch: a workgroup a child rewrites its row and counts references; those that are left copy the
// partial pages, whole (page, layer, pool) jobs in turn.
__global__ __launch_bounds__(kThreads)
void fork_rows(Wanted w, const int32_t *__restrict__ table, const int32_t *__restrict__ totals,
               const int32_t *__restrict__ base, const int32_t *__restrict__ list, int32_t *__restrict__ table_out,
               int32_t *__restrict__ lens_out, int32_t *__restrict__ refs_out, int32_t *__restrict__ missing, Pools pools)
{
    const int n_free = totals[kFree];
    // the child's page for the parent's partial one, -1 for none
    auto copy_of = [&](int c, int source) { return source >= 0 && base[c] < n_free ? list[base[c]] : -1; };
    if (blockIdx.x >= static_cast<unsigned>(w.n)) {
        const int64_t jobs = static_cast<int64_t>(w.n) * pools.n_layers * 2, step = gridDim.x - w.n;
        for (int64_t job = blockIdx.x - w.n; job < jobs; job += step) {
            const int64_t pair = job / (2 * pools.n_layers);
            int full;
            const int source = w.partial(static_cast<int>(pair), full), target = copy_of(static_cast<int>(pair), source);
            if (target >= 0) pools.copy(job, pair, source, target);
        }
        return;
    }
    const int c = blockIdx.x, parent = w.parents[c], child = w.children[c];
    if (c == 0 && threadIdx.x == 0) write_missing(totals, missing);
    if (static_cast<unsigned>(parent) >= static_cast<unsigned>(w.n_clips) ||
        static_cast<unsigned>(child) >= static_cast<unsigned>(w.n_clips))
        return;
    int full;
    const int fresh = copy_of(c, w.partial(c, full));
    const int32_t *from = table + static_cast<int64_t>(parent) * w.table_ld;
    const int32_t *was = table + static_cast<int64_t>(child) * w.table_ld;
    int32_t *to = table_out + static_cast<int64_t>(child) * w.table_ld;
    for (int e = threadIdx.x; e < w.table_ld; e += kThreads) {
        const int left = was[e];
        int page = from[e];
        if (static_cast<unsigned>(left) < static_cast<unsigned>(pools.n_pages)) atomicSub(&refs_out[left], 1);
        if (e >= full) {       // behind the full pages: the copy, and nothing that the parent has reserved ahead
            page = e == full ? fresh : -1;
            if (page >= 0) refs_out[page] = 1;
        } else if (static_cast<unsigned>(page) < static_cast<unsigned>(pools.n_pages)) {
            atomicAdd(&refs_out[page], 1);
        }
        to[e] = page;
    }
    if (threadIdx.x == 0) lens_out[child] = w.lens[parent];
}

// copy: page sources[i] to targets[i].
__global__ __launch_bounds__(kThreads)
void copy_pages(const int32_t *__restrict__ sources, const int32_t *__restrict__ targets, int n, Pools pools)
{
    const int64_t jobs = static_cast<int64_t>(n) * pools.n_layers * 2;
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const int64_t pair = job / (2 * pools.n_layers);
        pools.copy(job, pair, sources[pair], targets[pair]);
    }
}

__global__ __launch_bounds__(kThreads)
void copy_ints(const int32_t *__restrict__ from, int32_t *__restrict__ to, int64_t n)
{
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (i < n) to[i] = from[i];
}

// Whether entry e of clip b leaves the table in a free.
struct Leaves {
    const int32_t *lens, *drop;
    int page_size, sinks;
    int64_t window;

    __device__ bool operator()(int b, int e) const
    {
        if (drop && drop[b]) return true;
        // the next frame stands at position lens[b] and sees the positions above lens[b] - window
        const int64_t low = static_cast<int64_t>(e) * page_size;
        return window >= 0 && low >= sinks && low + page_size <= static_cast<int64_t>(lens[b]) - window + 1;
    }
};

// free in one launch, for tables that are soon read: workgroups 0 .. n_chunks - 1 go over the whole table and count in
// the LDS what leaves of their chunk's pages, those that are left write the table and the lengths.
__global__ __launch_bounds__(kThreads)
void free_small(const int32_t *__restrict__ table, const int32_t *__restrict__ refs, int n_clips, int table_ld,
                int n_pages, int n_chunks, Leaves leaves, int32_t *__restrict__ table_out,
                int32_t *__restrict__ lens_out, int32_t *__restrict__ refs_out)
{
    __shared__ int s_gone[kChunk];
    const int entries = n_clips * table_ld;
    if (static_cast<int>(blockIdx.x) >= n_chunks) {
        const int at = (static_cast<int>(blockIdx.x) - n_chunks) * kThreads + threadIdx.x;
        if (at < n_clips) lens_out[at] = leaves.drop && leaves.drop[at] ? 0 : leaves.lens[at];
        if (at >= entries) return;
        const int b = at / table_ld;
        table_out[at] = leaves(b, at - b * table_ld) ? -1 : table[at];
        return;
    }
    const int first = blockIdx.x * kChunk;
    for (int i = threadIdx.x; i < kChunk; i += kThreads) s_gone[i] = 0;
    __syncthreads();
#pragma unroll 4
    for (int at = threadIdx.x; at < entries; at += kThreads) {
        const uint32_t page = static_cast<uint32_t>(table[at]) - static_cast<uint32_t>(first);
        if (page < static_cast<uint32_t>(kChunk)) {
            const int b = at / table_ld;
            if (leaves(b, at - b * table_ld)) atomicAdd(&s_gone[page], 1);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kChunk && first + i < n_pages; i += kThreads) refs_out[first + i] = refs[first + i] - s_gone[i];
}

// free: what leaves the table, reference counts go down.
__global__ __launch_bounds__(kThreads)
void free_entries(const int32_t *__restrict__ table, int n_clips, int table_ld, int n_pages, Leaves leaves,
                  int32_t *__restrict__ table_out, int32_t *__restrict__ lens_out, int32_t *__restrict__ refs_out)
{
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (at < n_clips) lens_out[at] = leaves.drop && leaves.drop[at] ? 0 : leaves.lens[at];
    if (at >= static_cast<int64_t>(n_clips) * table_ld) return;
    const int b = static_cast<int>(at / table_ld), e = static_cast<int>(at - static_cast<int64_t>(b) * table_ld);
    int page = table[at];
    if (leaves(b, e)) {
        if (static_cast<unsigned>(page) < static_cast<unsigned>(n_pages)) atomicSub(&refs_out[page], 1);
        page = -1;
    }
    table_out[at] = page;
}

// compact, first launch: pages in use numbered live and more are sources, free pages below live are targets, both in
// order.
__global__ __launch_bounds__(kThreads)
void list_moves(const int32_t *__restrict__ refs, int n_pages, const int32_t *__restrict__ counts,
                int32_t *__restrict__ totals, int32_t *__restrict__ sources, int32_t *__restrict__ targets,
                int32_t *__restrict__ rank, int32_t *__restrict__ live_out)
{
    __shared__ int s_wave[kThreads / 64];
    const int live = used_below(refs, counts, n_pages, s_wave);
    const int below = used_below(refs, counts, live, s_wave);
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kChunk + threadIdx.x * kPerThread;
    int ref[kPerThread];
    int used = used_before(refs, n_pages, counts, blockIdx.x, first, ref, s_wave);
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
        totals[kLive] = live;
        totals[kMoves] = live - below;
    }
}

// compact, second launch: workgroups 0 .. n_renumber - 1 put new numbers into the table and reference counts at the
// new numbers, those that are left move the pages.
__global__ __launch_bounds__(kThreads)
void move_pages(int n_renumber, const int32_t *__restrict__ table, int64_t entries, const int32_t *__restrict__ refs,
                const int32_t *__restrict__ totals, const int32_t *__restrict__ sources,
                const int32_t *__restrict__ targets, const int32_t *__restrict__ rank, int32_t *__restrict__ table_out,
                int32_t *__restrict__ refs_out, Pools pools)
{
    const int live = totals[kLive], moves = totals[kMoves];
    if (blockIdx.x >= static_cast<unsigned>(n_renumber)) {
        const int64_t jobs = static_cast<int64_t>(moves) * pools.n_layers * 2, step = gridDim.x - n_renumber;
        for (int64_t job = blockIdx.x - n_renumber; job < jobs; job += step) {
            const int64_t pair = job / (2 * pools.n_layers);
            pools.copy(job, pair, sources[pair], targets[pair]);
        }
        return;
    }
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (at < entries) {
        int page = table[at];
        if (page >= live && page < pools.n_pages) page = refs[page] > 0 ? targets[rank[page]] : -1;
        table_out[at] = page;
    }
    if (at < pools.n_pages) {
        const int ref = refs[at];
        if (at >= live) refs_out[at] = 0;
        else if (ref > 0) refs_out[at] = ref;
    }
    if (at < moves) refs_out[targets[at]] = refs[sources[at]];
}

// append: a workgroup takes kAppendTokens new frames, finds their places, then moves their rows, a thread 16 bytes of
// a key row and of the value row beside it.
constexpr int kAppendTokens = 8;

__global__ __launch_bounds__(kThreads)
void append_rows(Heads k, Heads v, int64_t n_tokens, const int32_t *__restrict__ cu, int n_clips, int kv_heads,
                 int pieces, int element_bytes, int page_size, int n_pages, int table_ld,
                 const int32_t *__restrict__ table, const int32_t *__restrict__ lens, char *__restrict__ k_pool,
                 char *__restrict__ v_pool)
{
    __shared__ int64_t s_row[kAppendTokens];       // the frame's row at head 0 in the pools, -1 for none
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kAppendTokens;
    if (threadIdx.x < kAppendTokens) {
        const int64_t token = first + threadIdx.x;
        int64_t row = -1;
        int clip = static_cast<int>(token), nth = 0;
        bool there = token < n_tokens;
        if (there && cu) {
            clip = clip_of_row(cu, n_clips, static_cast<int>(token));
            nth = static_cast<int>(token) - cu[clip];
            there = nth >= 0 && token < cu[clip + 1];      // not outside every clip
        }
        if (there) {
            const int64_t position = static_cast<int64_t>(lens[clip]) + nth;
            if (position >= 0 && position < static_cast<int64_t>(table_ld) * page_size) {
                const int e = static_cast<int>(position) / page_size, slot = static_cast<int>(position) - e * page_size;
                const int page = table[static_cast<int64_t>(clip) * table_ld + e];
                if (static_cast<unsigned>(page) < static_cast<unsigned>(n_pages))
                    row = static_cast<int64_t>(page) * kv_heads * page_size + slot;
            }
        }
        s_row[threadIdx.x] = row;
    }
    __syncthreads();
    const int per_token = kv_heads * pieces;
#pragma unroll 4
    for (int at = threadIdx.x; at < kAppendTokens * per_token; at += kThreads) {
        const int n = at / per_token, rest = at - n * per_token, head = rest / pieces, piece = rest - head * pieces;
        const int64_t row = s_row[n], token = first + n;
        if (row < 0) continue;
        const int64_t to = ((row + static_cast<int64_t>(head) * page_size) * pieces + piece) * 16;
        const char *from_k = static_cast<const char *>(k.data) + (token * k.token + head * k.head) * element_bytes;
        const char *from_v = static_cast<const char *>(v.data) + (token * v.token + head * v.head) * element_bytes;
        *reinterpret_cast<u32x4 *>(k_pool + to) = *reinterpret_cast<const u32x4 *>(from_k + piece * 16);
        *reinterpret_cast<u32x4 *>(v_pool + to) = *reinterpret_cast<const u32x4 *>(from_v + piece * 16);
    }
}

unsigned copy_blocks(int64_t jobs) { return static_cast<unsigned>(jobs < kCopyBlocks ? jobs : kCopyBlocks); }

// First launch of reserve and fork (and before it, in large pools or with many clips, the counting ones).
void launch_take_free(const int32_t *refs, int n_pages, const Wanted &w, const Scratch &s, int32_t *list,
                      int32_t *refs_out, const IntCopy &one, const IntCopy &two, hipStream_t stream)
{
    const int n_chunks = static_cast<int>(chunks(n_pages));
    const bool counted = n_pages > kSelfCounted || w.n > kSelfCounted / 16;
    if (counted) {
        if (n_chunks) count_used<<<n_chunks, kThreads, 0, stream>>>(refs, n_pages, s.counts);
        rank_wanted_alone<<<1, kThreads, 0, stream>>>(w, s.base, s.totals);
    }
    take_free<<<n_chunks + 1 + ceil_div(one.n + two.n, kThreads), kThreads, 0, stream>>>(
        refs, n_pages, n_chunks, counted ? s.counts : nullptr, w, s.base, s.totals, list, refs_out, one, two);
}

}  // namespace

int64_t cache_scratch_bytes(int n_clips, int n_pages) { return scratch_ints(n_clips, n_pages) * 4; }

hipError_t launch_cache_append(const Heads &k, const Heads &v, int64_t n_tokens, const int32_t *cu, int n_clips,
                               int kv_heads, int dim, int element_bytes, int page_size, int n_pages, int table_ld,
                               const int32_t *table, const int32_t *lens, void *k_pool, void *v_pool,
                               hipStream_t stream)
{
    const int pieces = dim * element_bytes / 16;
    if (!fits(ceil_div(n_tokens, kAppendTokens), kThreads)) return hipErrorNotSupported;
    append_rows<<<ceil_div(n_tokens, kAppendTokens), kThreads, 0, stream>>>(
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
    const Wanted w = {table, lens, new_lens, nullptr, nullptr, n_clips, n_clips, table_ld, page_size, n_pages};
    launch_take_free(refs, n_pages, w, s, s.sources, refs_out, IntCopy{}, IntCopy{}, stream);
    const int64_t entries = static_cast<int64_t>(n_clips) * table_ld;
    fill_table<<<entries ? ceil_div(entries, kThreads) : 1, kThreads, 0, stream>>>(w, s.totals, s.base, s.sources,
                                                                                   table_out, refs_out, missing);
    return hipGetLastError();
}

hipError_t launch_cache_fork(const int32_t *table, const int32_t *lens, const int32_t *refs, const int32_t *parents,
                             const int32_t *children, int n_children, int n_clips, int table_ld, int page_size,
                             int n_pages, int n_layers, int64_t page_bytes, void *k_pool, void *v_pool,
                             int32_t *table_out, int32_t *lens_out, int32_t *refs_out, int32_t *missing,
                             void *workspace, hipStream_t stream)
{
    const Scratch s = scratch(workspace, n_clips, n_pages);
    // new_lens null makes it a fork; a fork of no children still copies the arrays and reports nothing missing
    const Wanted w = {table, lens, nullptr, parents, children, n_children, n_clips, table_ld, page_size, n_pages};
    const Pools pools = {static_cast<char *>(k_pool), static_cast<char *>(v_pool), n_pages, n_layers, page_bytes};
    launch_take_free(refs, n_pages, w, s, s.sources, refs_out,
                     IntCopy{table, table_out, static_cast<int64_t>(n_clips) * table_ld}, IntCopy{lens, lens_out, n_clips},
                     stream);
    if (n_children == 0) {
        fill_table<<<1, kThreads, 0, stream>>>(w, s.totals, s.base, s.sources, table_out, refs_out, missing);
        return hipGetLastError();
    }
    const int64_t jobs = static_cast<int64_t>(n_children) * n_layers * 2;
    fork_rows<<<n_children + copy_blocks(jobs), kThreads, 0, stream>>>(w, table, s.totals, s.base, s.sources, table_out,
                                                                       lens_out, refs_out, missing, pools);
    return hipGetLastError();
}

hipError_t launch_cache_free(const int32_t *table, const int32_t *lens, const int32_t *refs, const int32_t *drop,
                             int n_clips, int table_ld, int page_size, int n_pages, int64_t window, int sinks,
                             int32_t *table_out, int32_t *lens_out, int32_t *refs_out, hipStream_t stream)
{
    const Leaves leaves = {lens, drop, page_size, sinks, window};
    const int64_t entries = static_cast<int64_t>(n_clips) * table_ld, items = entries > n_clips ? entries : n_clips;
    const int64_t n_chunks = chunks(n_pages);
    if (entries <= kSoonRead && n_pages <= kSelfCounted) {
        const int64_t groups = n_chunks + ceil_div(items, kThreads);
        if (groups)
            free_small<<<static_cast<unsigned>(groups), kThreads, 0, stream>>>(table, refs, n_clips, table_ld, n_pages,
                                                                               static_cast<int>(n_chunks), leaves,
                                                                               table_out, lens_out, refs_out);
        return hipGetLastError();
    }
    if (n_pages > 0) copy_ints<<<ceil_div(n_pages, kThreads), kThreads, 0, stream>>>(refs, refs_out, n_pages);
    if (items > 0)
        free_entries<<<ceil_div(items, kThreads), kThreads, 0, stream>>>(table, n_clips, table_ld, n_pages, leaves,
                                                                         table_out, lens_out, refs_out);
    return hipGetLastError();
}

hipError_t launch_cache_compact(const int32_t *table, const int32_t *refs, int n_clips, int table_ld, int n_pages,
                                int n_layers, int64_t page_bytes, void *k_pool, void *v_pool, int32_t *table_out,
                                int32_t *refs_out, int32_t *live, void *workspace, hipStream_t stream)
{
    const Scratch s = scratch(workspace, n_clips, n_pages);
    const Pools pools = {static_cast<char *>(k_pool), static_cast<char *>(v_pool), n_pages, n_layers, page_bytes};
    const int n_chunks = static_cast<int>(chunks(n_pages));
    const bool counted = n_pages > kSelfCounted;
    if (counted) count_used<<<n_chunks, kThreads, 0, stream>>>(refs, n_pages, s.counts);
    list_moves<<<n_chunks ? n_chunks : 1, kThreads, 0, stream>>>(refs, n_pages, counted ? s.counts : nullptr, s.totals,
                                                                 s.sources, s.targets, s.rank, live);
    const int64_t entries = static_cast<int64_t>(n_clips) * table_ld, most = entries > n_pages ? entries : n_pages;
    const unsigned renumber = ceil_div(most, kThreads);
    const unsigned movers = copy_blocks(static_cast<int64_t>(n_pages / 2) * n_layers * 2);
    if (renumber + movers)
        move_pages<<<renumber + movers, kThreads, 0, stream>>>(static_cast<int>(renumber), table, entries, refs, s.totals,
                                                               s.sources, s.targets, s.rank, table_out, refs_out, pools);
    return hipGetLastError();
}

hipError_t launch_cache_copy(const int32_t *src, const int32_t *dst, int n_copies, int n_pages, int n_layers,
                             int64_t page_bytes, void *k_pool, void *v_pool, hipStream_t stream)
{
    const Pools pools = {static_cast<char *>(k_pool), static_cast<char *>(v_pool), n_pages, n_layers, page_bytes};
    copy_pages<<<copy_blocks(static_cast<int64_t>(n_copies) * n_layers * 2), kThreads, 0, stream>>>(src, dst, n_copies, pools);
    return hipGetLastError();
}

}  // namespace rvq
