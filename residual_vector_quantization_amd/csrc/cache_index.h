// Where a clip's frames lie in a paged cache: plain index arithmetic, shared by
// the kernels and by host code.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#define RVQ_HOST_DEVICE __host__ __device__
#else
#define RVQ_HOST_DEVICE
#endif

namespace rvq {

// Division of 0 <= n < 2^31 by a fixed d >= 1: with s = ceil(log2 d) and m = ceil(2^(31+s) / d), m d exceeds
// 2^(31+s) by less than d <= 2^s, so n m / 2^(31+s) exceeds n / d by less than 2^-31 n < 1 of a d-th: the floors agree.
struct Divisor {
    uint32_t by, multiplier, shift;
};

inline Divisor divisor(int32_t d)
{
    uint32_t s = 0;
    while ((uint64_t(1) << s) < static_cast<uint64_t>(d)) ++s;
    const uint64_t m = ((uint64_t(1) << (31 + s)) + d - 1) / d;
    return Divisor{static_cast<uint32_t>(d), static_cast<uint32_t>(m), 31 + s};
}

RVQ_HOST_DEVICE inline uint32_t divide(uint32_t n, const Divisor &d)
{
    return static_cast<uint32_t>((static_cast<uint64_t>(n) * d.multiplier) >> d.shift);
}

// The frames that the newest one of `len` sees, counted from 0: `first` sinks, then the window from `low` on.
struct Seen {
    int first, low, count;
};

RVQ_HOST_DEVICE inline Seen seen_frames(int len, int window, int sinks)
{
    Seen s;
    len = len > 0 ? len : 0;
    s.low = len > window ? len - window : 0;
    s.first = sinks < s.low ? sinks : s.low;
    s.count = s.first + (len - s.low);
    return s;
}

RVQ_HOST_DEVICE inline int seen_position(const Seen &s, int nth) { return nth < s.first ? nth : nth - s.first + s.low; }

// Whether a query at a position sees frame j.
RVQ_HOST_DEVICE inline bool sees_frame(int position, int j, int window, int sinks)
{
    return j <= position && (position - j < window || j < sinks);
}

// The frames that some query between positions p_first and p_last sees: sinks, then the window.
RVQ_HOST_DEVICE inline Seen seen_between(int p_first, int p_last, int window, int sinks)
{
    Seen s = {0, 0, 0};
    if (p_last < 0) return s;
    const int64_t low = static_cast<int64_t>(p_first) - window + 1;
    s.low = low > 0 ? static_cast<int>(low) : 0;
    const int before = sinks < s.low ? sinks : s.low;
    s.first = before < p_last + 1 ? before : p_last + 1;
    s.count = s.first + (p_last + 1 > s.low ? p_last + 1 - s.low : 0);
    return s;
}

// How the frames that queries p_first .. p_last see are shared out among `splits` workgroups, in tiles of kSharedTile: split
// n has the tiles n per .. (n + 1) per - 1. A workgroup that goes over its part again for one of the queries alone
// leaves out what that one does not see, but keeps its part: others may not go over theirs again, and the splits of a
// row have to hold every frame once.
constexpr int kSharedTile = 32;

struct Shared {
    Seen seen;
    int tiles, per;
};

RVQ_HOST_DEVICE inline Shared share(int p_first, int p_last, int window, int sinks, int splits)
{
    Shared s;
    s.seen = seen_between(p_first, p_last, window, sinks);
    s.tiles = (s.seen.count + kSharedTile - 1) / kSharedTile;
    s.per = (s.tiles + splits - 1) / splits;
    return s;
}

// Frame nth of them, or -1: there is none, or only the query at `position` counts (alone) and does not see it.
RVQ_HOST_DEVICE inline int shared_frame(const Shared &s, int nth, bool alone, int position, int window, int sinks)
{
    if (nth >= s.seen.count) return -1;
    const int j = seen_position(s.seen, nth);
    return alone && !sees_frame(position, j, window, sinks) ? -1 : j;
}

// Row (of head dim values) of a position's frame in a pool, or kNoPage where the table holds no page for it.
// `row` is the clip's row of the table. Pools have fewer than 2^32 - 2 rows.
constexpr uint32_t kNoPage = 0xffffffffu;
constexpr uint32_t kPastEnd = 0xfffffffeu;   // for callers: a frame that is not there
constexpr int64_t kMaxRows = 0xfffffffe;

RVQ_HOST_DEVICE inline uint32_t cache_row(const int32_t *row, int position, const Divisor &page_size, int table_ld,
                                         int n_pages, int kv_heads, int kv_head)
{
    const uint32_t e = divide(static_cast<uint32_t>(position), page_size);
    if (e >= static_cast<uint32_t>(table_ld)) return kNoPage;
    const uint32_t page = static_cast<uint32_t>(row[e]);
    if (page >= static_cast<uint32_t>(n_pages)) return kNoPage;
    return (page * static_cast<uint32_t>(kv_heads) + static_cast<uint32_t>(kv_head)) * page_size.by +
           (static_cast<uint32_t>(position) - e * page_size.by);
}

}  // namespace rvq
