// How a turn's frames are shared out among workgroups (cache_index.h) on the CPU, behind a C interface for the tests.
#include "cache_index.h"

// Adds 1 to counts[j] for every frame j that split `split` counts for the query at `position`, one of those at p_first ..
// p_last: in a pass over all of them, where each row leaves out what it does not see, or in one for that query alone.
extern "C" void shared_count(int p_first, int p_last, int window, int sinks, int splits, int split, int position, int alone,
                             int32_t *counts)
{
    const rvq::Shared s = rvq::share(p_first, p_last, window, sinks, splits);
    const int last = (split + 1) * s.per < s.tiles ? (split + 1) * s.per : s.tiles;
    for (int nth = split * s.per * rvq::kSharedTile; nth < last * rvq::kSharedTile; ++nth) {
        const int j = rvq::shared_frame(s, nth, alone != 0, position, window, sinks);
        if (j >= 0 && rvq::sees_frame(position, j, window, sinks)) ++counts[j];
    }
}

// Frames gone over by the splits together.
extern "C" int shared_frames(int p_first, int p_last, int window, int sinks) { return rvq::seen_between(p_first, p_last, window, sinks).count; }
