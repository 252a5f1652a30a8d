// The kernels' page arithmetic (cache_index.h) on the CPU, behind a C interface for the tests.
#include "cache_index.h"

extern "C" uint32_t index_divide(uint32_t n, int32_t d) { return rvq::divide(n, rvq::divisor(d)); }

extern "C" int index_seen(int len, int window, int sinks, int nth)
{
    const rvq::Seen s = rvq::seen_frames(len, window, sinks);
    return nth < 0 ? s.count : rvq::seen_position(s, nth);
}

extern "C" uint32_t index_row(const int32_t *row, int position, int page_size, int table_ld, int n_pages, int kv_heads,
                              int kv_head)
{
    return rvq::cache_row(row, position, rvq::divisor(page_size), table_ld, n_pages, kv_heads, kv_head);
}
