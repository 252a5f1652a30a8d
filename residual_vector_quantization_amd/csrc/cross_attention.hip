// Cross attention: packed queries that all see all of their clip's keys, which
// are packed too, of another length. rows_attention.h over packed keys.
#include "rows_attention.h"

namespace rvq {
namespace {

// Keys of a clip as the launch is laid out for: twice the average, no more than there are. Clips with more are split
// as far as others, so it changes only how evenly the work is shared out.
int64_t some_keys(const RowsArgs &a)
{
    const int64_t twice = a.n_clips ? 2 * a.k_tokens / a.n_clips : 0;
    return twice < a.k_tokens ? twice : a.k_tokens;
}

}  // namespace

int64_t cross_attention_bytes(const RowsArgs &a)
{
    int64_t floats;
    rows::plan(a, some_keys(a), floats);
    return floats * 4;
}

hipError_t launch_cross_attention(const RowsArgs &a, hipStream_t stream)
{
    int64_t floats;
    rows::Plan p = rows::plan(a, some_keys(a), floats);
    p.by_chiplet = true;
    return rows::launch<rows::Packed>(a, p, stream);
}

}  // namespace rvq
