// Attention of a chunk of new frames of every clip over its paged key-value
// cache: rows_attention.h over the pages of a cache. One frame of some clips
// and many of others may be mixed in a call.
#include "rows_attention.h"

namespace rvq {
namespace {

// The most frames that a clip's queries can see together.
int64_t most_keys(const RowsArgs &a)
{
    const int64_t capacity = static_cast<int64_t>(a.table_ld) * a.page_size;
    const int64_t seen = static_cast<int64_t>(a.window) + a.sinks + rows::kTileQueries;
    return seen < capacity ? seen : capacity;
}

}  // namespace

int64_t chunk_attention_bytes(const RowsArgs &a)
{
    int64_t floats;
    rows::plan(a, most_keys(a), floats);
    return floats * 4;
}

hipError_t launch_chunk_attention(const RowsArgs &a, hipStream_t stream)
{
    int64_t floats;
    rows::Plan p = rows::plan(a, most_keys(a), floats);
    p.page = divisor(a.page_size);
    return rows::launch<rows::Paged>(a, p, stream);
}

}  // namespace rvq
