// Attention of many rows per key head: heads of up to 256 columns, whose
// accumulators and queries fill most of both register files.
#include "mx_attn_rows.hpp"

namespace mx {

void launch_attn_rows_wide(const AttnArgs &a, bool fp8, int plan, int grid, hipStream_t s)
{
    launch_rows<256>(a, fp8, plan, grid, s);
}

}  // namespace mx
