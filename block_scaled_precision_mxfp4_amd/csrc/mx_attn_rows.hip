// Attention of many rows per key head: heads of up to 128 columns.
#include "mx_attn_rows.hpp"

namespace mx {

AttnRowsKernel attn_rows_kernel(int D, bool fp8, bool small)
{
    if (D <= 64)
        return rows_entry<64, true>(fp8);
    if (D <= 128)
        return small ? rows_entry<128, true>(fp8) : rows_entry<128, false>(fp8);
    return attn_rows_kernel_wide(fp8);
}

}  // namespace mx
