// Attention of many rows per key head: heads of up to 128 columns.
#include "mx_attn_rows.hpp"

namespace mx {

int attn_rows_tile(int D) { return D > 128 ? RowsShape<256>::TM : RowsShape<128>::TM; }
int attn_rows_per_cu(int) { return 1; }

void launch_attn_rows(const AttnArgs &a, bool fp8, int plan, int grid, hipStream_t s)
{
    if (a.c.D <= 64)
        launch_rows<64>(a, fp8, plan, grid, s);
    else if (a.c.D <= 128)
        launch_rows<128>(a, fp8, plan, grid, s);
    else
        launch_attn_rows_wide(a, fp8, plan, grid, s);
}

}  // namespace mx
