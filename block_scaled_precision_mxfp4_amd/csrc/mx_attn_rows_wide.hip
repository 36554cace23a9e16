// Attention of many rows per key head: heads of up to 256 columns, whose
// accumulators and queries fill most of both register files.
#include "mx_attn_rows.hpp"

namespace mx {

AttnRowsKernel attn_rows_kernel_wide(bool fp8) { return rows_entry<256, false>(fp8); }

}  // namespace mx
