// Attention of many rows per key head: heads of up to 256 columns, whose
// accumulators and queries fill most of both register files (one workgroup of
// four waves on a compute unit).  Two prompts of 1000 tokens, 16 heads on 4: 57 us,
// 0.31 PFLOP/s; 100 tokens over 16384: 96 us, 0.28; a prompt of 4096 203 us, 0.68.
#include "mx_attn_rows.hpp"

namespace mx {

AttnRowsKernel attn_rows_kernel_wide(bool fp8) { return rows_entry<256, false>(fp8); }

}  // namespace mx
