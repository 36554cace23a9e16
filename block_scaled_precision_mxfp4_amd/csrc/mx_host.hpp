// What the host sources of the library share.
#pragma once

#include "libmxgemm.h"

namespace mx {

// MXGEMM_OK on a gfx950 device (the current one); its compute units in *num_cu.
mxgemm_status check_device(int *num_cu = nullptr);

}  // namespace mx
