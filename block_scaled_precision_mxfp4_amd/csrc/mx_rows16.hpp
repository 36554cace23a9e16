// Cross-lane exchanges by row permutes, without LDS (gfx950).
#pragma once

#include "mx_device.hpp"

namespace mx {

// A butterfly's partner inside 16 lanes by row permutes (no LDS): steps 0..3
// are lane ^ 1, lane ^ 2, the mirrored lane of 8 and of 16 (whose quads and
// halves already agree).
__device__ __forceinline__ uint32_t row_partner(uint32_t v, int step)
{
    switch (step) {
    case 0: return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);
    case 1: return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);
    case 2: return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true);
    default: return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true);
    }
}

// Inclusive sum over the lanes of a wave: inside each row of 16 lanes by
// shifts (a lane without a source adds 0), then the last lane of rows 0 and 2 to
// the row behind it, and lane 31 to the upper half.
__device__ __forceinline__ int wave_scan(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
    return v;
}

}  // namespace mx
