// Launchers of the tiled kernel (mx_tile.hpp) for the product grouped by
// expert.
#include "mx_tile.hpp"

namespace mx {

// Product grouped by expert: tile shapes by A's format.  The grid covers the
// most row tiles that the rows can make among the experts (every expert's
// last one partly filled); workgroups past the last tile leave at once.
template <int BM, int BN, int WM, int WN, int AFMT>
static void launch_tile_grouped(const GroupedTileArgs &g, int64_t grid, hipStream_t s)
{
    if (g.scale16)
        hipLaunchKernelGGL((mx_tile_kernel<BM, BN, WM, WN, 0, true, false, AFMT, false, false, true>), dim3((unsigned)grid),
                           dim3(64 * WM * WN), 0, s, g);
    else
        hipLaunchKernelGGL((mx_tile_kernel<BM, BN, WM, WN, 0, false, false, AFMT, false, false, true>),
                           dim3((unsigned)grid), dim3(64 * WM * WN), 0, s, g);
}

template <int BM, int BN, int WM, int WN, int AFMT>
static void launch_tile_grouped_persist(const GroupedTileArgs &g, int64_t grid, hipStream_t s)
{
    hipLaunchKernelGGL((mx_tile_kernel<BM, BN, WM, WN, 0, true, false, AFMT, true, false, true>), dim3((unsigned)grid),
                       dim3(64 * WM * WN), 0, s, g);
}

#define MX_TILE_GROUPED(BM, BN, WM, WN) \
    {BM, BN, {launch_tile_grouped<BM, BN, WM, WN, 0>, launch_tile_grouped<BM, BN, WM, WN, 1>}, {nullptr, nullptr}}

const GroupedTileKernel *grouped_tile_kernels(int *count)
{
    static const GroupedTileKernel table[] = {
        {256, 256, {launch_tile_grouped<256, 256, 2, 4, 0>, nullptr}, {launch_tile_grouped_persist<256, 256, 2, 4, 0>, nullptr}},
        {192, 256, {launch_tile_grouped<192, 256, 2, 4, 0>, nullptr}, {launch_tile_grouped_persist<192, 256, 2, 4, 0>, nullptr}},
        {128, 256, {launch_tile_grouped<128, 256, 2, 4, 0>, launch_tile_grouped<128, 256, 2, 4, 1>},
         {nullptr, launch_tile_grouped_persist<128, 256, 2, 4, 1>}},
        MX_TILE_GROUPED(128, 128, 2, 2),
        MX_TILE_GROUPED(64, 128, 2, 2),
        MX_TILE_GROUPED(32, 128, 1, 4),
    };
    *count = (int)(sizeof(table) / sizeof(table[0]));
    return table;
}
#undef MX_TILE_GROUPED

}  // namespace mx
