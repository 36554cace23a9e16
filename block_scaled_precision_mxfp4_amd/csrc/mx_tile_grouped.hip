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
    if (g.scale16)
        hipLaunchKernelGGL((mx_tile_kernel<BM, BN, WM, WN, 0, true, false, AFMT, true, false, true>), dim3((unsigned)grid),
                           dim3(64 * WM * WN), 0, s, g);
    else
        hipLaunchKernelGGL((mx_tile_kernel<BM, BN, WM, WN, 0, false, false, AFMT, true, false, true>),
                           dim3((unsigned)grid), dim3(64 * WM * WN), 0, s, g);
}

// The tiles, largest first, with the mean rows per expert from which each was
// the fastest (MI355X, 32 experts, N = 4096, K = 2048, routings as uneven as a
// softmax of normal logits; us, FP4 / FP8 A):
//   rows per expert   4            16           64           256          1024
//   32 x 128          - / 17.1     31.2 / 32.8  52.1 / 54.5  130 / 138    413 / -
//   64 x 128          - / 21.0     31.3 / 31.0  42.6 / 50.5  92.6 / 121   288 / -
//   128 x 128         - / 32.0     32.3 / 48.8  43.8 / 65.6  83.5 / 139   245 / -
//   128 x 256         - / 27.1     - / 37.2     - / 50.8     - / 97.8     - / 289
//   256 x 256         -            43.3 / -     57.0 / -     88.3 / -     207 / -
const GroupedTileKernel *grouped_tile_kernels(int *count)
{
    static const GroupedTileKernel table[] = {
        {256, 256, {384, 0}, {launch_tile_grouped<256, 256, 2, 4, 0>, nullptr}, {nullptr, nullptr}},
        {128, 256, {0, 96}, {nullptr, launch_tile_grouped<128, 256, 2, 4, 1>},
         {nullptr, launch_tile_grouped_persist<128, 256, 2, 4, 1>}},
        {128, 128, {96, 0}, {launch_tile_grouped<128, 128, 2, 2, 0>, nullptr}, {nullptr, nullptr}},
        {64, 128, {16, 12}, {launch_tile_grouped<64, 128, 2, 2, 0>, launch_tile_grouped<64, 128, 2, 2, 1>}, {nullptr, nullptr}},
        {32, 128, {0, 0}, {launch_tile_grouped<32, 128, 1, 4, 0>, launch_tile_grouped<32, 128, 1, 4, 1>}, {nullptr, nullptr}},
    };
    *count = (int)(sizeof(table) / sizeof(table[0]));
    return table;
}

}  // namespace mx
