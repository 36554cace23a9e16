// Launchers of the tiled kernel (mx_tile.hpp) for the dense products.
#include "mx_tile.hpp"

namespace mx {

// D = bf16(beta * C), or +0 when beta == 0: the starting value the
// bf16-atomic split-K reduction adds its chunks onto.  One thread per pair
// of columns (ldd and N are even there).
__global__ void __launch_bounds__(256) mx_d_init_kernel(GemmArgs g)
{
    const int64_t pairs = (int64_t)g.M * (g.N / 2);
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= pairs)
        return;
    const int m = (int)(i / (g.N / 2)), n = (int)(i - (int64_t)m * (g.N / 2)) * 2;
    float v0 = 0.0f, v1 = 0.0f;
    if (g.beta != 0.0f) {
        if (g.c_f32) {
            const float *c = reinterpret_cast<const float *>(g.C) + (int64_t)m * g.ldc + n;
            v0 = g.beta * c[0];
            v1 = g.beta * c[1];
        } else {
            const uint16_t *c = reinterpret_cast<const uint16_t *>(g.C) + (int64_t)m * g.ldc + n;
            v0 = g.beta * bf16_to_f32(c[0]);
            v1 = g.beta * bf16_to_f32(c[1]);
        }
    }
    *reinterpret_cast<uint32_t *>(g.D + (int64_t)m * g.ldd + n) = bf16x2_rne(v0, v1);
}

void launch_d_init(const GemmArgs &g, hipStream_t s)
{
    const int64_t pairs = (int64_t)g.M * (g.N / 2);
    hipLaunchKernelGGL(mx_d_init_kernel, dim3((unsigned)((pairs + 255) / 256)), dim3(256), 0, s, g);
}

template <int BM, int BN, int WM, int WN, int BLAY, bool SAPACK>
static void launch_tile(const GemmArgs &g, int grid, hipStream_t s)
{
    constexpr bool SBPACK = BLAY == 1 || BLAY == 3;
    // SVEC: whole 8-block stages and 8-byte scale-row loads (packed scales
    // need only the former)
    const bool sa_ok = SAPACK ? g.KB % 8 == 0 : g.sa_fast != 0;
    const bool sb_ok = SBPACK ? g.KB % 8 == 0 : g.sb_fast != 0;
    // persistent form: 256 x 256 with packed A and B scales, B's codes
    // packed or MN-major (its other layouts spill in the tile loop; the
    // 256 x 128 tile and the 8-bit 128 x 256 tile measured no faster
    // persistent)
    if constexpr (BM == 256 && BN == 256 && (BLAY == 1 || BLAY == 3) && SAPACK) {
        if (g.persist_grid > 0 && sa_ok && sb_ok) {
            hipLaunchKernelGGL((mx_tile_kernel<BM, BN, WM, WN, BLAY, true, SAPACK, 0, true>), dim3(g.persist_grid),
                               dim3(64 * WM * WN), 0, s, g);
            return;
        }
    }
    if (sa_ok && sb_ok)
        hipLaunchKernelGGL((mx_tile_kernel<BM, BN, WM, WN, BLAY, true, SAPACK>), dim3(grid), dim3(64 * WM * WN), 0, s, g);
    else
        hipLaunchKernelGGL((mx_tile_kernel<BM, BN, WM, WN, BLAY, false, SAPACK>), dim3(grid), dim3(64 * WM * WN), 0, s, g);
}

// 8-bit A (FP8 E4M3 / BF8 E5M2), row-major A scales
template <int BM, int BN, int WM, int WN, bool BPACK, int AFMT>
static void launch_tile_a8(const GemmArgs &g, int grid, hipStream_t s)
{
    constexpr int BLAY = BPACK ? 1 : 0;
    if (g.sa_fast && (BPACK ? g.KB % 8 == 0 : g.sb_fast != 0))
        hipLaunchKernelGGL((mx_tile_kernel<BM, BN, WM, WN, BLAY, true, false, AFMT>), dim3(grid), dim3(64 * WM * WN), 0, s, g);
    else
        hipLaunchKernelGGL((mx_tile_kernel<BM, BN, WM, WN, BLAY, false, false, AFMT>), dim3(grid), dim3(64 * WM * WN), 0, s, g);
}

// FP6 A in the dense operand order (launch_fp6_pack), packed B and packed A
// scales; SVEC: whole 8-block stages; persistent under the conditions of the
// FP4 256 x 256 tile
template <int BM, int BN, int WM, int WN, int AFMT>
static void launch_tile_fp6_dense(const GemmArgs &g, int grid, hipStream_t s)
{
    if (g.persist_grid > 0 && g.KB % 8 == 0)
        hipLaunchKernelGGL((mx_tile_kernel<BM, BN, WM, WN, 1, true, true, AFMT, true, true>), dim3(g.persist_grid),
                           dim3(64 * WM * WN), 0, s, g);
    else if (g.KB % 8 == 0)
        hipLaunchKernelGGL((mx_tile_kernel<BM, BN, WM, WN, 1, true, true, AFMT, false, true>), dim3(grid),
                           dim3(64 * WM * WN), 0, s, g);
    else
        hipLaunchKernelGGL((mx_tile_kernel<BM, BN, WM, WN, 1, false, true, AFMT, false, true>), dim3(grid),
                           dim3(64 * WM * WN), 0, s, g);
}

#define MX_TILE_A8(BM, BN, WM, WN, OCC)                                                                    \
    {BM, BN, OCC,                                                                                          \
     {launch_tile_a8<BM, BN, WM, WN, false, 1>, launch_tile_a8<BM, BN, WM, WN, false, 2>,                  \
      launch_tile_a8<BM, BN, WM, WN, false, 3>, launch_tile_a8<BM, BN, WM, WN, false, 4>},                 \
     {launch_tile_a8<BM, BN, WM, WN, true, 1>, launch_tile_a8<BM, BN, WM, WN, true, 2>,                    \
      launch_tile_a8<BM, BN, WM, WN, true, 3>, launch_tile_a8<BM, BN, WM, WN, true, 4>}, "tile_a8_" #BM "x" #BN, \
     false}

const TileKernelA8 *tile_kernels_a8(int *count)
{
    // the dense FP6 tile: 8 waves of 64 x 128 (four A fragments of 24 bytes
    // and eight B fragments per step, the registers the FP4 tile's 128 x 64
    // waves use)
    static const TileKernelA8 table[] = {
        MX_TILE_A8(128, 256, 2, 4, 1),
        MX_TILE_A8(128, 128, 2, 2, 1),
        MX_TILE_A8(64, 64, 2, 2, 3),
        {256, 256, 1, {nullptr, nullptr, nullptr, nullptr},
         {nullptr, nullptr, launch_tile_fp6_dense<256, 256, 4, 2, 3>, launch_tile_fp6_dense<256, 256, 4, 2, 4>},
         "tile_fp6_256x256", true},
    };
    *count = (int)(sizeof(table) / sizeof(table[0]));
    return table;
}
#undef MX_TILE_A8

#define MX_TILE(BM, BN, WM, WN, OCC, DEEP)                                                              \
    {BM, BN, OCC, launch_tile<BM, BN, WM, WN, 0, false>, launch_tile<BM, BN, WM, WN, 1, false>,         \
     launch_tile<BM, BN, WM, WN, 1, true>, launch_tile_deep<BM, BN, WM, WN, false, false>,              \
     launch_tile_deep<BM, BN, WM, WN, true, false>, launch_tile_deep<BM, BN, WM, WN, true, true>,       \
     launch_tile<BM, BN, WM, WN, 2, false>, launch_tile<BM, BN, WM, WN, 3, false>,                      \
     launch_tile<BM, BN, WM, WN, 3, true>, DEEP, "tile_" #BM "x" #BN}

const TileKernel *tile_kernels(int *count)
{
    static const TileKernel table[] = {
        MX_TILE(256, 256, 2, 4, 1, false),
        MX_TILE(256, 128, 2, 2, 1, false),
        MX_TILE(128, 128, 2, 2, 2, false),
        MX_TILE(64, 64, 2, 2, 4, true),
    };
#undef MX_TILE
    *count = (int)(sizeof(table) / sizeof(table[0]));
    return table;
}

}  // namespace mx
