// Product grouped by expert on gfx950, few rows per expert: B is streamed.
//
// Expert e's rows offsets[e] .. offsets[e+1]-1 of D are its rows of A times
// its B[e]^T.  With few rows per expert the call is bound by reading the B of
// every expert that has rows, once; the grid has a line of workgroups for
// each of at most min(E, rows) such experts (found from the offsets by one
// ballot per 64 experts), each workgroup taking 16 NR rows of B.  Its four
// waves split K in pieces of 512, so that all of a workgroup's loads are in
// flight together, and add their partial sums through LDS in a fixed order.
// An expert with more than 16 MG rows is done in several passes over B.
#include "mx_device.hpp"
#include "mx_experts.hpp"
#include "mx_group.hpp"

#include <type_traits>

namespace mx {

template <bool FP8, int MG, int NR, bool SVEC>
__global__ void __launch_bounds__(256) mx_grouped_stream_kernel(GroupedTileArgs g)
{
    using a_t = typename std::conditional<FP8, v8i, v4i>::type;
    constexpr int AKB = FP8 ? 32 : 16;  // bytes of an A K-block
    __shared__ v4f s_part[4][MG * NR][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int e, m0, m1;
    if (!nth_group(g.offsets, g.E, g.M, blockIdx.y, lane, e, m0, m1))
        return;
    const int n0 = blockIdx.x * 16 * NR;
    const int rows_b = min(16 * NR, g.N - n0);
    const auto rb = make_rsrc_u(g.B + e * g.eb_b + n0 * g.ldb_b, (uint32_t)((rows_b - 1) * g.ldb_b + g.K / 2));
    const auto rsb = make_rsrc_u(g.SB + e * g.esb + n0 * g.ldsb, (uint32_t)((rows_b - 1) * g.ldsb + g.KB));
    const int q = lane & 15, j = lane >> 4;
    const uint32_t b_lane = (uint32_t)(q * g.ldb_b + j * 16);
    const int units = (g.KB + 15) >> 4;
    Epilogue ep{g.D, nullptr, g.alpha, 0.0f, m1, g.N, g.ldd, 0, g.d_vec, 0, 0};

    for (int m = m0; m < m1; m += 16 * MG) {
        // this pass's A rows: through the row list, or from row m on
        const uint8_t *A = g.A, *SA = g.SA;
        int64_t a_rows = g.a_count;
        int arow[MG];
#pragma unroll
        for (int mg = 0; mg < MG; ++mg) {
            const int i = mg * 16 + q;
            arow[mg] = m + i < m1 ? (g.a_rows ? g.a_rows[m + i] : i) : -1;
        }
        if (!g.a_rows) {
            A += m * g.lda_b;
            SA += m * g.ldsa;
            a_rows = min(16 * MG, m1 - m);
        }
#pragma unroll
        for (int mg = 0; mg < MG; ++mg)
            arow[mg] = (uint32_t)arow[mg] < (uint32_t)a_rows ? arow[mg] : -1;
        const auto ra = make_rsrc_u(A, (uint32_t)((a_rows - 1) * g.lda_b + (int64_t)g.KB * AKB));
        const auto rsa = make_rsrc_u(SA, (uint32_t)((a_rows - 1) * g.ldsa + g.KB));

        v4f acc[NR][MG];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int mg = 0; mg < MG; ++mg)
                acc[nr][mg] = v4f{0.f, 0.f, 0.f, 0.f};
        for (int u = wave; u < units; u += 4) {
            const int kb0 = u * 16;
            v4i b[4][NR], sbr[NR], sar[MG];
            a_t a[4][MG];
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
                sbr[nr] = load_scale_raw<SVEC>(rsb, g.ldsb, nr * 16 + q, kb0, g.KB, lane);
#pragma unroll
            for (int mg = 0; mg < MG; ++mg)
                sar[mg] = load_scale_raw<SVEC>(rsa, g.ldsa, max(arow[mg], 0), kb0, arow[mg] < 0 ? 0 : g.KB, lane);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int kb = kb0 + s * 4;
#pragma unroll
                for (int nr = 0; nr < NR; ++nr)
                    b[s][nr] = load16_stream(rb, kb + j < g.KB ? b_lane + (uint32_t)(nr * 16 * g.ldb_b + kb * 16) : kOOB);
#pragma unroll
                for (int mg = 0; mg < MG; ++mg) {
                    const uint32_t row = (uint32_t)(max(arow[mg], 0) * g.lda_b);
                    const bool on = arow[mg] >= 0;
                    if constexpr (FP8) {
                        // K 16j.. and 64 + 16j.. of the step
                        const uint32_t o = row + (uint32_t)(kb * 32 + j * 16);
                        const v4i lo = load16(ra, on && kb + j / 2 < g.KB ? o : kOOB);
                        const v4i hi = load16(ra, on && kb + 2 + j / 2 < g.KB ? o + 64 : kOOB);
                        a[s][mg] = v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                    } else {
                        a[s][mg] = load16(ra, on && kb + j < g.KB ? row + (uint32_t)((kb + j) * 16) : kOOB);
                    }
                }
            }
            uint32_t sbw[NR], saw[MG];
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
                sbw[nr] = scale_group_word<SVEC>(sbr[nr], lane);
#pragma unroll
            for (int mg = 0; mg < MG; ++mg)
                saw[mg] = scale_group_word<SVEC>(sar[mg], lane);
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                    for (int mg = 0; mg < MG; ++mg) {
                        if constexpr (FP8)
                            acc[nr][mg] = mma_sel_wide<kFmtHw[1]>(s, s, b[s][nr], a[s][mg], acc[nr][mg], (int)sbw[nr], (int)saw[mg]);
                        else
                            acc[nr][mg] = mma_sel(s, s, b[s][nr], a[s][mg], acc[nr][mg], (int)sbw[nr], (int)saw[mg]);
                    }
        }
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int mg = 0; mg < MG; ++mg)
                s_part[wave][nr * MG + mg][lane] = acc[nr][mg];
        __syncthreads();
        for (int f = wave; f < MG * NR; f += 4) {
            v4f sum = s_part[0][f][lane];
#pragma unroll
            for (int w = 1; w < 4; ++w)
                sum += s_part[w][f][lane];
            store_quad(ep, m + (f % MG) * 16 + q, n0 + (f / MG) * 16 + 4 * j, sum);
        }
        __syncthreads();
    }
}

template <bool FP8, int MG, int NR>
static void launch_stream_as(const GroupedTileArgs &g, hipStream_t s)
{
    const dim3 grid((unsigned)((g.N + 16 * NR - 1) / (16 * NR)), (unsigned)(g.E < g.M ? g.E : g.M));
    if (g.scale16)
        hipLaunchKernelGGL((mx_grouped_stream_kernel<FP8, MG, NR, true>), grid, dim3(256), 0, s, g);
    else
        hipLaunchKernelGGL((mx_grouped_stream_kernel<FP8, MG, NR, false>), grid, dim3(256), 0, s, g);
}

void launch_grouped_stream(bool fp8, const GroupedTileArgs &g, hipStream_t s)
{
    if (fp8)
        launch_stream_as<true, 1, 1>(g, s);
    else
        launch_stream_as<false, 1, 1>(g, s);
}

}  // namespace mx
