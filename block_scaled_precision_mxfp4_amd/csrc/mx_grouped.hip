// Product grouped by expert on gfx950, a handful of rows in all: B is streamed.
//
// Expert e's rows offsets[e] .. offsets[e+1]-1 of D are its rows of A times
// its B[e]^T.  With few rows the call is bound by the time to the first bytes
// and then by reading the B of every expert that has rows, once.  The grid has
// a line of workgroups for each group of up to 16 rows of one expert, as many
// as the rows can make (found from the offsets by a scan of each 64 experts).
// An expert with many rows has several lines, side by side, which share its B in
// L2, instead of one that passes over B again for each group: 64 experts, N =
// 256, K = 2048, 1024 rows that are all one expert's, 8.0 us against 189 (FP4)
// and 9.7 against 247 (FP8); the same rows spread evenly 8.8 against 9.0 and
// 10.5 against 10.8.  A workgroup's four waves take 64 / KS rows of B, KS waves
// sharing 16 rows and splitting K in pieces of 512 that go straight into
// registers, DEPTH pieces in flight per wave; the waves of a row group add
// their sums through LDS in a fixed order.  The first pieces of B are asked for
// before the row list, whose answer only A needs.
#include "mx_device.hpp"
#include "mx_experts.hpp"
#include "mx_group.hpp"

#include <type_traits>

namespace mx {

template <bool FP8, bool SVEC, int KS, int DEPTH>
__global__ void __launch_bounds__(256) mx_grouped_stream_kernel(GroupedArgs g)
{
    using a_t = typename std::conditional<FP8, v8i, v4i>::type;
    constexpr int AKB = FP8 ? 32 : 16;  // bytes of an A K-block
    __shared__ v4f s_part[4][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ks = wave % KS, wr = wave / KS;  // K share, row group
    int e, m, m1;  // expert, its first row here, its end
    if (!nth_rows(g.offsets, g.E, g.M, kStreamRows, blockIdx.y, lane, e, m, m1))
        return;
    const int n0 = (blockIdx.x * (4 / KS) + wr) * 16;
    const int rows_b = max(0, min(16, g.N - n0));  // (a row group past N reads and writes nothing)
    const int nb = rows_b ? n0 : 0;
    const auto rb = make_rsrc_u(g.B + e * g.eb_b + nb * g.ldb_b, rows_b ? (uint32_t)((rows_b - 1) * g.ldb_b + g.K / 2) : 0u);
    const auto rsb = make_rsrc_u(g.SB + e * g.esb + nb * g.ldsb, rows_b ? (uint32_t)((rows_b - 1) * g.ldsb + g.KB) : 0u);
    const int q = lane & 15, j = lane >> 4;
    const uint32_t b_lane = (uint32_t)(q * g.ldb_b + j * 16);
    const int units = (g.KB + 15) >> 4;
    const Epilogue ep{g.D, nullptr, g.alpha, 0.0f, m1, g.N, g.ldd, 0, g.d_vec, 0, 0};

    struct Piece {
        v4i b[4], sb, sa;
        a_t a[4];
    };
    // (a piece past K: nothing is read)
    auto load_b = [&](int u, Piece &p) __attribute__((always_inline)) {
        p.sb = load_scale_raw<SVEC>(rsb, g.ldsb, q, u * 16, g.KB, lane);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int kb = u * 16 + s * 4;
            p.b[s] = load16_stream(rb, kb + j < g.KB ? b_lane + (uint32_t)(kb * 16) : kOOB);
        }
    };

    Piece p[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        load_b(ks + d * KS, p[d]);
    // the lane's row of A: through the row list, or from row m on
    const int64_t first = g.a_rows ? 0 : m;
    const int a_rows = g.a_rows ? g.a_count : min(16, m1 - m);
    int row = m + q < m1 ? (g.a_rows ? g.a_rows[m + q] : q) : -1;
    const bool on = (uint32_t)row < (uint32_t)a_rows;
    row = on ? row : 0;
    const auto ra = make_rsrc_u(g.A + first * g.lda_b, (uint32_t)((a_rows - 1) * g.lda_b + (int64_t)g.KB * AKB));
    const auto rsa = make_rsrc_u(g.SA + first * g.ldsa, (uint32_t)((a_rows - 1) * g.ldsa + g.KB));
    const uint32_t a_lane = (uint32_t)(row * g.lda_b + j * 16);
    auto load_a = [&](int u, Piece &p) __attribute__((always_inline)) {
        p.sa = load_scale_raw<SVEC>(rsa, g.ldsa, row, u * 16, on ? g.KB : 0, lane);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int kb = u * 16 + s * 4;
            const uint32_t o = a_lane + (uint32_t)(kb * AKB);
            if constexpr (FP8) {
                // K 16j.. and 64 + 16j.. of the step
                const v4i lo = load16(ra, on && kb + j / 2 < g.KB ? o : kOOB);
                const v4i hi = load16(ra, on && kb + 2 + j / 2 < g.KB ? o + 64 : kOOB);
                p.a[s] = v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            } else {
                p.a[s] = load16(ra, on && kb + j < g.KB ? o : kOOB);
            }
        }
    };
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        load_a(ks + d * KS, p[d]);
    v4f acc = {0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](const Piece &p) __attribute__((always_inline)) {
        const int sbw = (int)scale_group_word<SVEC>(p.sb, lane), saw = (int)scale_group_word<SVEC>(p.sa, lane);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            if constexpr (FP8)
                acc = mma_sel_wide<kFmtHw[1]>(s, s, p.b[s], p.a[s], acc, sbw, saw);
            else
                acc = mma_sel(s, s, p.b[s], p.a[s], acc, sbw, saw);
        }
    };
    int u = ks;
    for (; u + KS * DEPTH < units; u += KS * DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            multiply(p[d]);
            load_b(u + (DEPTH + d) * KS, p[d]);
            load_a(u + (DEPTH + d) * KS, p[d]);
        }
    }
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        multiply(p[d]);  // (zeros past K)
    s_part[wave][lane] = acc;
    __syncthreads();
    if (ks == 0) {
#pragma unroll
        for (int w = 1; w < KS; ++w)
            acc += s_part[wave + w][lane];
    }
    // (the matrix instructions read every lane's operands whatever lanes
    // are active: the sums are pinned here, or they and their operands
    // would be moved behind the store's bounds check, where lanes outside
    // D no longer make theirs)
    asm volatile("" : "+v"(acc));
    if (ks == 0)
        store_quad(ep, m + q, n0 + 4 * j, acc);
}

// Two waves a row group, two pieces in flight each.  On MI355X (32 experts, N =
// 4096, K = 2048; cold weights): one token's 4 experts 7.2 us FP4, 7.6 FP8,
// against 7.8 and 10.7 with four waves splitting K (a workgroup per 16 rows:
// twice as many to start) and 6.8 and 7.8 with none splitting it and four
// pieces in flight, which is 10.2 against 7.3 us where K is 4096 and N 2880.
constexpr int kStreamKs = 2, kStreamDepth = 2;

template <bool FP8>
static void launch_stream_as(const GroupedArgs &g, hipStream_t s)
{
    constexpr int R = 64 / kStreamKs;  // rows of B per workgroup
    const dim3 grid((unsigned)((g.N + R - 1) / R), (unsigned)grouped_stream_lines(g.M, g.E));
    if (g.scale16)
        hipLaunchKernelGGL((mx_grouped_stream_kernel<FP8, true, kStreamKs, kStreamDepth>), grid, dim3(256), 0, s, g);
    else
        hipLaunchKernelGGL((mx_grouped_stream_kernel<FP8, false, kStreamKs, kStreamDepth>), grid, dim3(256), 0, s, g);
}

void launch_grouped_stream(bool fp8, const GroupedArgs &g, hipStream_t s)
{
    if (fp8)
        launch_stream_as<true>(g, s);
    else
        launch_stream_as<false>(g, s);
}

}  // namespace mx
