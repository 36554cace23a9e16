// Product grouped by expert on gfx950, the tiled kernel: each workgroup of WM x
// WN waves computes a BM x BN tile of one expert's rows of D.
//
// The tile's expert and rows come from the device's offsets, its rows of A
// through the row list where there is one: a lane keeps the byte offsets of
// the rows it loads in registers, so gathered rows cost what consecutive ones
// do.  Per 256-K stage, double-buffered:
//   - operand rows go from HBM/L2 straight into LDS with 16-byte-per-lane
//     buffer loads, 8 rows x 128 bytes (whole lines) an instruction;
//   - each thread brings one row's scale bytes, A's or B's: 16 bytes every
//     other stage, for it and the next (a row's 8 bytes per stage cost a whole
//     line each time: 217 -> 207 us at 8192 tokens x top 4, N = 4096, K =
//     2048), stored to LDS as 8 bytes a row.  A matrix instruction's lane reads
//     its row's four bytes of the 128-K step and shifts its K-block's to byte
//     0 (op_sel 0), so that no words are assembled.
// A stage is one basic block (a branch in it, also one that a whole wave
// takes, made the accumulators leave their registers: 207 -> 753 us).
//
// A operand rows of a 16-row group (2 KiB of LDS): row r, 16-byte chunk c at
// slot (r/8)*64 + (r%8)*8 + (c ^ sw(r)), sw(r) = 2*bit1(r) + 4*bit3(r): a
// fragment read (row lane%16, chunk 4ks + lane/16) touches every bank once.
// An 8-bit A stage is two such tiles, one per 128-K step; a lane's operand is
// chunks g and g+4 of its step's tile, the two 16-element runs K 16g.. and
// 64+16g.. the 8-bit instruction reads.
//
// SVEC: scale rows in whole 16-byte aligned groups of 16 K-blocks.  Otherwise
// the scale loads are unaligned and end at the row's end, the bytes are
// shifted when they are stored (not when they arrive: that wait stood before
// the stage's multiplies, 449 -> 232 us at K = 2080), and the codes past K,
// those of the next row or of its padding, are multiplied, by the scale bytes
// 0 that stand there for both operands: 2^-254 times at most 36 * 32 is below
// half of fp32's least value, so that nothing is added.  An 8-bit A may hold a
// NaN there and is masked.
//
// PERSIST: one workgroup per CU walks its tiles (hardware ids blockIdx + i *
// grid, through the XCD remap).  The experts' table is made once in LDS; the
// next tile's rows are looked up and their row list read behind the last
// stage's multiplies; its first stage is loaded into buffer 0 before D is
// written through buffer 1's A half, so that the latency hides behind the
// epilogue.  8-bit A on 128 x 256, 8192 tokens x top 4, K = 2048: 304 -> 289
// us; the FP4 256 x 256 tile has no registers left for it (13 spilled, 207 ->
// 212 us).
//
// Bound (FP4, 256 x 256, the shape above: 195-203 us, 2.7-2.8 PFLOP/s): a stage
// takes about 4300 cycles of which 2048 are matrix instructions, as in the
// dense kernel on row-major operands (181 us for the same flops in one group;
// 156 us with packed ones); partly filled tiles are 12 % of the work.
#include "mx_device.hpp"
#include "mx_experts.hpp"
#include "mx_group.hpp"
#include "mx_pipe.hpp"

#include <type_traits>

namespace mx {

// (of known address space: a load through a pointer made from an integer
// would also take the LDS's path)
typedef __attribute__((address_space(1))) uint8_t global_u8;

// A row's scale bytes of 8 K-blocks from kb on at any alignment: one load that
// ends at the row's end at the latest, to be shifted by scale_row_shift.  base
// is wave-uniform, row the lane's offset.
__device__ __forceinline__ uint64_t load_scale_row_any(const global_u8 *base, uint32_t row, int kb, int KB)
{
    typedef uint64_t __attribute__((aligned(1))) any_u64;
    return *reinterpret_cast<const __attribute__((address_space(1))) any_u64 *>(base + max(min(kb, KB - 8), 0) + row);
}

// ... of a whole row of fewer than 8 blocks, byte by byte, as if the load
// had begun 8 - KB bytes before it.
__device__ __forceinline__ uint64_t load_scale_row_short(const global_u8 *base, uint32_t row, int KB)
{
    uint64_t w = 0;
    for (int i = 0; i < KB; ++i)
        w |= (uint64_t)base[row + i] << (8 * (8 - KB + i));
    return w;
}

// ... to block kb's byte first and zeros for blocks at or past KB.
__device__ __forceinline__ uint64_t scale_row_shift(uint64_t w, int kb, int KB)
{
    const int past = kb - min(kb, KB - 8);
    return past < 8 ? w >> (8 * past) : 0;
}

// D[m + r][n + c] = bf16(alpha * acc), staged through the wave's private LDS
// region as store_tile_staged does, with buffer stores whose range ends the
// tile: every lane stores the same number of times whatever part of the tile
// is inside.  `lane` comes in through an opaque register, so that the
// addresses are formed per tile instead of being kept over the tile loop,
// where they would be spilled.  rD covers D from the tile's first
// element to the last one inside, `m` and `n` are the wave tile's place in the
// tile, columns from n_end on (a multiple of 8) are dropped by an offset past
// the range, rows past the end by the range itself.
template <int FM, int FN>
__device__ __forceinline__ void store_range_tile_staged(__amdgpu_buffer_rsrc_t rD, uint32_t ldd, float alpha, int m, int n,
                                                        int n_end, const v4f (&acc)[FN][FM], uint8_t *lds, int lane)
{
    constexpr int RB = FN * 32, CH = RB / 16, RPI = 64 / CH;
    static_assert(CH == 2 || CH == 4 || CH == 8 || CH == 16, "row chunking");
    auto sw = [](int r) { return CH == 16 ? (r & 15) : ((r >> 1) & (CH - 1)); };
#pragma unroll
    for (int fn = 0; fn < FN; ++fn)
#pragma unroll
        for (int fm = 0; fm < FM; ++fm) {
            const int r = fm * 16 + (lane & 15);
            const int j = fn * 2 + (lane >> 5);
            v2u o;
            o[0] = bf16x2_rne(alpha * acc[fn][fm][0], alpha * acc[fn][fm][1]);
            o[1] = bf16x2_rne(alpha * acc[fn][fm][2], alpha * acc[fn][fm][3]);
            *reinterpret_cast<v2u *>(lds + r * RB + ((j ^ sw(r)) * 16) + ((lane >> 4) & 1) * 8) = o;
        }
    const int r0 = lane / CH, c = lane & (CH - 1);
    const uint32_t off = n + c * 8 < n_end ? ((uint32_t)(m + r0) * ldd + (uint32_t)(n + c * 8)) * 2 : 0x80000000u;
#pragma unroll
    for (int i = 0; i < FM * 16 / RPI; ++i) {
        const int r = i * RPI + r0;
        const v4i v = *reinterpret_cast<const v4i *>(lds + r * RB + ((c ^ sw(r)) * 16));
        __builtin_amdgcn_raw_buffer_store_b128(v, rD, off + (uint32_t)(i * RPI) * ldd * 2, 0, kStream);
    }
}

template <int BM, int BN, int WM, int WN, bool SVEC, bool FP8, bool PERSIST>
__global__ void __launch_bounds__(64 * WM * WN) mx_tile_grouped_kernel(GroupedArgs g)
{
    constexpr int AREG = FP8 ? 2 : 1;          // FP4-shaped A tiles per stage
    constexpr int NW = WM * WN, NT = 64 * NW;  // waves, threads
    constexpr int TM = BM / WM, TN = BN / WN;  // wave tile
    constexpr int FM = TM / 16, FN = TN / 16;  // 16-row fragments per wave
    static_assert(NW == 4 || NW == 8, "four or eight waves");
    constexpr uint32_t kFar = 0x80000100u;     // past every range, also with a stage's offsets added
    constexpr int A_STAGE = BM * 128 * AREG, B_STAGE = BN * 128;  // bytes per stage
    constexpr int A_CH = A_STAGE / 1024, B_CH = B_STAGE / 1024;   // 1 KiB load instructions
    static_assert(A_CH % NW == 0 && B_CH % NW == 0, "loads split evenly over waves");
    static_assert(NW % 2 == 0 && (BM / 8) % 2 == 0, "a wave's loads are all of one 8-row half");
    // scale rows: A's in waves 0 .. XA-1, B's in the next XB
    constexpr int XA = (BM + 63) / 64, XB = (BN + 63) / 64;
    static_assert(XA + XB <= NW, "one scale row per thread, a wave's of one operand");

    // The two halves of each double buffer are distinct LDS objects and every
    // access names one of them at compile time: the compiler can then tell
    // the next stage's direct-to-LDS loads from this stage's fragment reads
    // and does not make the reads wait for the loads.
    __shared__ __attribute__((aligned(1024))) uint8_t s_a0[A_STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t s_a1[A_STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t s_b0[B_STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t s_b1[B_STAGE];
    __shared__ uint32_t s_sc0[NT * 2];
    __shared__ uint32_t s_sc1[NT * 2];
    __shared__ int s_lo[PERSIST ? kGroupTable : 1], s_hi[PERSIST ? kGroupTable : 1], s_upto[PERSIST ? kGroupTable : 1];
    __shared__ int s_total;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wave_m = wave % WM, wave_n = wave / WM;

    // ---- the tile
    int e = 0, m0 = 0, m_end = 0, n0 = 0;      // expert, first row, the expert's end, first column
    int raw_a[A_CH / NW], raw_x = 0;           // row numbers as read: A's rows, the scale row
    uint32_t a_row[A_CH / NW], x_row = 0;      // byte offsets of A's rows (with the chunk) and of the scale row
    const uint8_t *a_base = nullptr, *b_base = nullptr;
    const global_u8 *x_base = nullptr;
    bool x_in = false;                         // the scale row is there
    uint32_t a_bytes = 0, b_bytes = 0;
    __amdgpu_buffer_rsrc_t rsx = make_rsrc(nullptr, 0);
    // chunk of lane l in the wave's 8-row half (the rows' swizzle)
    const int kc_lane = (lane & 7) ^ (2 * ((lane >> 4) & 1)) ^ (4 * (wave & 1));
    const uint32_t b_lane = (uint32_t)((lane >> 3) * g.ldb_b + kc_lane * 16);
    // stages; the persistent form needs an even count (a stage past K
    // multiplies zeros)
    const int nst = PERSIST ? (g.KB + 15) / 16 * 2 : (g.KB + 7) / 8;

    // rows of the tile: of A's load i, and of the thread's scales (A's or B's)
    auto a_tile_row = [&](int i) __attribute__((always_inline)) { return ((i * NW + wave) % (BM / 8)) * 8 + (lane >> 3); };
    const int x_tile_row = wave < XA ? tid : tid - XA * 64;
    // first part: expert, rows and columns, and the row list's values, which
    // are used in the second one, after whatever hides their latency.  Rows
    // past the expert's end are -1: the plain form reads its last row's number
    // for them and drops it in row_of, because a condition here makes each
    // load wait (45.0 -> 43.8 us for 2036 rows of 64 experts, N = 1440, K =
    // 2880); in the persistent form, whose wait is hidden, the condition here is
    // the faster one (279 against 284 us, the shape below)
    auto find_tile = [&](int wg, int total) __attribute__((always_inline)) {
        GroupTile gt;
        if constexpr (PERSIST) {
            if (!table_tile(s_lo, s_hi, s_upto, g.E, BM, g.tiles_n, g.group_m, xcd_remap(wg, total), lane, gt))
                return false;
        } else {
            if (!group_tile(g.offsets, g.E, g.M, BM, g.tiles_n, g.group_m, wg, lane, gt))
                return false;
        }
        e = __builtin_amdgcn_readfirstlane(gt.e);
        m0 = __builtin_amdgcn_readfirstlane(gt.m0);
        m_end = __builtin_amdgcn_readfirstlane(gt.m1);
        n0 = __builtin_amdgcn_readfirstlane(gt.tn) * BN;
        if constexpr (PERSIST) {
            auto read = [&](int r) __attribute__((always_inline)) {
                return m0 + r < m_end ? (g.a_rows ? g.a_rows[m0 + r] : r) : -1;
            };
#pragma unroll
            for (int i = 0; i < A_CH / NW; ++i)
                raw_a[i] = read(a_tile_row(i));
            raw_x = wave < XA && x_tile_row < BM ? read(x_tile_row) : -1;
        } else if (g.a_rows) {
#pragma unroll
            for (int i = 0; i < A_CH / NW; ++i)
                raw_a[i] = g.a_rows[min(m0 + a_tile_row(i), m_end - 1)];
            raw_x = g.a_rows[min(m0 + x_tile_row, m_end - 1)];
        }
        return true;
    };
    auto row_of = [&](int r, int raw) __attribute__((always_inline)) {
        return PERSIST ? raw : m0 + r < m_end ? (g.a_rows ? raw : r) : -1;
    };
    auto set_tile_b = [&]() __attribute__((always_inline)) {
        b_base = g.B + e * g.eb_b + n0 * g.ldb_b;
        b_bytes = (uint32_t)((min(BN, g.N - n0) - 1) * g.ldb_b + (int64_t)g.KB * 16);
    };
    auto set_tile_a = [&]() __attribute__((always_inline)) {
        // without a row list the tile's own rows, from its first one on
        const int64_t first = g.a_rows ? 0 : m0;
        const int rows_a = g.a_rows ? g.a_count : min(BM, m_end - m0);
        const int rows_b = min(BN, g.N - n0);
#pragma unroll
        for (int i = 0; i < A_CH / NW; ++i) {
            const int r = row_of(a_tile_row(i), raw_a[i]);
            a_row[i] = (uint32_t)r < (uint32_t)rows_a ? (uint32_t)(r * g.lda_b) + (uint32_t)(kc_lane * 16) : kFar;
        }
        a_base = g.A + first * g.lda_b;
        a_bytes = (uint32_t)((rows_a - 1) * g.lda_b + (int64_t)g.KB * 16 * AREG);
        const bool xa = wave < XA, xb = !xa && wave < XA + XB;
        const int r = xa ? row_of(x_tile_row, raw_x) : x_tile_row;
        const int rows_x = xa ? rows_a : rows_b;
        const int64_t ldx = xa ? g.ldsa : g.ldsb;
        x_in = (xa ? x_tile_row < BM : xb && x_tile_row < BN) && (uint32_t)r < (uint32_t)rows_x;
        x_row = x_in ? (uint32_t)(r * ldx) : SVEC ? kFar : 0u;
        const uint64_t xp = (uint64_t)(uintptr_t)(xa ? g.SA + first * g.ldsa : g.SB + e * g.esb + n0 * g.ldsb);
        const uint32_t xlo = __builtin_amdgcn_readfirstlane((uint32_t)xp);  // (to unsigned: no sign is extended)
        const uint32_t xhi = __builtin_amdgcn_readfirstlane((uint32_t)(xp >> 32));
        x_base = (const global_u8 *)(((uint64_t)xhi << 32) | xlo);
        rsx = make_rsrc_u((const void *)(uintptr_t)xp, xa || xb ? (uint32_t)((rows_x - 1) * ldx + g.KB) : 0u);
    };
    int unit = blockIdx.x, units = 0;
    if constexpr (PERSIST) {
        if (wave == 0) {
            const int total = make_group_table(g.offsets, g.E, g.M, BM, s_lo, s_hi, s_upto, lane);
            if (lane == 0)
                s_total = total;
        }
        __syncthreads();
        // (no more than rows can make when the offsets ascend: what they hold
        // does not decide how long this runs)
        const int some = min(g.E, g.M);
        units = min(__builtin_amdgcn_readfirstlane(s_total), (g.M - some) / BM + some) * g.tiles_n;
        if (unit >= units)
            return;
    }
    if (!find_tile(unit, units))
        return;

    // ---- stage loaders.  Per stage the base advances along K and the range
    // shrinks by the same amount; a stage that must not load gets an empty
    // range: every load returns zeros without traffic.
    auto issue_operands = [&](int kt, bool on, auto bufc, auto whichc) __attribute__((always_inline)) {
        constexpr int BUF = decltype(bufc)::value, WHICH = decltype(whichc)::value;  // WHICH: 1 A, 2 B, 3 both
        uint8_t *dst_a = BUF ? s_a1 : s_a0;
        uint8_t *dst_b = BUF ? s_b1 : s_b0;
        const int kb_s = kt * 8;
        if constexpr (PERSIST && !SVEC)
            on = on && kb_s < g.KB;
        const uint32_t a_k = (uint32_t)kb_s * 16 * AREG, b_k = (uint32_t)kb_s * 16;
        const auto ra = make_rsrc(a_base + a_k, on ? a_bytes - a_k : 0u);
        const auto rb = make_rsrc(b_base + b_k, on ? b_bytes - b_k : 0u);
#pragma unroll
        for (int i = 0; i < (WHICH & 1 ? A_CH / NW : 0); ++i) {
            const int c = i * NW + wave;
            uint32_t off = a_row[i];
            if constexpr (FP8) {
                const int step = c / (BM / 8);  // 128-K step of the stage
                off += (uint32_t)(step * 128);
                if constexpr (!SVEC)  // (chunk kc covers half of K-block kc / 2)
                    off = kb_s + 4 * step + kc_lane / 2 < g.KB ? off : kOOB;
            }
            load16_to_lds(ra, (lds_void *)(dst_a + c * 1024), off);
        }
#pragma unroll
        for (int i = 0; i < (WHICH & 2 ? B_CH / NW : 0); ++i) {
            const int c = i * NW + wave;
            load16_to_lds(rb, (lds_void *)(dst_b + c * 1024), b_lane + (uint32_t)(c * 8 * g.ldb_b));
        }
    };
    [[maybe_unused]] v4i x_raw = {0, 0, 0, 0};
    [[maybe_unused]] uint64_t x_any[2] = {0, 0};
    [[maybe_unused]] int x_kb = 0;
    // (past the last stage: inside the rows or the range, never used)
    auto issue_scales = [&](int kt, bool on, auto bufc) __attribute__((always_inline)) {
        constexpr int BUF = decltype(bufc)::value;
        const int kb_s = kt * 8;
        if constexpr (BUF == 0 && SVEC) {
            x_raw = load16(rsx, on ? x_row + kb_s : kOOB);
        } else if constexpr (BUF == 0) {
            x_any[0] = load_scale_row_any(x_base, x_row, kb_s, g.KB);
            x_any[1] = load_scale_row_any(x_base, x_row, kb_s + 8, g.KB);
            x_kb = kb_s;
        }
    };
    auto commit_scales = [&](auto bufc) __attribute__((always_inline)) {
        constexpr int BUF = decltype(bufc)::value;
        uint32_t *dst = (BUF ? s_sc1 : s_sc0) + tid * 2;
        if constexpr (SVEC)
            *reinterpret_cast<v2i *>(dst) = v2i{x_raw[2 * BUF], x_raw[2 * BUF + 1]};
        else
            *reinterpret_cast<uint64_t *>(dst) = x_in ? scale_row_shift(x_any[BUF], x_kb + 8 * BUF, g.KB) : 0;
    };

    // LDS byte offset of this lane's 16 bytes of a fragment inside its 16-row
    // group (row lane%16, K-block lane/16 of step 0; step 1 flips chunk bit 2)
    const int fr = lane & 15;
    const int sw_fr = 2 * ((fr >> 1) & 1) + 4 * ((fr >> 3) & 1);
    const uint32_t rl0 = (uint32_t)(((fr >> 3) * 64 + (fr & 7) * 8 + ((lane >> 4) ^ sw_fr)) * 16);
    const uint32_t rl1 = rl0 ^ 64u;

    // ---- main loop
    // Accumulators get their first value from the first stage's matrix
    // instructions (zero accumulator input), never from a register move, so
    // the register allocator keeps them in the accumulation registers.
    v4f acc[FN][FM];
    using B0 = std::integral_constant<int, 0>;
    using B1 = std::integral_constant<int, 1>;
    using Both = std::integral_constant<int, 3>;

    // One stage: prefetch stage kt+1 into the other buffer, multiply stage kt,
    // then wait for the prefetch and publish its scales.  LOADS_AT places the
    // prefetch: -1 lets the compiler interleave it, P >= 0 issues it just
    // before fragment step P (P = ks * FN + fn).
    auto stage = [&](int kt, auto bufc, auto firstc, auto loadsc) __attribute__((always_inline)) {
        constexpr int BUF = decltype(bufc)::value;
        constexpr bool FIRST = decltype(firstc)::value;
        constexpr int LOADS_AT = decltype(loadsc)::value;
        using Next = std::integral_constant<int, BUF ^ 1>;
        const bool more = kt + 1 < nst;
        auto prefetch = [&]() __attribute__((always_inline)) {
            if constexpr (LOADS_AT >= 0)
                __builtin_amdgcn_sched_barrier(0);
            issue_operands(kt + 1, more, Next{}, Both{});
            issue_scales(kt + 1, more, Next{});
            if constexpr (LOADS_AT >= 0)
                __builtin_amdgcn_sched_barrier(0);
        };
        if constexpr (LOADS_AT <= 0)
            prefetch();
        const uint8_t *sa_tile = BUF ? s_a1 : s_a0;
        const uint8_t *sb_tile = BUF ? s_b1 : s_b0;
        const uint32_t *ssc = BUF ? s_sc1 : s_sc0;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            using a_t = typename std::conditional<FP8, v8i, v4i>::type;
            a_t af[FM];
            uint32_t sa[FM], sb[FN];
            const uint32_t rl = ks ? rl1 : rl0;
            const uint32_t *sc = ssc + fr * 2 + ks;
#pragma unroll
            for (int fm = 0; fm < FM; ++fm)
                sa[fm] = sc[(wave_m * TM + fm * 16) * 2] >> (8 * (lane >> 4));
#pragma unroll
            for (int fn = 0; fn < FN; ++fn)
                sb[fn] = sc[(XA * 64 + wave_n * TN + fn * 16) * 2] >> (8 * (lane >> 4));
#pragma unroll
            for (int fm = 0; fm < FM; ++fm) {
                if constexpr (FP8) {
                    const uint8_t *t = sa_tile + ks * (BM * 128) + (wave_m * FM + fm) * 2048;
                    const v4i lo = *reinterpret_cast<const v4i *>(t + rl0);
                    const v4i hi = *reinterpret_cast<const v4i *>(t + rl1);
                    af[fm] = v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                } else {
                    af[fm] = *reinterpret_cast<const v4i *>(sa_tile + (wave_m * FM + fm) * 2048 + rl);
                }
            }
#pragma unroll
            for (int fn = 0; fn < FN; ++fn) {
                if constexpr (LOADS_AT > 0) {
                    if (ks * FN + fn == LOADS_AT)
                        prefetch();
                }
                const v4i bf = *reinterpret_cast<const v4i *>(sb_tile + (wave_n * FN + fn) * 2048 + rl);
#pragma unroll
                for (int fm = 0; fm < FM; ++fm) {
                    const v4f from = FIRST && ks == 0 ? v4f{0.f, 0.f, 0.f, 0.f} : acc[fn][fm];
                    if constexpr (FP8)
                        acc[fn][fm] = mfma_fp4_wide<kFmtHw[1], 0, 0>(bf, af[fm], from, (int)sb[fn], (int)sa[fm]);
                    else
                        acc[fn][fm] = mfma_fp4<0, 0>(bf, af[fm], from, (int)sb[fn], (int)sa[fm]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        wait_vmcnt<0>();
        commit_scales(Next{});
        __syncthreads();
    };

    // (B first: the row list is still under way)
    set_tile_b();
    if constexpr (!PERSIST)
        issue_operands(0, true, B0{}, std::integral_constant<int, 2>{});
    set_tile_a();
    issue_operands(0, true, B0{}, std::integral_constant<int, PERSIST ? 3 : 1>{});
    if (!SVEC && !PERSIST && g.KB < 8) {
        // (one stage, with no scale loads of its own: the first stage's bring
        // those of two)
        x_any[0] = load_scale_row_short(x_base, x_row, g.KB);
    } else {
        issue_scales(0, true, B0{});
    }
    wait_vmcnt<0>();
    commit_scales(B0{});
    __syncthreads();
    using First = std::true_type;
    using Rest = std::false_type;
    for (;;) {
        [[maybe_unused]] const int this_m0 = m0, this_n0 = n0, this_end = m_end;
        [[maybe_unused]] bool next_found = false;
        // stage 0 is peeled (it initialises the accumulators); then pairs of
        // stages keep the buffer choice static
        auto run = [&](auto loadsc) __attribute__((always_inline)) {
            stage(0, B0{}, First{}, loadsc);
            int kt = 1;
            for (; kt + 2 <= nst; kt += 2) {
                stage(kt, B1{}, Rest{}, loadsc);
                stage(kt + 1, B0{}, Rest{}, loadsc);
            }
            if constexpr (PERSIST)  // (every operand load of this tile is out)
                next_found = unit + (int)gridDim.x < units && find_tile(unit + (int)gridDim.x, units);
            if (kt < nst)
                stage(kt, B1{}, Rest{}, loadsc);
        };
        if constexpr (NW == 8) {
            // eight waves, two per SIMD (w and w + 4): one prefetches before
            // its first multiply, the other before fragment step 3, so that
            // one multiplies while the other waits on the load path
            if (wave >= 4)
                run(std::integral_constant<int, 3>{});
            else
                run(std::integral_constant<int, 0>{});
        } else {
            run(std::integral_constant<int, -1>{});
        }
        if constexpr (!PERSIST)
            break;
        if (next_found) {
            // the next tile's first stage into buffer 0 (its last readers
            // passed the barrier ending stage nst - 2)
            set_tile_b();
            set_tile_a();
            issue_operands(0, true, B0{}, Both{});
            issue_scales(0, true, B0{});
        }
        // D through the last stage's A buffer, 1/PARTS of the wave tile at a
        // time in a region of the wave's own: naming that one array lets the
        // compiler tell the staging from the loads into the other buffer
        int lane_e = lane;
        asm volatile("" : "+v"(lane_e));
        constexpr int PARTS = NW * TM * TN * 2 <= A_STAGE ? 1 : NW * TM * TN <= A_STAGE ? 2 : 4;
        constexpr int QREG = (TM / PARTS) * TN * 2;
        static_assert(!PERSIST || (NW * QREG <= A_STAGE && FM % PARTS == 0), "partial-tile staging fits the A buffer");
        uint8_t *buf = s_a1 + wave * QREG;
        const auto rD = make_rsrc_u(g.D + (int64_t)this_m0 * g.ldd + this_n0,
                                    (uint32_t)(((min(BM, this_end - this_m0) - 1) * g.ldd + min(BN, g.N - this_n0)) * 2));
        if constexpr (PERSIST) {
#pragma unroll
            for (int part = 0; part < PARTS; ++part) {
                v4f q[FN][FM / PARTS];
#pragma unroll
                for (int fn = 0; fn < FN; ++fn)
#pragma unroll
                    for (int i = 0; i < FM / PARTS; ++i)
                        q[fn][i] = acc[fn][part * (FM / PARTS) + i];
                store_range_tile_staged<FM / PARTS, FN>(rD, (uint32_t)g.ldd, g.alpha, wave_m * TM + part * (TM / PARTS),
                                                        wave_n * TN, g.N - this_n0, q, buf, lane_e);
            }
        }
        if (!next_found)
            return;
        // the first-stage loads were issued before this wave's STORES stores:
        // in-order completion makes them landed at STORES outstanding
        constexpr int STORES = FM * 16 / (64 / (FN * 2));
        wait_vmcnt<STORES>();
        commit_scales(B0{});
        // the stage and its scales are in place, and every wave is done with
        // its staging region before the next stage is loaded over it
        __syncthreads();
        unit += (int)gridDim.x;
    }

    // ---- epilogue of the plain grid
    const Epilogue ep{g.D, nullptr, g.alpha, 0.0f, m_end, g.N, g.ldd, 0, g.d_vec, 0, 0};
    if (g.d_stage) {
        // every wave has passed the last stage's barrier (after waiting for
        // its loads): the operand buffers are free; each wave takes a private
        // TM x TN bf16 region
        constexpr int REG = TM * TN * 2;
        constexpr int RPA = A_STAGE / REG, RPB = B_STAGE / REG;
        static_assert(NW <= 2 * RPA + 2 * RPB, "staging regions fit the operand buffers");
        uint8_t *buf;
        if (wave < RPA)
            buf = s_a0 + wave * REG;
        else if (wave < 2 * RPA)
            buf = s_a1 + (wave - RPA) * REG;
        else if (wave < 2 * RPA + RPB)
            buf = s_b0 + (wave - 2 * RPA) * REG;
        else
            buf = s_b1 + (wave - 2 * RPA - RPB) * REG;
        store_tile_staged<FM, FN>(ep, m0 + wave_m * TM, n0 + wave_n * TN, acc, buf);
        return;
    }
#pragma unroll
    for (int fn = 0; fn < FN; ++fn)
#pragma unroll
        for (int fm = 0; fm < FM; ++fm) {
            // (pinned outside the store's bounds check: the matrix
            // instructions need every lane's operands)
            v4f sum = acc[fn][fm];
            asm volatile("" : "+v"(sum));
            store_quad(ep, m0 + wave_m * TM + fm * 16 + fr, n0 + wave_n * TN + fn * 16 + 4 * (lane >> 4), sum);
        }
}

// Product grouped by expert: tile shapes by A's format.  The grid covers the
// most row tiles that the rows can make among the experts (every expert's
// last one partly filled); workgroups past the last tile leave at once.
template <int BM, int BN, int WM, int WN, bool FP8, bool PERSIST = false>
static void launch_tile_grouped(const GroupedArgs &g, int64_t grid, hipStream_t s)
{
    const dim3 wgs((unsigned)grid), threads(64 * WM * WN);
    if (g.scale16)
        hipLaunchKernelGGL((mx_tile_grouped_kernel<BM, BN, WM, WN, true, FP8, PERSIST>), wgs, threads, 0, s, g);
    else
        hipLaunchKernelGGL((mx_tile_grouped_kernel<BM, BN, WM, WN, false, FP8, PERSIST>), wgs, threads, 0, s, g);
}

// The tiles, largest first, with the mean rows per expert from which each is
// taken (MI355X, 32 experts, N = 4096, K = 2048, routings as uneven as a softmax
// of normal logits, weights that the last-level cache does not hold; us, FP4 /
// FP8 A):
//   rows per expert   4            16           64           256          1024
//   32 x 128          28.3 / 30.2  35.8 / 37.3  52.3 / 55.3  132 / 141    404 / 445
//   64 x 128          29.1 / 32.0  37.5 / 36.4  45.3 / 53.2  92.3 / 119   283 / 390
//   128 x 128         31.8 / -     35.9 / -     47.3 / -     79.7 / -     247 / -
//   128 x 256         - / 37.5     - / 39.8     - / 56.0     - / 91.6     - / 288
//   256 x 256         38.4 / -     43.4 / -     54.0 / -     74.9 / -     195 / -
//   bytes / 5.1 TB/s  28           29           32           43 / 45      88 / 94
// The one taken is a column's fastest but for FP4 at 16 and 256 rows, 5 and 6 %
// slower here; with fewer experts or columns the larger tiles leave compute units
// idle.
const GroupedTileKernel *grouped_tile_kernels(int *count)
{
    static const GroupedTileKernel table[] = {
        {256, 256, {384, 0}, {launch_tile_grouped<256, 256, 2, 4, false>, nullptr}, {nullptr, nullptr}},
        {128, 256, {0, 96}, {nullptr, launch_tile_grouped<128, 256, 2, 4, true>},
         {nullptr, launch_tile_grouped<128, 256, 2, 4, true, true>}},
        {128, 128, {96, 0}, {launch_tile_grouped<128, 128, 2, 2, false>, nullptr}, {nullptr, nullptr}},
        {64, 128, {16, 12}, {launch_tile_grouped<64, 128, 2, 2, false>, launch_tile_grouped<64, 128, 2, 2, true>}, {nullptr, nullptr}},
        {32, 128, {0, 0}, {launch_tile_grouped<32, 128, 1, 4, false>, launch_tile_grouped<32, 128, 1, 4, true>}, {nullptr, nullptr}},
    };
    *count = (int)(sizeof(table) / sizeof(table[0]));
    return table;
}

}  // namespace mx
