// Attention of many rows per key head (chunks, whole prompts): the waves of a
// workgroup hold 32 rows each and share the keys, 64 (32 for wide heads) at a
// time, in LDS.  Bound by the matrix units and, beside them, the exponentials.
#include "mx_attn_plan.hpp"

namespace mx {

namespace {

template <int DP>
struct RowsShape {
    static constexpr int NW = DP == 256 ? 4 : 8;
    static constexpr int TM = NW * 32;           // rows of a tile
    static constexpr int KT = DP == 256 ? 32 : 64;  // keys of a stage
    static constexpr int STAGE = 2 * KT * DP * 2;
    static constexpr int ST = 4;
    static constexpr int BYTES = ST * STAGE;
};

template <int DP, bool FP8>
__global__ void __launch_bounds__((RowsShape<DP>::NW * 64)) mx_attn_rows_kernel(AttnArgs a, int mode)
{
    using L = AttnLds<DP, false>;  // in LDS the elements are bf16
    using SH = RowsShape<DP>;
    constexpr int NW = SH::NW, TM = SH::TM, KT = SH::KT, ST = SH::ST, STAGE = SH::STAGE;
    constexpr int NB = KT / 32;
    constexpr int RW = KT / NW;               // rows of a stage that a wave loads: 8, within 16 keys
    constexpr int IPW = RW / L::RPI;          // its load instructions, of K and of V
    constexpr int PPW = RW * DP / 8 / 64;     // 8 bits: its pieces of 8 codes
    static_assert(RW == 8 && IPW >= 1, "a wave's rows of a stage");
    __shared__ __attribute__((aligned(1024))) uint8_t ring[SH::BYTES];
    __shared__ int s_last;

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wg = blockIdx.x;
    const AttnFirst first_loads = attn_first(a, lane);

    // this lane's places in the cache's rows and in a stage
    uint32_t ko[FP8 ? PPW : IPW], vo[FP8 ? PPW : IPW], kw[FP8 ? PPW : 1], vw[FP8 ? PPW : 1];
    const int half = (wave & 1) * 8;  // its first row among 16 keys
    if constexpr (FP8) {
#pragma unroll
        for (int i = 0; i < PPW; ++i) {
            const int r = (i * 64 + lane) / (DP / 8), c = lane % (DP / 8);
            ko[i] = vo[i] = c * 8 < a.c.D ? (uint32_t)((half + r) * a.c.token_b + c * 8) : kOOB;
            kw[i] = (wave * RW + r) * L::ROWB + L::k_chunk(half + r, c) * 16;
            vw[i] = KT * L::ROWB + (wave * RW + r) * L::ROWB + L::v_chunk(half + r, c) * 16;
        }
    } else {
#pragma unroll
        for (int j = 0; j < IPW; ++j) {
            const int r = half + j * L::RPI + lane / L::CH, c = lane % L::CH;
            const int kc = L::k_chunk(r, c) * 16, vc = L::v_chunk(r, c) * 16;
            ko[j] = kc < 2 * a.c.D ? (uint32_t)(r * a.c.token_b + kc) : kOOB;
            vo[j] = vc < 2 * a.c.D ? (uint32_t)(r * a.c.token_b + vc) : kOOB;
        }
    }
    uint32_t ka[L::KF], va[L::ND];
    L::k_addr(lds_addr(ring), lane, ka);
    L::v_addr(lds_addr(ring) + KT * L::ROWB, lane, va);

    AttnPlan plan;
    if (!attn_plan(a, first_loads, TM, mode, wg, gridDim.x, lane, plan))
        return;
    int at = wg * plan.chunk;
    const int end = min(at + plan.chunk, plan.total);
    int s = plan.s, seq_start = plan.start;
    AttnSeq q = plan.q;
    int cost = seq_steps(a, q, TM, plan.per), units = seq_units(a, q, TM);
    while (at < end) {
        while (at >= seq_start + units * cost) {
            seq_start += units * cost;
            if (++s >= a.c.seqs)
                return;
            q = load_seq(a.c, a.T, s);
            cost = seq_steps(a, q, TM, plan.per);
            units = seq_units(a, q, TM);
        }
        const int u = (at - seq_start) / cost, unit_start = seq_start + u * cost;
        // the tiles with the most keys first
        const int nth = quotient(u, a.by_kv_heads), head = u - nth * a.c.kv_heads;
        const int tile = seq_tiles(q, a.group, TM) - 1 - nth;
        const int piece_end = min(end, unit_start + cost);
        const int r0 = tile * TM, rows = min(q.n * a.group - r0, TM);
        int lo, hi;
        tile_keys(a, q, quotient(r0, a.by_group), quotient(r0 + rows - 1, a.by_group), lo, hi);
        const KeyRange keys = step_keys(lo, hi, (at - unit_start), (piece_end - unit_start), plan.per);
        const int k0 = max(keys.lo, lo / KT * KT), k1 = keys.hi;
        const int nt = max((k1 - k0 + KT - 1) / KT, 0);  // stages

        const uint8_t *k_head = a.c.k + head * a.c.head_b, *v_head = a.c.v + head * a.c.head_b;
        const int my_key = k0 + (wave >> 1) * 16;  // the 16 keys that this wave's rows are among
        AttnPages table;
        table.open(a.c, s, my_key >> a.c.page_shift, lane);
        v2u kr[PPW], vr[PPW];
        // loads of stage i: into LDS, or (8 bits) into registers
        auto issue = [&](int i) __attribute__((always_inline)) {
            const int key = my_key + i * KT;
            const AttnRows x = attn_rows(a.c, k_head, v_head, table.page(key >> a.c.page_shift, lane), key, i < nt ? q.len : 0);
            if constexpr (FP8) {
#pragma unroll
                for (int j = 0; j < PPW; ++j) {
                    kr[j] = load8(x.k, ko[j]);
                    vr[j] = load8(x.v, vo[j]);
                }
            } else {
                uint8_t *to = ring + (i % ST) * STAGE + wave * RW * L::ROWB;
#pragma unroll
                for (int j = 0; j < IPW; ++j) {
                    load16_to_lds(x.k, (lds_void *)(to + j * 1024), ko[j]);
                    load16_to_lds(x.v, (lds_void *)(to + KT * L::ROWB + j * 1024), vo[j]);
                }
            }
        };
        auto put = [&](int i) __attribute__((always_inline)) {
            if constexpr (FP8) {
                uint8_t *to = ring + (i % ST) * STAGE;
#pragma unroll
                for (int j = 0; j < PPW; ++j) {
                    *reinterpret_cast<v4i *>(to + kw[j]) = bf16_of_fp8(kr[j]);
                    *reinterpret_cast<v4i *>(to + vw[j]) = bf16_of_fp8(vr[j]);
                }
            }
        };

        AttnState<L::ND> ts[1];
        AttnState<L::ND> &t = ts[0];
        t.reset();
        const AttnScale sc = attn_scale(a, head);
        const int w0 = r0 + wave * 32, wrows = min(max(rows - wave * 32, 0), 32);  // this wave's rows
        const int row = lane & 31;
        const int rr = w0 + min(row, max(wrows - 1, 0));
        const AttnRow my = attn_row(a, rr, head);
        const int idx = my.token, pos = q.len - q.n + idx;
        const int row_hi = a.causal ? min(pos + 1, q.len) : (pos < 0 ? 0 : q.len);
        const int row_lo = a.window > 0 ? pos - a.window + 1 : 0;
        // keys that every row of the wave sees, and that some see
        const int all_lo = a.window > 0 ? __builtin_amdgcn_readlane(row_lo, 31) : 0;
        const int all_hi = __builtin_amdgcn_readlane(row_hi, 0);
        const int any_lo = a.window > 0 ? __builtin_amdgcn_readlane(row_lo, 0) : 0;
        const int any_hi = wrows > 0 ? __builtin_amdgcn_readlane(row_hi, 31) : 0;
        v4i qf[1][L::NS];
        load_q<DP, false>(a, a.Q + (int64_t)(q.t0 + idx) * a.ldq + my.head * a.c.D,
                          row < wrows && !sc.zero, lane, qf[0]);
        negate_q(qf[0], sc.negate);
        if (nt > 0) {
            constexpr int AHEAD = ST - 1;
            if constexpr (FP8) {
                issue(0);
                put(0);
                issue(1);
            } else {
#pragma unroll
                for (int i = 0; i < AHEAD; ++i)
                    issue(i);
            }
            for (int i = 0; i < nt; ++i) {
                // stage i is there, and everyone is done with stage i - 1
                if constexpr (FP8)
                    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
                else
                    stage_sync<(AHEAD - 1) * 2 * IPW>();
                if constexpr (FP8) {
                    put(i + 1);
                    issue(i + 2);
                } else {
                    issue(i + AHEAD);
                }
                const uint32_t slot = (uint32_t)((i % ST) * STAGE);
                const int key = k0 + i * KT;
                if (key >= any_hi || key + KT <= any_lo)
                    continue;
                v16f x[NB];
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    v16f y[1];
                    scores<DP, false, 1>(ka, slot + b * L::BLOCK, qf, y);
                    x[b] = y[0];
                }
                const bool masked = key < all_lo || key + KT > all_hi;
                if (masked)
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        mask_scores(x[b], row_lo - key - 32 * b, row_hi - key - 32 * b, lane);
                v4i p[NB][2];
                softmax_blocks(t, x, sc.c, p);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const v4i pb[1][2] = {{p[b][0], p[b][1]}};
                    const int bl[1] = {row_lo - key - 32 * b}, bh[1] = {row_hi - key - 32 * b};
                    values<DP, false, 1>(va, slot + b * L::BLOCK, pb, ts, masked, bl, bh, lane);
                }
            }
        }
        attn_wait_vm<0>();
        const AttnArgs end_args = args_again();
        t.l = row_sum(t.l);
        __syncthreads();  // the ring is free
        const int first = unit_start / plan.chunk, last = (unit_start + cost - 1) / plan.chunk;
        bool done = first == last;
        if (!done) {
            // a partial result: a wave's registers as they are
            constexpr int64_t PW = 64 * (L::ND * 16 + 2);  // floats of a wave
            const __amdgpu_buffer_rsrc_t to =
                make_rsrc_u(end_args.partials + (2 * (int64_t)wg + (unit_start > wg * plan.chunk ? 1 : 0)) * (NW * PW) + wave * PW, PW * 4);
            if (wrows > 0) {
#pragma unroll
                for (int d = 0; d < L::ND; ++d)
#pragma unroll
                    for (int g = 0; g < 16; g += 4)
                        store16_coherent(to, (uint32_t)(((d * 4 + (g >> 2)) * 64 + lane) * 16),
                                         v4f{t.o[d][g], t.o[d][g + 1], t.o[d][g + 2], t.o[d][g + 3]});
                __builtin_amdgcn_raw_buffer_store_b64(v2u{__float_as_uint(t.m), __float_as_uint(t.l)}, to,
                                                      (uint32_t)(L::ND * 16 * 256 + lane * 8), 0, kCoherent);
            }
            done = split_arrive_last_via(end_args.counters + first, last - first + 1, &s_last);
            if (done && wrows > 0) {
                const int off = unit_start > first * plan.chunk ? 1 : 0;
                t.reset();
                for (int w = 0; w <= last - first; ++w) {
                    const __amdgpu_buffer_rsrc_t from = make_rsrc_u(
                        end_args.partials + (2 * (int64_t)(first + w) + (w == 0 ? off : 0)) * (NW * PW) + wave * PW, PW * 4);
                    const v2u ml = __builtin_amdgcn_raw_buffer_load_b64(from, (uint32_t)(L::ND * 16 * 256 + lane * 8), 0, kCoherent);
                    const float mw = __uint_as_float(ml[0]), n = fmaxf(t.m, mw);
                    const float f0 = n == kNegInf ? 1.0f : exp2_fast(t.m - n), f1 = n == kNegInf ? 1.0f : exp2_fast(mw - n);
                    t.m = n;
                    t.l = t.l * f0 + __uint_as_float(ml[1]) * f1;
#pragma unroll
                    for (int d = 0; d < L::ND; ++d)
#pragma unroll
                        for (int g = 0; g < 16; g += 4) {
                            const v4f x = load16_coherent(from, (uint32_t)(((d * 4 + (g >> 2)) * 64 + lane) * 16));
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                t.o[d][g + e] = t.o[d][g + e] * f0 + x[e] * f1;
                        }
                }
            }
        }
        if (done && wrows > 0)
            finish_tile<DP>(end_args, q, head, w0, wrows, t.m, t.l, t.o, ring + wave * (32 * DP * 2), lane);
        __syncthreads();  // the ring is free again
        at = piece_end;
    }
}

int padded(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

template <int DP>
void launch(const AttnArgs &a, bool fp8, int plan, int grid, hipStream_t s)
{
    if (fp8)
        mx_attn_rows_kernel<DP, true><<<grid, RowsShape<DP>::NW * 64, 0, s>>>(a, plan);
    else
        mx_attn_rows_kernel<DP, false><<<grid, RowsShape<DP>::NW * 64, 0, s>>>(a, plan);
}

}  // namespace

int attn_rows_tile(int D) { return padded(D) == 256 ? RowsShape<256>::TM : RowsShape<128>::TM; }
int attn_rows_per_cu(int) { return 1; }

void launch_attn_rows(const AttnArgs &a, bool fp8, int plan, int grid, hipStream_t s)
{
    switch (padded(a.c.D)) {
    case 64: return launch<64>(a, fp8, plan, grid, s);
    case 128: return launch<128>(a, fp8, plan, grid, s);
    default: return launch<256>(a, fp8, plan, grid, s);
    }
}

}  // namespace mx
