// Attention of many rows per key head (chunks, whole prompts): the waves of a
// workgroup hold 32 rows each and share the keys, 64 (32 for wide heads) at a
// time, in LDS.  Bound by the matrix units and, beside them, the exponentials.
#pragma once

#include "mx_attn_plan.hpp"

namespace mx {

// Waves of a workgroup, keys of a stage and stages in LDS.  SMALL: half the rows
// and two workgroups on a compute unit, which fill each other's barriers and ends;
// the large shape reads keys and values half as often.  A prompt of 8192 tokens,
// 32 heads of 128 (550 GFLOP of the causal half): 541 to 634 us by the card, 0.87 to
// 1.0 PFLOP/s, where a large bf16 product of the library's reaches 1.2 to 1.3;
// counters: the matrix units busy 48 % of the cycles, the vector units 50 %.  On one
// SIMD the two overlap only in part (two waves of 32-cycle products with 8 vector
// instructions to each take 335 us where the products alone take 245 and the
// vector instructions 175), so that what is left is in the vector instructions of
// a score: multiply-add, exponential (8 cycles), maximum, sum, half a conversion.
template <int DP, bool SMALL>
struct RowsShape {
    static constexpr int NW = DP == 256 || SMALL ? 4 : 8;
    static constexpr int TM = NW * 32;                      // rows of a tile
    static constexpr int KT = DP == 256 || (SMALL && DP == 128) ? 32 : 64;  // keys of a stage
    static constexpr int STAGE = 2 * KT * DP * 2;
    static constexpr int ST = SMALL && DP == 64 ? 3 : 4;
    static constexpr int BYTES = ST * STAGE;
    static constexpr int PER_CU = SMALL && DP < 256 ? 2 : 1;
};

template <int DP, bool FP8, bool SMALL>
__global__ void __launch_bounds__((RowsShape<DP, SMALL>::NW * 64), (SMALL && DP < 256 ? 2 : 1)) mx_attn_rows_kernel(AttnArgs a, int mode)
{
    using L = AttnLds<DP, false>;  // in LDS the elements are bf16
    using SH = RowsShape<DP, SMALL>;
    constexpr int NW = SH::NW, TM = SH::TM, KT = SH::KT, ST = SH::ST, STAGE = SH::STAGE;
    constexpr int NB = KT / 32;
    constexpr int RW = KT / NW;               // rows of a stage that a wave loads: 8 or 16, within 16 keys
    constexpr int IPW = RW / L::RPI;          // its load instructions, of K and of V
    constexpr int PPW = RW * DP / 8 / 64;     // 8 bits: its pieces of 8 codes
    static_assert((RW == 8 || RW == 16) && IPW >= 1 && PPW >= 1, "a wave's rows of a stage");
    __shared__ __attribute__((aligned(1024))) uint8_t ring[SH::BYTES];
    __shared__ int s_last;
    __shared__ __attribute__((aligned(16))) uint8_t s_pages[NW][AttnPages::LDS];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const AttnFirst first_loads = attn_first(a, lane);

    // this lane's places in the cache's rows and in a stage
    uint32_t ko[FP8 ? PPW : IPW], vo[FP8 ? PPW : IPW], kw[FP8 ? PPW : 1], vw[FP8 ? PPW : 1];
    const int half = wave * RW % 16;  // its first row among 16 keys
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
    const uint32_t ka = L::k_first(lds_addr(ring), lane), va = L::v_first(lds_addr(ring) + KT * L::ROWB, lane);

    AttnTile plan;
    if (!attn_tiles(a, first_loads, TM, mode, blockIdx.x, gridDim.x, lane, plan))
        return;
    const int wg = plan.wg;
    int at = plan.at;
    while (at < plan.end) {
        int tile = seq_tiles(plan.q, a.group, TM) - 1 - plan.nth;  // the tiles with the most keys first
        int steps = tile_steps(a, plan.q, tile, TM, plan), cost = unit_steps(plan, steps);
        while (at >= plan.start + cost) {
            plan.start += cost;
            ++plan.nth;
            while (--tile < 0) {
                plan.nth = 0;
                if (++plan.head == a.c.kv_heads) {
                    if (++plan.s >= a.c.seqs)
                        return;
                    plan.q = load_seq(a.c, a.T, plan.s);
                    plan.head = 0;
                }
                tile = seq_tiles(plan.q, a.group, TM);
            }
            steps = tile_steps(a, plan.q, tile, TM, plan);
            cost = unit_steps(plan, steps);
        }
        const AttnSeq q = plan.q;
        const int head = plan.head, unit_start = plan.start;
        const int piece_end = min(plan.end, unit_start + cost);
        if (at >= unit_start + steps) {  // (its keys are other workgroups')
            at = piece_end;
            continue;
        }
        const int r0 = tile * TM, rows = min(q.n * a.group - r0, TM);
        int lo, hi;
        keys_of_tile(a, q, tile, TM, lo, hi);
        const KeyRange keys = step_keys(lo, hi, (at - unit_start), min(piece_end - unit_start, steps), plan.per);
        const int k0 = max(keys.lo, lo / KT * KT), k1 = keys.hi;
        const int nt = k1 > k0 ? key_blocks(k1 - k0, KT) : 0;  // stages

        const uint8_t *k_head = a.c.k + head * a.c.head_b, *v_head = a.c.v + head * a.c.head_b;
        const uint32_t my_key = (uint32_t)k0 + wave * RW / 16 * 16;  // the 16 keys that this wave's rows are among
        AttnPages table;
        if (nt > 0)
            table.open(a.c, plan.s, (int)(my_key >> a.c.page_shift), s_pages[wave], lane);
        v2u kr[PPW], vr[PPW];
        // loads of stage i: into LDS, or (8 bits) into registers
        auto issue = [&](int i) __attribute__((always_inline)) {
            const uint32_t key = my_key + i * KT;
            const int entry = (int)(key >> a.c.page_shift);
            int page, same;
            table.get(entry, entry, lane, page, same);
            const AttnRows x = attn_rows(a.c, k_head, v_head, page, key, i < nt ? q.len : key);
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
        const int row_lo = first_key(a, pos);
        // keys that every row of the wave sees, and that some see
        const int all_lo = a.window > 0 ? __builtin_amdgcn_readlane(row_lo, 31) : 0;
        const int all_hi = __builtin_amdgcn_readlane(row_hi, 0);
        const int any_lo = a.window > 0 ? __builtin_amdgcn_readlane(row_lo, 0) : 0;
        const int any_hi = wrows > 0 ? __builtin_amdgcn_readlane(row_hi, 31) : 0;
        v4i qf[L::NS];
        load_q<DP, false>(a, a.Q + (int64_t)(q.t0 + idx) * a.ldq + my.head * a.c.D,
                          row < wrows && !sc.zero, lane, qf);
        negate_q(qf, sc.negate);
        // Blocks of 32 keys, counted from k0: [s0, s1) are seen by some row of the
        // wave, [f0, f1) by all of them
        const int blocks = nt * NB;
        const int s0 = max(any_lo - k0, 0) / 32, s1 = min(((any_hi - k0 - 1) >> 5) + 1, blocks);
        const int f0 = (max(all_lo - k0, 0) + 31) / 32, f1 = min((all_hi - k0) >> 5, s1);
        v16f x;  // scores of the block whose exponentials are next
        auto slot = [&](int c) { return (uint32_t)((c / NB % ST) * STAGE + c % NB * L::BLOCK); };
        if (nt > 0) {
            constexpr int AHEAD = ST - 2;
            // Barrier i: stage i is there, and everyone is done with stage i - 2,
            // whose slot stage i + AHEAD takes.  (Every wave passes every barrier
            // once; where in its work is its own affair.)
            int synced = 0;
            auto sync = [&] __attribute__((always_inline)) {
                if constexpr (FP8) {
                    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
                    put(synced + 1);
                    issue(synced + 2);
                } else {
                    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((AHEAD - 1) * 2 * IPW) : "memory");
                    issue(synced + AHEAD);
                }
                ++synced;
            };
            // Stages whose blocks, and the one before, are seen by all rows: for
            // each block c its scores beside the exponentials of block c - 1, then
            // that block's values beside the maximum of c.  Both products come in
            // groups of two matrix instructions (64 cycles); the groups' fragments
            // are read LA groups before (an LDS read takes 130 cycles and more with
            // eight waves reading), over the stages' borders too, and behind each
            // group stands a piece of the other work: a wave issues one instruction
            // in 4 cycles, so what is put there runs while the matrix unit works.
            auto hot = [&](int i0, int i1) __attribute__((always_inline)) {
                constexpr int LA = 3, R = LA + 1;
                constexpr int NK = L::NS / 2, NV = L::ND, NI = NK + NV;  // groups of a block: scores, values
                constexpr int T = NB * NI;
                constexpr bool WRAP = NB > 1;
                static_assert(T % R == 0, "fragments by group");
                v4i fk[R][2];
                v2u fv[R][2][2];
                auto read = [&](auto nc, int i) __attribute__((always_inline)) {
                    constexpr int N = nc.value % T, B = N / NI, G = N % NI, F = N % R;
                    const int c = (i + nc.value / T) * NB + B;
                    if constexpr (G < NK) {
                        const uint32_t at = ka + slot(c);
                        fk[F][0] = lds_read16<0>(L::k_at(at, 2 * G));
                        fk[F][1] = lds_read16<0>(L::k_at(at, 2 * G + 1));
                    } else {
                        constexpr int S = (G - NK) / (L::ND / 2), D0 = (G - NK) % (L::ND / 2) * 2;
                        const uint32_t at = va + slot(c - 1);
#pragma unroll
                        for (int d = 0; d < 2; ++d) {
                            fv[F][d][0] = lds_read_tr16<S * 16 * L::ROWB>(L::v_at(at, D0 + d));
                            fv[F][d][1] = lds_read_tr16<(S * 16 + 8) * L::ROWB>(L::v_at(at, D0 + d));
                        }
                    }
                };
                // reads of the groups behind group n that are under way with it
                auto later = [](int n) constexpr {
                    int r = 0;
                    for (int k = n + 1; k <= n + LA; ++k)
                        if (WRAP || k < T)
                            r += k % T % NI < NK ? 2 : 4;
                    return r;
                };
                auto start = [&](int i) __attribute__((always_inline)) {
                    static_for<LA>([&](auto nc) { read(nc, i); });
                };
                if (synced <= i0)
                    sync();
                if constexpr (WRAP)
                    start(i0);
                v4i p[2];
                v16f acc;
                float less, most;
                for (int i = i0; i < i1; ++i) {
                    if constexpr (!WRAP) {
                        if (synced <= i)
                            sync();
                        start(i);
                    }
                    static_for<T>([&](auto nc) {
                        constexpr int N = nc.value, B = N / NI, G = N % NI, F = N % R;
                        if constexpr (WRAP || N + LA < T)
                            read(std::integral_constant<int, N + LA>{}, i);
                        if constexpr (G < NK) {
                            lds_wait_n<later(N)>(fk[F]);
                            if constexpr (G == 0) {
                                acc = v16f{};
                                less = less_max(t.m);
                            }
                            acc = mfma32(fk[F][0], qf[2 * G], acc);
                            acc = mfma32(fk[F][1], qf[2 * G + 1], acc);
                            constexpr int EACH = (8 + NK - 2) / (NK - 1);  // (pairs; none behind the last group: x is free there)
#pragma unroll
                            for (int n = G * EACH; n < (G + 1) * EACH && n < 8; ++n)
                                exponential_pair(t, x, n, sc.c, less, p);
                            if constexpr (G == NK - 1)
                                x = acc;
                        } else {
                            constexpr int I = G - NK, S = I / (L::ND / 2), D0 = I % (L::ND / 2) * 2, MAX = 16 / NV;
                            lds_wait_n<later(N)>(fv[F]);
#pragma unroll
                            for (int d = 0; d < 2; ++d) {
                                const v2u (&w)[2] = fv[F][d];
                                t.o[D0 + d] = mfma32(v4i{(int)w[0][0], (int)w[0][1], (int)w[1][0], (int)w[1][1]}, p[S], t.o[D0 + d]);
                            }
                            if constexpr (I == 0)
                                most = x[0];
#pragma unroll
                            for (int n = I * MAX; n < (I + 1) * MAX; ++n)
                                most = fmaxf(most, x[n]);
                            if constexpr (I == NV - 1)
                                raise_to(t, most, sc.c);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                        // (the values of stage i - 1 are read: barrier i + 1 may come)
                        if constexpr (WRAP && N == NI - 1)
                            sync();
                    });
                }
                lds_wait_n<0>(fk, fv);
            };
            if constexpr (FP8) {
                issue(0);
                put(0);
                issue(1);
            } else {
#pragma unroll
                for (int i = 0; i < AHEAD; ++i)
                    issue(i);
            }
            const int hot0 = f0 / NB + 1, hot1 = f1 / NB;
            for (int i = 0; i <= nt; ++i) {
                if (i >= hot0 && i < hot1) {
                    hot(i, hot1);
                    i = hot1;
                }
                if (synced <= i)
                    sync();
#pragma unroll 1
                for (int c = i * NB; c < (i + 1) * NB; ++c) {
                    if (c - 1 >= s0 && c - 1 < s1) {
                        v4i p[1][2];
                        exponentials(t, x, sc.c, p[0]);
                        const int lo_c[1] = {row_lo - (k0 + (c - 1) * 32)}, hi_c[1] = {row_hi - (k0 + (c - 1) * 32)};
                        values<DP, false, 1>(va + slot(c - 1), p, ts, c - 1 < f0 || c - 1 >= f1, lo_c, hi_c, lane);
                    }
                    if (c >= s0 && c < s1) {
                        x = scores_one<DP>(ka + slot(c), qf);
                        if (c < f0 || c >= f1)
                            mask_scores(x, row_lo - (k0 + c * 32), row_hi - (k0 + c * 32), lane);
                        raise_max(t, x, sc.c);
                    }
                }
            }
        }
        attn_wait_vm<0>();
        const AttnArgs end_args = args_again();
        const int end_lane = anew(lane);
        t.l = row_sum(t.l);
        __syncthreads();  // the ring is free
        const int first = unit_start / plan.chunk, last = (unit_start + steps - 1) / plan.chunk;  // its workgroups
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
                        store16_coherent(to, (uint32_t)(((d * 4 + (g >> 2)) * 64 + end_lane) * 16),
                                         v4f{t.o[d][g], t.o[d][g + 1], t.o[d][g + 2], t.o[d][g + 3]});
                __builtin_amdgcn_raw_buffer_store_b64(v2u{__float_as_uint(t.m), __float_as_uint(t.l)}, to,
                                                      (uint32_t)(L::ND * 16 * 256 + end_lane * 8), 0, kCoherent);
            }
            done = split_arrive_last_via(end_args.counters + first, last - first + 1, &s_last);
            if (done && wrows > 0) {
                const int off = unit_start > first * plan.chunk ? 1 : 0;
                const int parts = last - first + 1;
                auto part = [&](int w) __attribute__((always_inline)) {
                    return make_rsrc_u(end_args.partials + (2 * (int64_t)(first + w) + (w == 0 ? off : 0)) * (NW * PW) + wave * PW, PW * 4);
                };
                auto m_and_l = [&](int w) __attribute__((always_inline)) {
                    return __builtin_amdgcn_raw_buffer_load_b64(part(w), (uint32_t)(L::ND * 16 * 256 + end_lane * 8), 0, kCoherent);
                };
                // first what the parts' maxima and sums come to, then O by 32
                // columns: PB parts in flight (one after another 64 parts took 300 us)
                constexpr int PB = 2;
                float m = kNegInf;
                t.l = 0.0f;
                for (int w0 = 0; w0 < parts; w0 += PB) {
                    v2u ml[PB];
#pragma unroll
                    for (int i = 0; i < PB; ++i)
                        ml[i] = m_and_l(min(w0 + i, parts - 1));
#pragma unroll
                    for (int i = 0; i < PB; ++i)
                        if (w0 + i < parts) {
                            const float mw = __uint_as_float(ml[i][0]), n = fmaxf(m, mw);
                            const float f0 = n == kNegInf ? 1.0f : exp2_fast(m - n), f1 = n == kNegInf ? 1.0f : exp2_fast(mw - n);
                            m = n;
                            t.l = t.l * f0 + __uint_as_float(ml[i][1]) * f1;
                        }
                }
                t.m = m;
#pragma unroll
                for (int d = 0; d < L::ND; ++d) {
                    t.o[d] = v16f{};
#pragma unroll 1
                    for (int w0 = 0; w0 < parts; w0 += PB) {
                        v2u ml[PB];
                        v4f y[PB][4];
#pragma unroll
                        for (int i = 0; i < PB; ++i)
                            if (w0 + i < parts) {
                                ml[i] = m_and_l(w0 + i);
#pragma unroll
                                for (int g = 0; g < 4; ++g)
                                    y[i][g] = load16_coherent(part(w0 + i), (uint32_t)(((d * 4 + g) * 64 + end_lane) * 16));
                            }
#pragma unroll
                        for (int i = 0; i < PB; ++i)
                            if (w0 + i < parts) {
                                const float f = m == kNegInf ? 1.0f : exp2_fast(__uint_as_float(ml[i][0]) - m);
#pragma unroll
                                for (int g = 0; g < 16; ++g)
                                    t.o[d][g] = fmaf(y[i][g >> 2][g & 3], f, t.o[d][g]);
                            }
                    }
                }
            }
        }
        if (done && wrows > 0)
            finish_tile<DP>(end_args, q, head, w0, wrows, t.m, t.l, t.o, ring + wave * (32 * DP * 2), end_lane);
        __syncthreads();  // the ring is free again
        at = piece_end;
    }
}

template <int DP, bool SMALL>
AttnRowsKernel rows_entry(bool fp8)
{
    using SH = RowsShape<DP, SMALL>;
    auto bf16 = [](const AttnArgs &a, int plan, int grid, hipStream_t s) {
        mx_attn_rows_kernel<DP, false, SMALL><<<grid, SH::NW * 64, 0, s>>>(a, plan);
    };
    auto f8 = [](const AttnArgs &a, int plan, int grid, hipStream_t s) {
        mx_attn_rows_kernel<DP, true, SMALL><<<grid, SH::NW * 64, 0, s>>>(a, plan);
    };
    return {SH::TM, SH::PER_CU, fp8 ? (AttnLaunchFn)f8 : (AttnLaunchFn)bf16};
}

}  // namespace mx
