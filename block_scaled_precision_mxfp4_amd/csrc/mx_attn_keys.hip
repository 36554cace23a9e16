// Attention of few rows per key head (decode, short chunks): the waves of a
// workgroup share a tile of 32 or 64 rows and take its keys 32 at a time in turn,
// so that a long context is spread over every wave of the card.  Bound by HBM:
// every key and value is read once a tile.  64 tokens over 8192 keys, 8 key heads
// of 128 in bf16: 213 us, 6.3 TB/s (a large copy: 4.7); 16 over 4096, heads of 256:
// 35 us, 4.8 TB/s.  One token over 4096 (16.8 MB) takes 12 us, mostly one after
// another: plan and page ids 1.3, first keys, 2 blocks a wave, parts, their sum.
// 8 x 5 tokens over 16384 in 8 bits, 8 query heads a key head: 36 us, 2.4 TB/s:
// its units are cut into parts, one workgroup a compute unit, so that a SIMD has
// one wave of 64 rows, whose products and exponentials do not overlap.
//
// Each wave has a ring of its own in LDS, filled by direct-to-LDS loads of
// whole rows (page ids come by LDS as well, a page's descriptor ends with the
// sequence), and waits for nothing but its own loads: no barrier until the
// waves' results are merged.  The rings hold up to 128 KiB of a compute
// unit's loads in flight (8 TB/s for about 2 us need 60 KiB).
#include "mx_attn_plan.hpp"

namespace mx {

namespace {

// waves of a workgroup and slots of a wave's ring: the most that fit 128 KiB
// (64 KiB where two workgroups then share a compute unit)
template <int DP, bool FP8, int NT>
struct KeysShape {
    static constexpr int STAGE = 2 * AttnLds<DP, FP8>::BLOCK;
    static constexpr int NW = STAGE > 16384 ? 2 : 4;
    static constexpr int ST = STAGE > 8192 || (STAGE > 4096 && NT == 1) ? 2 : 4;
    static constexpr int BYTES = NW * ST * STAGE;
    static constexpr int PER_CU = BYTES <= 65536 ? 2 : 1;
};

template <int DP, bool FP8, int NT>
__global__ void __launch_bounds__((KeysShape<DP, FP8, NT>::NW * 64)) mx_attn_keys_kernel(AttnArgs a, int mode)
{
    using L = AttnLds<DP, FP8>;
    using SH = KeysShape<DP, FP8, NT>;
    constexpr int NW = SH::NW, ST = SH::ST, STAGE = SH::STAGE;
    constexpr int NI = 2 * L::NIH;        // load instructions of a block of K, or of V
    constexpr int QC = DP / 8;            // 8-column pieces of a row
    constexpr int TM = NT * kAttnTile;    // rows of a tile
    static_assert(TM * DP * 4 <= ST * STAGE, "a wave's ring holds its rows of O");
    __shared__ __attribute__((aligned(1024))) uint8_t ring[SH::BYTES];
    __shared__ float s_ml[NW][TM][2];
    __shared__ int s_last;
    __shared__ __attribute__((aligned(16))) uint8_t s_pages[NW][AttnPages::LDS];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wg = blockIdx.x;
    const AttnFirst first_loads = attn_first(a, lane);

    uint32_t ko[L::NIH], vo[L::NIH];
    L::load_offsets(a.c, lane, ko, vo);
    uint8_t *mine = ring + wave * (ST * STAGE);
    const uint32_t ka = L::k_first(lds_addr(mine), lane), va = L::v_first(lds_addr(mine) + L::BLOCK, lane);

    AttnPlan plan;
    if (!attn_plan(a, first_loads, TM, 1, mode, wg, gridDim.x, lane, plan))
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
        const int tile = quotient(u, a.by_kv_heads), head = u - tile * a.c.kv_heads;
        const int piece_end = min(end, unit_start + cost);
        // its rows, and the keys that they see
        const int r0 = tile * TM, rows = min(q.n * a.group - r0, TM);
        int lo, hi;
        tile_keys(a, q, quotient(r0, a.by_group), quotient(r0 + rows - 1, a.by_group), lo, hi);
        const KeyRange keys = step_keys(lo, hi, (at - unit_start), (piece_end - unit_start), plan.per);
        const int b0 = max(keys.lo, lo) / 32, b1 = keys.lo < keys.hi ? key_blocks(keys.hi, 32) : b0;  // (a step behind the last key: none)
        const int nb = max((b1 - b0 - wave + NW - 1) / NW, 0);  // this wave's blocks: b0 + wave, + NW, ...

        const uint8_t *k_head = a.c.k + head * a.c.head_b, *v_head = a.c.v + head * a.c.head_b;
        AttnPages table;
        auto issue = [&](int i) __attribute__((always_inline)) {
            const uint32_t key0 = (uint32_t)(b0 + wave + i * NW) * 32, len = i < nb ? q.len : key0;
            int pg0, pg1;
            table.get((int)(key0 >> a.c.page_shift), (int)((key0 + 16) >> a.c.page_shift), lane, pg0, pg1);
            const AttnRows x = attn_rows(a.c, k_head, v_head, pg0, key0, len);
            const AttnRows y = attn_rows(a.c, k_head, v_head, pg1, key0 + 16, len);
            uint8_t *to = mine + (i % ST) * STAGE;
#pragma unroll
            for (int j = 0; j < L::NIH; ++j)
                load16_to_lds_stream(x.k, (lds_void *)(to + j * 1024), ko[j]);
#pragma unroll
            for (int j = 0; j < L::NIH; ++j)
                load16_to_lds_stream(y.k, (lds_void *)(to + L::BLOCK / 2 + j * 1024), ko[j]);
#pragma unroll
            for (int j = 0; j < L::NIH; ++j)
                load16_to_lds_stream(x.v, (lds_void *)(to + L::BLOCK + j * 1024), vo[j]);
#pragma unroll
            for (int j = 0; j < L::NIH; ++j)
                load16_to_lds_stream(y.v, (lds_void *)(to + L::BLOCK + L::BLOCK / 2 + j * 1024), vo[j]);
        };

        AttnState<L::ND> t[NT];
        const AttnScale sc = attn_scale(a, head);
        const int row = lane & 31;
        AttnRow my[NT];  // this lane's row of each 32, and the keys that it sees
        int row_lo[NT], row_hi[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            t[n].reset();
            my[n] = attn_row(a, r0 + min(n * 32 + row, rows - 1), head);
            const int pos = q.len - q.n + my[n].token;
            row_hi[n] = a.causal ? min(pos + 1, q.len) : (pos < 0 ? 0 : q.len);
            row_lo[n] = first_key(a, pos);
        }
        if (nb > 0) {
            table.open(a.c, s, ((b0 + wave) * 32) >> a.c.page_shift, s_pages[wave], lane);
            v4i qf[NT][L::NS];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                load_q<DP, FP8>(a, a.Q + (int64_t)(q.t0 + my[n].token) * a.ldq + my[n].head * a.c.D, n * 32 + row < rows && !sc.zero, lane, qf[n]);
            }
#pragma unroll
            for (int i = 0; i < ST - 1; ++i)
                issue(i);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                negate_q(qf[n], sc.negate);
            // keys that every row of the tile sees
            const int all_lo = a.window > 0 ? __builtin_amdgcn_readlane(row_lo[NT - 1], 31) : 0;
            const int all_hi = __builtin_amdgcn_readlane(row_hi[0], 0);
            for (int i = 0; i < nb; ++i) {
                issue(i + ST - 1);
                const uint32_t slot = (uint32_t)((i % ST) * STAGE);
                const int key0 = (b0 + wave + i * NW) * 32;
                attn_wait_vm<NI + (ST - 1) * 2 * NI>();
                v16f x[NT];
                scores<DP, FP8, NT>(ka + slot, qf, x);
                const bool masked = key0 < all_lo || all_hi - key0 < 32;
                int lo_b[NT], hi_b[NT];
                v4i p[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    lo_b[n] = row_lo[n] - key0;
                    hi_b[n] = row_hi[n] - key0;
                    if (masked)
                        mask_scores(x[n], lo_b[n], hi_b[n], lane);
                    raise_max(t[n], x[n], sc.c);
                    exponentials(t[n], x[n], sc.c, p[n]);
                }
                attn_wait_vm<(ST - 1) * 2 * NI>();
                values<DP, FP8, NT>(va + slot, p, t, masked, lo_b, hi_b, lane);
            }
        }
        // merge the waves: O to the wave's ring, rows of DP floats whose
        // 16-byte chunks are swizzled by the row
        attn_wait_vm<0>();
        const AttnArgs e = args_again();
        const int end_thread = anew(threadIdx.x), end_lane = end_thread & 63;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = n * 32 + (end_lane & 31);
            t[n].l = row_sum(t[n].l);
            if (r < rows) {
                float *o = reinterpret_cast<float *>(mine) + r * DP;
#pragma unroll
                for (int d = 0; d < L::ND; ++d)
#pragma unroll
                    for (int g = 0; g < 16; g += 4) {
                        const int ch = d * 8 + (g >> 2) * 2 + (end_lane >> 5);
                        *reinterpret_cast<v4f *>(o + ((ch ^ (r & 15)) * 4)) =
                            v4f{t[n].o[d][g], t[n].o[d][g + 1], t[n].o[d][g + 2], t[n].o[d][g + 3]};
                    }
                if (end_lane < 32) {
                    s_ml[wave][r][0] = t[n].m;
                    s_ml[wave][r][1] = t[n].l;
                }
            }
        }
        __syncthreads();
        // the unit's workgroups (at most one unit that goes on behind a workgroup
        // starts in it: its counter is that workgroup's), and this one's place for
        // a partial result
        const int first = unit_start / plan.chunk, last = (unit_start + cost - 1) / plan.chunk;
        constexpr int FLOATS = TM * (DP + 2);
        const __amdgpu_buffer_rsrc_t part = make_rsrc_u(
            e.partials + (2 * (int64_t)wg + (unit_start > wg * plan.chunk ? 1 : 0)) * FLOATS, FLOATS * 4);
        auto finish_unit_row = [&](int r, int c8, float m, float l, const float (&o)[8], bool live) __attribute__((always_inline)) {
            const AttnRow to = attn_row(e, r0 + r, head);
            finish_row(e, head, q.t0 + to.token, to.head, c8 * 8, m, l, [&](int i) { return o[i]; }, live);
        };
        // what the waves have in LDS, added up: the result, or this workgroup's part of it
        auto merge = [&](bool result) __attribute__((always_inline)) {
            for (int it = end_thread; it < ((rows * QC + 63) & ~63); it += NW * 64) {
                const int r = it / QC, c8 = it % QC;
                const bool live = r < rows && c8 * 8 < e.c.D;
                const int rr = min(r, rows - 1);
                float m = kNegInf, l = 0.0f, o[8] = {};
#pragma unroll
                for (int w = 0; w < NW; ++w)
                    m = fmaxf(m, s_ml[w][rr][0]);
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    const float f = m == kNegInf ? 1.0f : exp2_fast(s_ml[w][rr][0] - m);
                    l += f * s_ml[w][rr][1];
                    const float *src = reinterpret_cast<const float *>(ring + w * (ST * STAGE)) + rr * DP;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const v4f x = *reinterpret_cast<const v4f *>(src + (((2 * c8 + h) ^ (rr & 15)) * 4));
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            o[4 * h + i] += f * x[i];
                    }
                }
                if (result) {
                    finish_unit_row(rr, c8, m, l, o, live);
                } else if (live) {
                    store16_coherent(part, (uint32_t)((r * DP + c8 * 8) * 4), v4f{o[0], o[1], o[2], o[3]});
                    store16_coherent(part, (uint32_t)((r * DP + c8 * 8 + 4) * 4), v4f{o[4], o[5], o[6], o[7]});
                    if (c8 == 0)
                        __builtin_amdgcn_raw_buffer_store_b64(v2u{__float_as_uint(m), __float_as_uint(l)}, part,
                                                              (uint32_t)((TM * DP + 2 * r) * 4), 0, kCoherent);
                }
            }
        };
        bool done = first == last;
        if (!done) {
            merge(false);
            done = split_arrive_last_via(e.counters + first, last - first + 1, &s_last);
            if (done) {
                // The first workgroup's part of this unit is its last one unless the
                // unit starts with it; the others' is their first
                constexpr int PB = 8;  // parts in flight
                const int parts = last - first + 1;
                const __amdgpu_buffer_rsrc_t all = make_rsrc_u(e.partials + 2 * (int64_t)first * FLOATS, (uint32_t)parts * (2 * FLOATS * 4));
                const uint32_t off = unit_start > first * plan.chunk ? FLOATS * 4 : 0;
                // parts from, from + step, ... of one piece of a row
                auto add_parts = [&](int r, int c8, int from, int step, float &m, float &l, float (&o)[8]) __attribute__((always_inline)) {
                    for (int w0 = from; w0 < parts; w0 += step * PB) {
                        v2u ml[PB];
                        v4f x[PB][2];
#pragma unroll
                        for (int i = 0; i < PB; ++i) {
                            const int w = w0 + i * step;
                            if (w < parts) {
                                const uint32_t base = (uint32_t)w * (2 * FLOATS * 4) + (w == 0 ? off : 0);
                                ml[i] = __builtin_amdgcn_raw_buffer_load_b64(all, base + (uint32_t)((TM * DP + 2 * r) * 4), 0, kCoherent);
                                x[i][0] = load16_coherent(all, base + (uint32_t)((r * DP + c8 * 8) * 4));
                                x[i][1] = load16_coherent(all, base + (uint32_t)((r * DP + c8 * 8 + 4) * 4));
                            }
                        }
#pragma unroll
                        for (int i = 0; i < PB; ++i) {
                            if (w0 + i * step < parts) {
                                const float mw = __uint_as_float(ml[i][0]), n = fmaxf(m, mw);
                                const float f0 = n == kNegInf ? 1.0f : exp2_fast(m - n), f1 = n == kNegInf ? 1.0f : exp2_fast(mw - n);
                                m = n;
                                l = l * f0 + __uint_as_float(ml[i][1]) * f1;
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    o[k] = o[k] * f0 + x[i][k >> 2][k & 3] * f1;
                            }
                        }
                    }
                };
                if (parts <= PB) {
                    // few parts: every thread adds up its own pieces of rows
                    for (int it = end_thread; it < ((rows * QC + 63) & ~63); it += NW * 64) {
                        const int r = min(it / QC, rows - 1), c8 = it % QC;
                        float m = kNegInf, l = 0.0f, o[8] = {};
                        add_parts(r, c8, 0, 1, m, l, o);
                        finish_unit_row(r, c8, m, l, o, it / QC < rows && c8 * 8 < e.c.D);
                    }
                    done = false;
                } else {
                    // each wave adds up every NW-th one, into its ring
                    for (int it = end_lane; it < rows * QC; it += 64) {
                        const int r = it / QC, c8 = it % QC;
                        float m = kNegInf, l = 0.0f, o[8] = {};
                        add_parts(r, c8, wave, NW, m, l, o);
                        float *dst = reinterpret_cast<float *>(mine) + r * DP;
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            *reinterpret_cast<v4f *>(dst + (((2 * c8 + h) ^ (r & 15)) * 4)) = v4f{o[4 * h], o[4 * h + 1], o[4 * h + 2], o[4 * h + 3]};
                        if (c8 == 0) {
                            s_ml[wave][r][0] = m;
                            s_ml[wave][r][1] = l;
                        }
                    }
                    __syncthreads();
                }
            }
        }
        if (done)
            merge(true);
        __syncthreads();  // the rings and s_ml are free again
        at = piece_end;
    }
}

template <int DP, bool FP8, int NT>
void launch(const AttnArgs &a, int plan, int grid, hipStream_t s)
{
    mx_attn_keys_kernel<DP, FP8, NT><<<grid, KeysShape<DP, FP8, NT>::NW * 64, 0, s>>>(a, plan);
}

template <int DP, bool FP8>
constexpr AttnKeysKernel entry()
{
    if constexpr (DP < 256)
        return {{KeysShape<DP, FP8, 1>::PER_CU, KeysShape<DP, FP8, 2>::PER_CU}, {launch<DP, FP8, 1>, launch<DP, FP8, 2>}};
    else
        return {{KeysShape<DP, FP8, 1>::PER_CU, 1}, {launch<DP, FP8, 1>, nullptr}};
}

int padded(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

}  // namespace

int64_t attn_partial_floats(int D) { return 32 * ((int64_t)padded(D) + 4); }  // (the rows kernel's: an m and l per lane)

AttnKeysKernel attn_keys_kernel(int D, bool fp8)
{
    switch (padded(D)) {
    case 64: return fp8 ? entry<64, true>() : entry<64, false>();
    case 128: return fp8 ? entry<128, true>() : entry<128, false>();
    default: return fp8 ? entry<256, true>() : entry<256, false>();
    }
}

}  // namespace mx
