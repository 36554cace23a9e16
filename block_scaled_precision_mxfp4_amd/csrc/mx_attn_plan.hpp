// How the attention kernels' work is handed out, found on the device: the host
// knows the new tokens and sequences but no length.
//
// A unit is one tile of a sequence's rows and one key head.  Its cost is the
// 128-key groups of its sequence, and all units' groups, in order (sequence,
// row tile, key head), are one line that is cut into equal pieces, one per
// workgroup.  A unit that a cut goes through is done by several workgroups:
// each leaves a partial result, and the last one to arrive adds them up.  With
// `whole` every unit counts 1, and with as many workgroups as there can be units
// none is cut.
#pragma once

#include "mx_attn.hpp"
#include "mx_rows16.hpp"

namespace mx {

struct AttnPlan {
    int total;      // groups of all units
    int s;          // sequence that group `at` is in
    int start;      // first group of the sequence's units
};

// Groups of a sequence as a lane sees it
__device__ __forceinline__ void plan_costs(const AttnArgs &a, const AttnSeq &q, int tile, int whole, int &groups)
{
    const int units = seq_tiles(q, a.group, tile) * a.c.kv_heads;
    groups = units > 0 ? units * (whole ? 1 : seq_groups(q, a.group, tile, a.window)) : 0;
}

// By one wave, the same result in every lane: the line's length and the
// sequence that piece number `piece` of `pieces` starts in.  False: there is
// nothing (the piece is past the end, or the offsets count more than T tokens,
// as those that do not ascend may).
__device__ __forceinline__ bool attn_plan(const AttnArgs &a, int tile, int whole, int piece, int pieces, int lane, AttnPlan &p,
                                          int &chunk)
{
    const int S = a.c.seqs;
    const int per = (S + 63) / 64;  // sequences of a lane, in order
    int groups = 0, tokens = 0;
    for (int i = 0; i < per; ++i) {
        const int s = lane * per + i;
        if (s < S) {
            const AttnSeq q = seq_from(a.c, a.T, a.c.offsets[s], a.c.offsets[s + 1], a.c.lens[s]);
            int g;
            plan_costs(a, q, tile, whole, g);
            groups += g;
            tokens = min(tokens + q.n, a.T + 1);
        }
    }
    const int g_to = wave_scan(groups);
    const int all_tokens = __builtin_amdgcn_readlane(wave_scan(tokens), 63);
    p.total = __builtin_amdgcn_readlane(g_to, 63);
    chunk = (p.total + pieces - 1) / pieces;
    const int at = piece * chunk;
    if (all_tokens > a.T || at >= p.total)
        return false;
    const int l = __ffsll((unsigned long long)__builtin_amdgcn_ballot_w64(at < g_to)) - 1;
    p.start = __builtin_amdgcn_readlane(g_to - groups, l);
    p.s = l * per;
    if (per == 1)
        return true;
    // within that lane's sequences
    for (int s0 = p.s;; s0 += 64) {
        const int s = s0 + lane;
        int g = 0;
        if (s < min((l + 1) * per, S)) {
            const AttnSeq q = seq_from(a.c, a.T, a.c.offsets[s], a.c.offsets[s + 1], a.c.lens[s]);
            plan_costs(a, q, tile, whole, g);
        }
        const int g2 = p.start + wave_scan(g);
        const uint64_t past = __builtin_amdgcn_ballot_w64(at < g2);
        if (past) {
            const int m = __ffsll((unsigned long long)past) - 1;
            p.s = s0 + m;
            p.start = __builtin_amdgcn_readlane(g2 - g, m);
            return true;
        }
        p.start = __builtin_amdgcn_readlane(g2, 63);
        if (s0 + 64 >= (l + 1) * per)
            return false;
    }
}

}  // namespace mx
