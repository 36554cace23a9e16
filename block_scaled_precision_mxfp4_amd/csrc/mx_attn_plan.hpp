// How the attention kernels' work is handed out, found on the device: the host
// knows the new tokens and sequences but no length.
//
// A unit is one tile of a sequence's rows and one key head.  Its cost is its
// sequence's 128-key groups, in steps of `per` groups, and all units' steps, in
// order (sequence, row tile, key head), are one line that is cut into equal
// pieces, one per workgroup.  A unit that a cut goes through is done by several
// workgroups: each leaves a partial result, and the last one to arrive adds
// them up.
//   kPlanWhole  a unit is one step, as many workgroups as there can be units
//   kPlanLine   steps of one group: equal work, but most workgroups do the end
//               of one unit and the start of another, each with its latency
//   kPlanParts  few units: steps as long as it takes for every workgroup to
//               have one step at most (one token over 4096 keys, 8 key heads:
//               21 us in line, where 4 of 132 workgroups did parts of two units)
#pragma once

#include "mx_attn.hpp"
#include "mx_rows16.hpp"

namespace mx {

struct AttnPlan {
    int total;   // steps of all units
    int chunk;   // steps of a workgroup
    int per;     // groups of a step
    int s;       // sequence that the workgroup's first step is in
    int start;   // first step of that sequence's units
    AttnSeq q;   // that sequence
};

__device__ __forceinline__ int seq_steps(const AttnArgs &a, const AttnSeq &q, int tile, int per)
{
    return (seq_groups(a, q, tile) + per - 1) / per;
}
__device__ __forceinline__ int seq_units(const AttnArgs &a, const AttnSeq &q, int tile)
{
    return seq_tiles(q, a.group, tile) * a.c.kv_heads;
}

__device__ __forceinline__ AttnSeq seq_of_lane(const AttnArgs &a, int s)
{
    return seq_from(a.c, a.T, a.c.offsets[s], a.c.offsets[s + 1], a.c.lens[s]);
}
__device__ __forceinline__ AttnSeq lane_seq(const AttnSeq &q, int lane)
{
    return {__builtin_amdgcn_readlane(q.t0, lane), __builtin_amdgcn_readlane(q.n, lane), __builtin_amdgcn_readlane(q.len, lane)};
}
__device__ __forceinline__ int wave_total(int x) { return __builtin_amdgcn_readlane(wave_scan(x), 63); }

// The keys of steps [from, to) of a unit that sees [lo, hi), from a whole group on
struct KeyRange {
    int lo, hi;
};
__device__ __forceinline__ KeyRange step_keys(int lo, int hi, int from, int to, int per)
{
    const int first = lo / kAttnGroup * kAttnGroup;
    const int64_t k0 = first + (int64_t)from * per * kAttnGroup, k1 = first + (int64_t)to * per * kAttnGroup;
    return {(int)min(k0, (int64_t)hi), (int)min(k1, (int64_t)hi)};
}

// The first loads of attn_plan, to be under way while the workgroup does
// something else
struct AttnFirst {
    int o0, o1, len;
};
__device__ __forceinline__ AttnFirst attn_first(const AttnArgs &a, int lane)
{
    AttnFirst f = {0, 0, 0};
    if (a.c.seqs <= 64 && lane < a.c.seqs)
        f = {a.c.offsets[lane], a.c.offsets[lane + 1], a.c.lens[lane]};
    return f;
}

// By one wave, the same result in every lane: the plan, and where workgroup
// `wg` of `wgs` starts.  False: it has nothing (or the offsets count more than T
// tokens, as those that do not ascend may).
__device__ __forceinline__ bool attn_plan(const AttnArgs &a, const AttnFirst &f, int tile, int mode, int wg, int wgs, int lane,
                                          AttnPlan &p)
{
    const int S = a.c.seqs;
    const int each = (S + 63) / 64;  // sequences of a lane, in order
    AttnSeq q = {0, 0, 0};
    int units = 0, steps = 0, tokens = 0;
    p.per = mode == kPlanWhole ? 1 << 24 : 1;
    for (int i = 0; i < each; ++i) {
        const int s = lane * each + i;
        if (s < S) {
            q = each == 1 ? seq_from(a.c, a.T, f.o0, f.o1, f.len) : seq_of_lane(a, s);
            const int u = seq_units(a, q, tile);
            units += u;
            steps += u * seq_steps(a, q, tile, p.per);
            tokens = min(tokens + q.n, a.T + 1);
        }
    }
    if (wave_total(tokens) > a.T)
        return false;
    int to = wave_scan(steps);
    p.total = __builtin_amdgcn_readlane(to, 63);
    p.chunk = (p.total + wgs - 1) / wgs;
    if (mode == kPlanParts && each == 1 && p.chunk > 0) {
        // the host takes this with at most half as many units as workgroups,
        // so that steps of total / (wgs - units) groups are long enough
        const int groups = units > 0 ? steps / units : 0;
        const int all = wave_total(units);
        const int most = (p.total + wgs - all - 1) / max(wgs - all, 1);
        int per = p.chunk, n = 0;
        for (int i = 0; i < 4; ++i) {
            n = wave_total(units * ((groups + per - 1) / per));
            if (n <= wgs)
                break;
            per = min(max(per + 1, per * n / wgs), max(most, 1));
        }
        if (n > wgs)
            per = max(most, 1);
        p.per = per;
        steps = units * ((groups + per - 1) / per);
        to = wave_scan(steps);
        p.total = __builtin_amdgcn_readlane(to, 63);
        p.chunk = (p.total + wgs - 1) / wgs;
    }
    const int at = wg * p.chunk;
    if (at >= p.total)
        return false;
    const int l = __ffsll((unsigned long long)__builtin_amdgcn_ballot_w64(at < to)) - 1;
    p.start = __builtin_amdgcn_readlane(to - steps, l);
    p.s = l * each;
    if (each == 1) {
        p.q = lane_seq(q, l);
        return true;
    }
    // within that lane's sequences
    for (int s0 = p.s;; s0 += 64) {
        const int s = s0 + lane;
        int n = 0;
        if (s < min((l + 1) * each, S)) {
            q = seq_of_lane(a, s);
            n = seq_units(a, q, tile) * seq_steps(a, q, tile, p.per);
        }
        const int upto = p.start + wave_scan(n);
        const uint64_t past = __builtin_amdgcn_ballot_w64(at < upto);
        if (past) {
            const int m = __ffsll((unsigned long long)past) - 1;
            p.s = s0 + m;
            p.start = __builtin_amdgcn_readlane(upto - n, m);
            p.q = lane_seq(q, m);
            return true;
        }
        p.start = __builtin_amdgcn_readlane(upto, 63);
        if (s0 + 64 >= (l + 1) * each)
            return false;
    }
}

}  // namespace mx
