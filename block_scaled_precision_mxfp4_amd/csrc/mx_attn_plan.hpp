// How the attention kernels' work is handed out, found on the device: the host
// knows the new tokens and sequences but no length.
//
// A unit is one tile of a sequence's rows and one key head.  Its cost is counted
// in steps of some 128-key groups, and all units' steps, in order (sequence, row
// tile, key head), are one line that is cut into equal pieces, one per workgroup.
// A unit that a cut goes through is done by several workgroups: each leaves a
// partial result, and the last one to arrive adds them up.
//   kPlanLine   steps of one group: equal work, but most workgroups do the end
//               of one unit and the start of another, each with its latency
//   kPlanParts  (keys kernel) few units: steps as long as it takes for every
//               workgroup to have one step at most (one token over 4096 keys, 8
//               key heads: 21 us in line, where 4 of 132 workgroups did parts of
//               two units)
//   kPlanWhole  (rows kernel) many units: a workgroup does a whole one
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
__device__ __forceinline__ int wave_max(int x)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        x = max(x, __shfl_xor(x, d));
    return __builtin_amdgcn_readfirstlane(x);
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
// `wg` of `wgs` starts, in steps of per0 groups (kPlanParts: its own).  False: it has nothing (or the offsets count more than T
// tokens, as those that do not ascend may).
__device__ __forceinline__ bool attn_plan(const AttnArgs &a, const AttnFirst &f, int tile, int per0, int mode, int wg, int wgs,
                                          int lane, AttnPlan &p)
{
    const int S = a.c.seqs;
    const int each = (S + 63) / 64;  // sequences of a lane, in order
    AttnSeq q = {0, 0, 0};
    int units = 0, steps = 0, tokens = 0;
    p.per = per0;
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

// ---- the rows kernel's tiles
//
// Up to 64 sequences, whose tiles' own costs count: a tile of a causal prompt
// sees the keys up to its last row.  In line each tile's groups are its steps, and
// kAttnUnitSteps behind them stand for the time that any unit takes (loads of its
// rows and first keys, its output); whole units go out by their keys, most first
// (within 64 levels), so that the last to start are the shortest.  More sequences: every tile of a sequence costs
// the sequence's groups, and whole units go out in order.  us, with every tile at
// its sequence's groups / as it is: 8 texts of 469 to 1497 tokens, 16 heads of 64,
// not causal 68 / 62 (whole units in order / longest first); two prompts of 1000
// tokens, 16 heads of 256 78 / 57; 509 tokens behind a window of 128 19 / 17; a
// prompt of 2048 tokens 67 / 63 (without the steps beside the keys 112: its last
// workgroups did nine units of one group each).
struct AttnTile {
    int wg;        // the workgroup's place in the line
    int at, end;   // its steps
    int chunk;     // steps of a workgroup
    int s, head, nth;  // sequence, key head, and tile from the sequence's last, that the step `at` is in
    int start;     // first step of that unit
    int per;       // groups of a step
    bool exact;    // tiles have their own costs
    AttnSeq q;
};

// Keys that tile `tile` sees
__device__ __forceinline__ void keys_of_tile(const AttnArgs &a, const AttnSeq &q, int tile, int size, int &lo, int &hi)
{
    const int r0 = tile * size, r1 = min(q.n * a.group, r0 + size) - 1;
    tile_keys(a, q, quotient(r0, a.by_group), quotient(r1, a.by_group), lo, hi);
}

// Steps with keys of one unit of tile `tile`
__device__ __forceinline__ int tile_steps(const AttnArgs &a, const AttnSeq &q, int tile, int size, const AttnTile &p)
{
    if (!p.exact)
        return seq_steps(a, q, size, p.per);
    int lo, hi;
    keys_of_tile(a, q, tile, size, lo, hi);
    return max(key_blocks(hi, kAttnGroup) - lo / kAttnGroup, 1);
}

// Steps of one unit: those with keys and the others
__device__ __forceinline__ int unit_steps(const AttnTile &p, int steps) { return steps + (p.exact ? kAttnUnitSteps : 0); }

// Tiles of a sequence that see a key at `from` or behind (causal: those from
// row (from - first position) * group on)
__device__ __forceinline__ int tiles_that_see(const AttnArgs &a, const AttnSeq &q, int tiles, int size, int from)
{
    if (from <= 0)
        return tiles;
    if (from > q.len)
        return 0;
    if (!a.causal)
        return tiles;  // (a sequence shorter than its new tokens: its tiles are of the longest's level)
    const int before = max(from - 1 - (q.len - q.n), 0) * a.group / size;  // whole tiles of rows that do not
    return max(tiles - before, 0);
}

// By one wave, the same result in every lane: the first unit of workgroup `wg`
// of `wgs`.  False: it has nothing, or the offsets count more than T tokens.
__device__ __forceinline__ bool attn_tiles(const AttnArgs &a, const AttnFirst &f, int size, int mode, int wg, int wgs, int lane,
                                           AttnTile &p)
{
    const int S = a.c.seqs, Hk = a.c.kv_heads;
    const bool whole = mode == kPlanWhole;
    p.wg = wg;
    p.exact = S <= 64;
    p.per = whole ? 1 << 24 : 1;
    int sum = 0;  // steps of a head of the sequence
    if (p.exact) {
        AttnSeq q = {0, 0, 0};
        if (lane < S)
            q = seq_from(a.c, a.T, f.o0, f.o1, f.len);
        if (wave_total(min(q.n, a.T + 1)) > a.T)
            return false;
        const int tiles = seq_tiles(q, a.group, size);
        const int units = wave_total(tiles) * Hk;
        int steps = 0, to = 0, total = 0;
        bool whole = mode == kPlanWhole;
        if (!whole) {
            const int last = tiles > 0 ? unit_steps(p, tile_steps(a, q, tiles - 1, size, p)) : 0;
            steps = last;
            for (uint64_t many = __builtin_amdgcn_ballot_w64(tiles > 1); many; many &= many - 1) {
                const int m = __ffsll((unsigned long long)many) - 1;
                const AttnSeq one = lane_seq(q, m);
                const int n = __builtin_amdgcn_readlane(tiles, m);
                int part = 0;
                for (int t = lane; t < n; t += 64)
                    part += unit_steps(p, tile_steps(a, one, t, size, p));
                part = wave_total(part);
                if (lane == m)
                    steps = part;
            }
            to = wave_scan(steps * Hk);
            total = __builtin_amdgcn_readlane(to, 63);
            p.chunk = (total + wgs - 1) / wgs;
            whole = units <= wgs && wave_max(last) <= p.chunk + p.chunk / 16 + 2;  // (cuts would save little)
        }
        if (whole) {
            const int rank = quotient(wg, a.by_kv_heads);
            if (wg >= units)
                return false;
            const int shift = max(26 - __clz(max(wave_max(q.len), 1)), 0);  // level of a tile: keys >> shift, 0 .. 63
            // the level of the tile of that rank: the least with no more tiles above it
            int level = 0;
#pragma unroll
            for (int d = 32; d > 0; d >>= 1)
                if (wave_total(tiles_that_see(a, q, tiles, size, (level + d) << shift)) > rank)
                    level += d;
            const int above = tiles_that_see(a, q, tiles, size, (int)min((int64_t)(level + 1) << shift, (int64_t)0x7FFFFFFF));
            const int here = tiles_that_see(a, q, tiles, size, level << shift) - above;
            to = wave_scan(here);
            const int r = rank - wave_total(above);
            const int l = __ffsll((unsigned long long)__builtin_amdgcn_ballot_w64(r < to)) - 1;
            p.nth = __builtin_amdgcn_readlane(above, l) + r - __builtin_amdgcn_readlane(to - here, l);
            p.head = wg - rank * Hk;
            p.at = p.start = 0;
            p.end = p.chunk = 1;
            p.s = l;
            p.q = lane_seq(q, l);
            p.exact = false;  // (one step)
            p.per = 1 << 24;
            return true;
        }
        // Few sequences: an XCD's workgroups, every eighth, stand next to each other,
        // so that a head's keys and values come into one L2 (512 tokens over 8192 99 /
        // 93 us).  Many: tiles bound by HBM and by the matrix units go to every XCD
        // (512 tokens in a batch of 32 decoding ones 95 us, next to each other 100).
        if (S < 8 && wgs % 8 == 0)
            p.wg = wg % 8 * (wgs / 8) + wg / 8;
        p.at = p.wg * p.chunk;
        p.end = min(p.at + p.chunk, total);
        if (p.at >= total)
            return false;
        const int l = __ffsll((unsigned long long)__builtin_amdgcn_ballot_w64(p.at < to)) - 1;
        p.start = __builtin_amdgcn_readlane(to - steps * Hk, l);
        sum = __builtin_amdgcn_readlane(steps, l);
        p.s = l;
        p.q = lane_seq(q, l);
    } else {
        AttnPlan line;
        if (!attn_plan(a, f, size, p.per, mode, wg, wgs, lane, line))
            return false;
        p.chunk = line.chunk;
        p.at = wg * p.chunk;
        p.end = min(p.at + p.chunk, line.total);
        p.start = line.start;
        p.s = line.s;
        p.q = line.q;
        sum = seq_tiles(p.q, a.group, size) * seq_steps(a, p.q, size, p.per);
    }
    // the head and the tile
    p.head = (p.at - p.start) / sum;
    p.start += p.head * sum;
    const int tiles = seq_tiles(p.q, a.group, size);
    for (int n0 = 0; n0 < tiles; n0 += 64) {
        const int i = n0 + lane;
        const int steps = i < tiles ? unit_steps(p, tile_steps(a, p.q, tiles - 1 - i, size, p)) : 0;
        const int upto = p.start + wave_scan(steps);
        const uint64_t past = __builtin_amdgcn_ballot_w64(p.at < upto);
        if (past) {
            const int m = __ffsll((unsigned long long)past) - 1;
            p.nth = n0 + m;
            p.start = __builtin_amdgcn_readlane(upto - steps, m);
            return true;
        }
        p.start = __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}

}  // namespace mx
