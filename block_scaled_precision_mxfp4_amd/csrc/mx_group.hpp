// Which expert and rows a workgroup of the grouped product has, from the
// device's offsets (gfx950).  By one wave, the same result in every lane;
// offsets are clamped to [0, rows], so that no address beyond the rows is
// formed whatever they hold.
#pragma once

#include "mx_device.hpp"
#include "mx_rows16.hpp"

namespace mx {

__device__ __forceinline__ void group_range(const int32_t *offsets, int E, int rows, int e, int &lo, int &hi)
{
    lo = e < E ? min(max(offsets[e], 0), rows) : 0;
    hi = e < E ? min(max(offsets[e + 1], 0), rows) : 0;
}

// The nth group (from 0) of up to bm rows of one expert, counted through the
// experts in order: the expert, the group's first row and the expert's end;
// false if there are fewer.
__device__ __forceinline__ bool nth_rows(const int32_t *offsets, int E, int rows, int bm, int nth, int lane, int &e, int &m0,
                                         int &m1)
{
    for (int e0 = 0; e0 < E; e0 += 64) {
        int lo, hi;
        group_range(offsets, E, rows, e0 + lane, lo, hi);
        const int n = (max(hi - lo, 0) + bm - 1) / bm;
        const int upto = wave_scan(n);
        const uint64_t past = __ballot(nth < upto);
        if (past) {
            const int at = __ffsll((unsigned long long)past) - 1;
            const int first = __builtin_amdgcn_readlane(lo, at);
            e = e0 + at;
            m0 = first + (nth - __builtin_amdgcn_readlane(upto - n, at)) * bm;
            m1 = __builtin_amdgcn_readlane(hi, at);
            // (offsets that do not ascend can make the sums overflow:
            // whatever came out, the rows are the expert's)
            return m0 >= first && m0 < m1;
        }
        nth -= __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}

struct GroupTile {
    int e;       // expert
    int m0, m1;  // the tile's first row, the expert's end
    int tn;      // column tile
};

// Tile lg of all, in an expert with rows first .. end - 1 whose last row tile
// is number upto - 1.
__device__ __forceinline__ bool tile_in_group(int lg, int first, int end, int upto, int bm, int tiles_n, int group_m,
                                              bool ok, GroupTile &t)
{
    t.m1 = end;
    const int mt = (end - first + bm - 1) / bm;
    const int in = lg - (upto - mt) * tiles_n;  // tile inside the expert
    const int grp = in / (group_m * tiles_n);
    const int gsz = max(min(mt - grp * group_m, group_m), 1);
    const int within = in - grp * group_m * tiles_n;
    t.m0 = first + (grp * group_m + within % gsz) * bm;
    t.tn = within / gsz;
    // (offsets that do not ascend can make the sums overflow: whatever came
    // out, a tile is inside its expert)
    return ok && t.m0 >= first && t.m0 < end && t.tn >= 0 && t.tn < tiles_n;
}

// The tile of workgroup wg among all experts' bm-row tiles x tiles_n column
// tiles; false past the last one.  The workgroups of one XCD take consecutive
// tiles; inside an expert these are columns of up to group_m row tiles, which
// share a tile of B.
__device__ __forceinline__ bool group_tile(const int32_t *offsets, int E, int rows, int bm, int tiles_n, int group_m,
                                           int wg, int lane, GroupTile &t)
{
    int total = 0;
    int lo = 0, hi = 0, upto = 0;  // of the last 64 experts looked at
    for (int e0 = 0; e0 < E; e0 += 64) {
        group_range(offsets, E, rows, e0 + lane, lo, hi);
        upto = total + wave_scan((max(hi - lo, 0) + bm - 1) / bm);
        total = __builtin_amdgcn_readlane(upto, 63);
    }
    if (wg >= total * tiles_n)
        return false;
    const int lg = xcd_remap(wg, total * tiles_n);
    const int want = lg / tiles_n;  // row tile among all
    if (E > 64) {
        int before = 0;
        for (int e0 = 0;; e0 += 64) {
            group_range(offsets, E, rows, e0 + lane, lo, hi);
            upto = before + wave_scan((max(hi - lo, 0) + bm - 1) / bm);
            const int last = __builtin_amdgcn_readlane(upto, 63);
            if (want < last || e0 + 64 >= E) {
                t.e = e0;
                break;
            }
            before = last;
        }
    } else {
        t.e = 0;
    }
    const int at = __ffsll((unsigned long long)__ballot(want < upto)) - 1;
    t.e += at;
    return tile_in_group(lg, __builtin_amdgcn_readlane(lo, at), __builtin_amdgcn_readlane(hi, at),
                         __builtin_amdgcn_readlane(upto, at), bm, tiles_n, group_m, at >= 0 && t.e < E, t);
}

// The same from a table in LDS (s_lo, s_hi, s_upto: an expert's rows and the
// row tiles up to and with its own), which a persistent workgroup makes once
// with make_group_table: no memory is read per tile.
__device__ __forceinline__ int make_group_table(const int32_t *offsets, int E, int rows, int bm, int *s_lo, int *s_hi,
                                                int *s_upto, int lane)
{
    int total = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
        int lo, hi;
        group_range(offsets, E, rows, e0 + lane, lo, hi);
        const int upto = total + wave_scan((max(hi - lo, 0) + bm - 1) / bm);
        total = __builtin_amdgcn_readlane(upto, 63);
        if (e0 + lane < E) {
            s_lo[e0 + lane] = lo;
            s_hi[e0 + lane] = hi;
            s_upto[e0 + lane] = upto;
        }
    }
    return total;
}

__device__ __forceinline__ bool table_tile(const int *s_lo, const int *s_hi, const int *s_upto, int E, int bm, int tiles_n,
                                           int group_m, int lg, int lane, GroupTile &t)
{
    const int want = lg / tiles_n;
    for (int e0 = 0; e0 < E; e0 += 64) {
        const bool past = e0 + lane < E && want < s_upto[e0 + lane];
        const uint64_t m = __ballot(past);
        if (m) {
            t.e = e0 + __ffsll((unsigned long long)m) - 1;
            return tile_in_group(lg, s_lo[t.e], s_hi[t.e], s_upto[t.e], bm, tiles_n, group_m, true, t);
        }
    }
    return false;
}

}  // namespace mx
