// The router's choice on gfx950: from logits [T][E] each token's top k
// experts with softmax weights, and the row list that orders the T*k chosen
// (token, slot) pairs by expert for the grouped product.
//
// Selection.  16 lanes share a token, four tokens a wave; lane l keeps the
// experts l, l + 16, ... as unsigned keys that order like the values (-inf
// and NaN: key 0, never chosen; -0 is +0 first, so that equal values tie).
// Each of the k rounds takes the largest key, then the lowest expert that has
// it: two butterfly reductions over the 16 lanes with row permutes (no LDS).
// Weights are exp(x - max) / sum in fp32, the sum over the chosen experts or
// over all of them.
//
// Grouping, without atomics, so that the order is that of the tokens.  A
// unit's slots, those of 64 tokens, are ranked together: for 64 consecutive slots a wave finds
// the lanes with the same expert from one ballot per bit of the expert's
// number; the rank inside the wave is a population count, and a count per
// (wave, expert) in LDS, summed over the waves in order, makes it the rank
// inside the unit.  With one workgroup (T <= 64) the offsets follow in the
// same launch; otherwise every workgroup leaves its counts in the workspace and
// a second kernel adds the counts of the workgroups before it.  From 65 to
// 4096 tokens a unit is 16 tokens: four times as many compute units share the
// rounds, and counts of a byte keep the second launch's reads as they were
// (64-token units against 16, both launches, us: 509 tokens of 64 experts, top
// 6, 8.1 / 7.1; 1024 of 128, top 8, 10.4 / 8.5; 4096 of 512 63 / 32; 4096 of 128
// 11.3 / 11.4; at 2048 of 256, top 2, they lose, 10.0 / 10.7).
//
// Bound by latency: one token of 32 experts, top 4, 3.6 us (waves without a token
// skip the rounds: 0.3 less, 1 token of 1024 experts 53 -> 22).  Long
// inputs: 16384 tokens of 128 experts, top 8 (8.4 MB of logits, 1.6 us at the
// copy's rate), 14.0 us: the selection's rounds, about 60 instructions each,
// then the second launch, whose every workgroup reads all workgroups' counts (4
// units a workgroup there, for a quarter of these reads: 7.0 -> 10.0 us; 16 or
// 32 reads in flight instead of 8: no gain).
#include "mx_device.hpp"
#include "mx_experts.hpp"
#include "mx_rows16.hpp"

namespace mx {

__device__ __forceinline__ uint32_t row_max(uint32_t v)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v = max(v, row_partner(v, i));
    return v;
}

__device__ __forceinline__ uint32_t row_min(uint32_t v)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v = min(v, row_partner(v, i));
    return v;
}

__device__ __forceinline__ float row_sum(float v)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v += __uint_as_float(row_partner(__float_as_uint(v), i));
    return v;
}

__device__ __forceinline__ uint32_t key_of(float x)
{
    const uint32_t u = __float_as_uint(x + 0.0f);
    if (!(x > -INFINITY))  // -inf or NaN
        return 0;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float value_of(uint32_t key)
{
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// exp(x - m), 1 where x is the maximum itself (also a maximum of +inf)
__device__ __forceinline__ float share(float x, float m) { return x == m ? 1.0f : expf(x - m); }

// start[e] = sum of count[0 .. e-1], start[E] the total; by one wave
__device__ __forceinline__ void exclusive_scan(const int *count, int *start, int E, int lane)
{
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
        const int e = e0 + lane;
        const int c = e < E ? count[e] : 0;
        const int s = wave_scan(c);
        if (e < E)
            start[e] = carry + s - c;
        carry += __builtin_amdgcn_readlane(s, 63);
    }
    if (lane == 0)
        start[E] = carry;
}

// V: experts per lane (E <= 16 V); NT: threads (NT / 16 tokens a pass); TOK:
// tokens ranked together
template <int V, int NT, bool BF16, int TOK>
__global__ void __launch_bounds__(NT) mx_route_select_kernel(RouteArgs r)
{
    constexpr int NW = NT / 64;
    constexpr int TPP = NT / 16;                     // tokens per pass
    constexpr int MAXCH = TOK * kRouteMaxTopK / 64;
    constexpr int CPW = MAXCH / NW > 0 ? MAXCH / NW : 1;  // 64-slot chunks per wave
    extern __shared__ int s_mem[];
    int *s_base = s_mem;                             // [E + 1] rows of this workgroup per expert so far
    int *s_start = s_mem + r.E + 1;                  // [E + 1]
    int16_t *s_id = reinterpret_cast<int16_t *>(s_start + r.E + 1);  // [TOK k]
    uint16_t *s_cnt = reinterpret_cast<uint16_t *>(s_id + TOK * kRouteMaxTopK);  // [chunks][E]

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int l = lane & 15;
    const int k = r.k, E = r.E;
    const int chunks = (TOK * k + 63) / 64;
    for (int e = tid; e < E; e += NT)
        s_base[e] = 0;

    for (int unit = 0; unit < r.units; ++unit) {
        const int64_t t0 = ((int64_t)blockIdx.x * r.units + unit) * TOK;
        if (t0 >= r.T)
            break;
        for (int i = tid; i < chunks * E; i += NT)
            s_cnt[i] = 0;
#pragma unroll 1
        for (int pass = 0; pass < TOK / TPP; ++pass) {
            const int u = pass * TPP + tid / 16;  // token of the unit
            const int64_t t = t0 + u;
            const bool live = t < r.T;
            if (t0 + pass * TPP + wave * 4 >= r.T) {  // (none of the wave's four)
                if (l < k)
                    s_id[u * k + l] = -1;
                continue;
            }
            uint32_t key[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int e = v * 16 + l;
                float x = -INFINITY;
                if (live && e < E) {
                    if constexpr (BF16)
                        x = bf16_to_f32(reinterpret_cast<const uint16_t *>(r.logits)[t * r.ldl + e]);
                    else
                        x = reinterpret_cast<const float *>(r.logits)[t * r.ldl + e];
                }
                key[v] = key_of(x);
            }
            uint32_t best = 0;
#pragma unroll
            for (int v = 0; v < V; ++v)
                best = max(best, key[v]);
            best = row_max(best);
            const float m = value_of(best);
            float total = 0.0f;
            if (!r.renorm) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    total += key[v] ? share(value_of(key[v]), m) : 0.0f;
                total = row_sum(total);
            }
            int mine = -1;        // lane j keeps the j-th choice
            uint32_t mine_key = 0;
            for (int j = 0; j < k; ++j) {
                uint32_t at = 0xFFFFFFFFu;
#pragma unroll
                for (int v = V - 1; v >= 0; --v)
                    at = key[v] == best ? (uint32_t)(v * 16 + l) : at;
                at = row_min(at);
                if (l == j && best) {
                    mine = (int)at;
                    mine_key = best;
                }
                uint32_t next = 0;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    key[v] = (uint32_t)(v * 16 + l) == at ? 0 : key[v];
                    next = max(next, key[v]);
                }
                best = row_max(next);
            }
            const float p = mine >= 0 ? share(value_of(mine_key), m) : 0.0f;
            if (r.renorm)
                total = row_sum(p);
            if (l < k) {
                s_id[u * k + l] = (int16_t)mine;
                if (live) {
                    r.ids[t * k + l] = mine;
                    r.weights[t * k + l] = mine >= 0 ? p / total : 0.0f;
                }
            }
        }
        __syncthreads();
        // ranks: chunk c = 64 consecutive slots, by wave c % NW
        int rank[CPW], id[CPW];
#pragma unroll
        for (int i = 0; i < CPW; ++i) {
            const int c = i * NW + wave;
            rank[i] = 0;
            id[i] = -1;
            if (c < chunks) {
                if (TOK == 64 || c * 64 + lane < TOK * k)
                    id[i] = s_id[c * 64 + lane];
                uint64_t same = __ballot(id[i] >= 0);
                for (int b = 0; (1 << b) < E; ++b) {
                    const bool bit = (id[i] >> b) & 1;
                    const uint64_t ones = __ballot(bit);
                    same &= bit ? ones : ~ones;
                }
                const uint64_t before = same & ((1ull << lane) - 1);
                rank[i] = __popcll(before);
                if (id[i] >= 0 && before == 0)
                    s_cnt[c * E + id[i]] = (uint16_t)__popcll(same);
            }
        }
        __syncthreads();
        for (int e = tid; e < E; e += NT) {
            int run = 0;
            for (int c = 0; c < chunks; ++c) {
                const int n = s_cnt[c * E + e];
                s_cnt[c * E + e] = (uint16_t)run;
                run += n;
            }
            s_start[e] = run;  // this unit's rows of expert e
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < CPW; ++i) {
            const int c = i * NW + wave;
            const int64_t slot = t0 * k + c * 64 + lane;
            if (c * 64 + lane < TOK * k && slot < (int64_t)r.T * k)
                r.pos[slot] = id[i] >= 0 ? s_base[id[i]] + s_cnt[c * E + id[i]] + rank[i] : -1;
        }
        __syncthreads();
        for (int e = tid; e < E; e += NT)
            s_base[e] += s_start[e];
        __syncthreads();
    }

    if (r.blocks > 1) {
        for (int e = tid; e < E; e += NT) {
            if constexpr (TOK == kRouteFew)  // (one unit: 16 at most)
                reinterpret_cast<uint8_t *>(r.counts)[(int64_t)blockIdx.x * E + e] = (uint8_t)s_base[e];
            else
                reinterpret_cast<int32_t *>(r.counts)[(int64_t)blockIdx.x * E + e] = s_base[e];
        }
        return;
    }
    // one workgroup, one unit: the ranks are final, the offsets follow
    if (wave == 0)
        exclusive_scan(s_base, s_start, E, lane);
    __syncthreads();
    for (int e = tid; e <= E; e += NT)
        r.offsets[e] = s_start[e];
    const int n = r.T * k;
    for (int i = tid; i < n; i += NT) {
        if (i >= s_start[E])
            r.rows[i] = -1;
    }
#pragma unroll
    for (int i = 0; i < CPW; ++i) {
        const int c = i * NW + wave;
        const int slot = c * 64 + lane;
        if (c < k && slot < n) {
            const int e = s_id[slot];
            if (e >= 0) {
                const int p = s_start[e] + r.pos[slot];  // written by this thread above
                r.pos[slot] = p;
                r.rows[p] = slot / k;
            }
        }
    }
}

// Second launch: workgroup b's ranks become positions.
template <typename Count>
__global__ void __launch_bounds__(1024) mx_route_place_kernel(RouteArgs r)
{
    extern __shared__ int s_mem[];
    const int E = r.E, k = r.k;
    int *s_total = s_mem, *s_before = s_mem + E, *s_start = s_mem + 2 * E;  // [E], [E], [E + 1]
    const int tid = threadIdx.x;
    for (int e = tid; e < E; e += 1024)
        s_total[e] = s_before[e] = 0;
    __syncthreads();
    // 1024 / ep workgroups' counts at a time (E <= 1024); integer sums
    int ep = 1;
    while (ep < E)
        ep *= 2;
    const int e = tid & (ep - 1);
    if (e < E) {
        int total = 0, before = 0;
        // (a batch's loads are in flight together)
        for (int b0 = tid / ep; b0 < r.blocks; b0 += 8 * (1024 / ep)) {
            int c[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int b = b0 + i * (1024 / ep);
                c[i] = b < r.blocks ? (int)reinterpret_cast<const Count *>(r.counts)[(int64_t)b * E + e] : 0;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                total += c[i];
                before += b0 + i * (1024 / ep) < (int)blockIdx.x ? c[i] : 0;
            }
        }
        atomicAdd(&s_total[e], total);
        atomicAdd(&s_before[e], before);
    }
    __syncthreads();
    if (tid < 64)
        exclusive_scan(s_total, s_start, E, tid);
    __syncthreads();
    if (blockIdx.x == 0)
        for (int i = tid; i <= E; i += 1024)
            r.offsets[i] = s_start[i];
    const int64_t slots = (int64_t)r.T * k;
    const int64_t first = (int64_t)blockIdx.x * r.units * r.unit * k;
    const int64_t last = min(slots, first + (int64_t)r.units * r.unit * k);
    for (int64_t i = first + tid; i < last; i += 1024) {
        const int id = r.ids[i];
        if (id >= 0) {
            const int p = s_start[id] + s_before[id] + r.pos[i];
            r.pos[i] = p;
            r.rows[p] = (int32_t)(i / k);
        }
        if (i >= s_start[E])
            r.rows[i] = -1;
    }
}

template <int V, int NT, int TOK>
static void launch_select_unit(const RouteArgs &r, hipStream_t s)
{
    const size_t lds = (size_t)(2 * (r.E + 1)) * 4 + TOK * kRouteMaxTopK * 2 + (size_t)((TOK * r.k + 63) / 64) * r.E * 2;
    if (r.bf16)
        hipLaunchKernelGGL((mx_route_select_kernel<V, NT, true, TOK>), dim3(r.blocks), dim3(NT), lds, s, r);
    else
        hipLaunchKernelGGL((mx_route_select_kernel<V, NT, false, TOK>), dim3(r.blocks), dim3(NT), lds, s, r);
}

template <int V, int NT>
static void launch_select(const RouteArgs &r, hipStream_t s)
{
    if (r.unit == kRouteFew)
        launch_select_unit<V, 16 * kRouteFew, kRouteFew>(r, s);
    else
        launch_select_unit<V, NT, kRouteUnit>(r, s);
}

void launch_route(const RouteArgs &r, hipStream_t s)
{
    // 64 tokens a pass where a lane's keys leave room for 16 waves, 32 for 8
    if (r.E <= 32)
        launch_select<2, 1024>(r, s);
    else if (r.E <= 64)
        launch_select<4, 1024>(r, s);
    else if (r.E <= 128)
        launch_select<8, 1024>(r, s);
    else if (r.E <= 256)
        launch_select<16, 1024>(r, s);
    else if (r.E <= 512)
        launch_select<32, 512>(r, s);
    else
        launch_select<64, 256>(r, s);
    if (r.blocks > 1 && r.unit == kRouteFew)
        hipLaunchKernelGGL(mx_route_place_kernel<uint8_t>, dim3(r.blocks), dim3(1024), (size_t)(3 * r.E + 1) * 4, s, r);
    else if (r.blocks > 1)
        hipLaunchKernelGGL(mx_route_place_kernel<int32_t>, dim3(r.blocks), dim3(1024), (size_t)(3 * r.E + 1) * 4, s, r);
}

}  // namespace mx
