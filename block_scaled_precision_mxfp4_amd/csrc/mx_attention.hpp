// Arguments and launchers of the attention kernels over a paged cache (append
// with rotary positions, attention of new tokens).  Host-side only plain
// types; no device code.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace mx {

// A paged cache and the batch that uses it (strides in bytes).
struct CacheArgs {
    uint8_t *k, *v;
    int64_t page_b, head_b, token_b;
    const int32_t *pages;    // [seqs][ld_pages]
    int64_t ld_pages;
    const int32_t *offsets;  // [seqs + 1]
    const int32_t *lens;     // [seqs]
    const float *k_scale, *v_scale;  // [kv_heads] or null
    int num_pages, page_shift, seqs, max_pages, kv_heads;
    int D;
};

// n / d for 0 <= n < 2^31 by a multiplication: d > 1 takes s = ceil(log2 d), m =
// ceil(2^(31 + s) / d) and (n * m) >> (31 + s), off by n (m d - 2^(31 + s)) / (d
// 2^(31 + s)) < 1 / d; m = 0 stands for d = 1.
struct Divisor {
    uint32_t m;
    int shift;  // s - 1, behind the high word
};
inline Divisor divisor(int d)
{
    int s = 0;
    while (((int64_t)1 << s) < d)
        ++s;
    return d > 1 ? Divisor{(uint32_t)((((uint64_t)1 << (31 + s)) + d - 1) / d), s - 1} : Divisor{0, 0};
}

// ---- append (mx_append.hip)
struct AppendArgs {
    CacheArgs c;
    const uint16_t *Q, *K, *V;  // bf16 rows; Q, or K and V, may be null
    uint16_t *QO;
    int64_t ldq, ldk, ldv, ldqo;
    const int32_t *positions;   // [T] or null
    const double *freq;         // [rot / 2], radians a position
    float factor;
    int T, heads, rot, interleaved, fp8;
};
void launch_append(const AppendArgs &a, int num_cu, hipStream_t s);

// ---- attention
constexpr int kAttnTile = 32;    // rows (token, head of a group) that a wave holds
constexpr int kAttnGroup = 128;  // keys that work is handed out by
constexpr int kAttnUnitSteps = 2;  // that a unit of the rows kernel counts beside its keys' (mx_attn_plan.hpp)
constexpr int kAttnPieces = 512; // workgroups that may leave partial results, at most
constexpr int kAttnCounterBytes = 4096;
constexpr int kPlanWhole = 0, kPlanLine = 1, kPlanParts = 2;  // mx_attn_plan.hpp
struct AttnArgs {
    CacheArgs c;
    const uint16_t *Q;
    uint16_t *O;             // bf16 [T][ldo] or null
    float *lse;              // [T][heads] or null
    uint8_t *A, *S;          // quantized rows or null
    const float *sinks;      // [heads] or null
    int64_t ldq, ldo, lda_b, lds;
    float scale;
    int T, heads, group;     // group: query heads of a key head
    Divisor by_group, by_kv_heads;
    int causal, window, a_fp8;
    int *counters;           // [kAttnPieces], zero between calls
    float *partials;
};
// The kernel whose waves take keys in turn (mx_attn_keys.hip): workgroups per
// compute unit; tiles of 32 and of 64 rows (may be null).
typedef void (*AttnLaunchFn)(const AttnArgs &, int plan, int grid, hipStream_t);
struct AttnKeysKernel {
    int per_cu[2];
    AttnLaunchFn launch[2];
};
AttnKeysKernel attn_keys_kernel(int D, bool fp8);
// Floats of 32 rows of a partial result, at most
int64_t attn_partial_floats(int D);
// The kernel whose waves hold 32 rows each (mx_attn_rows.hpp): rows of its
// tiles, workgroups per compute unit.
struct AttnRowsKernel {
    int tile, per_cu;
    AttnLaunchFn launch;
};
AttnRowsKernel attn_rows_kernel(int D, bool fp8, bool small);
AttnRowsKernel attn_rows_kernel_wide(bool fp8);  // D > 128 (mx_attn_rows_wide.hip)

}  // namespace mx
