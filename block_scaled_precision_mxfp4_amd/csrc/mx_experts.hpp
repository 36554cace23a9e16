// Arguments and launchers of the mixture-of-experts kernels (router choice,
// product grouped by expert, gated activation with quantizer, norms with
// residual and quantizer).  Host-side only plain types; no device code.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace mx {

// ---- router choice (mx_route.hip)
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopK = 16;
constexpr int kRouteUnit = 64;        // tokens whose slots are ranked together
constexpr int kRouteFew = 16;         // ... of up to kRouteFewTokens tokens in more than one workgroup
constexpr int kRouteFewTokens = 4096;
constexpr int kRouteMaxBlocks = 256;  // workgroups of the selection; each takes whole units
struct RouteArgs {
    const void *logits;  // f32 or bf16 [T][ldl]
    int32_t *ids;        // [T][k]
    float *weights;      // [T][k]
    int32_t *pos;        // [T][k]
    int32_t *offsets;    // [E + 1]
    int32_t *rows;       // [T * k]
    void *counts;        // workspace [blocks][E] (blocks > 1): uint8 with kRouteFew, else int32
    int T, E, k;
    int64_t ldl;
    int bf16, renorm;
    int unit;            // tokens ranked together: kRouteUnit or kRouteFew
    int units;           // units per workgroup
    int blocks;
};
void launch_route(const RouteArgs &r, hipStream_t s);

// ---- gated activation and quantizer (mx_glu.hip)
struct GluArgs {
    const uint16_t *X;    // bf16 [M][ldx]: gate columns 0..K-1, up columns K..2K-1
    const int32_t *live;  // device count of rows to do, or null
    uint8_t *A, *S;
    int M, K;
    int64_t ldx, lda_b, lds;
    int64_t blocks;       // M * K / 32
    int fp8;
};
int64_t glu_grid(int64_t blocks);
void launch_glu(const GluArgs &g, hipStream_t s);

// ---- norms around a block (mx_norm.hip)
constexpr int kNormMaxK = 16384;
struct NormArgs {
    const uint16_t *Y;       // block output, bf16 [y_rows][ldy]
    const int32_t *pos;      // [T][top_k] rows of Y, or null (row t)
    const float *weights;    // [T][top_k]
    const uint16_t *w_post, *gate, *X, *w_pre;  // each may be null
    uint16_t *H, *Z;         // may be null
    uint8_t *A, *S;          // may be null (both)
    int T, K, top_k, y_rows;
    int64_t ldy, ldg, ldx, ldh, ldz, lda_b, lds;
    float res_scale, eps;
    int fp8;
};
int norm_threads(int K);  // a workgroup's, one per token (twice as many with few tokens)
void launch_norm(const NormArgs &n, int num_cu, hipStream_t s);

// ---- product grouped by expert
struct GroupedArgs {
    uint16_t *D;             // bf16 [M][ldd]
    const uint8_t *A, *B;    // [a_count][lda_b] FP4 or FP8, [E][N][ldb_b] FP4 (byte pitches)
    const uint8_t *SA, *SB;  // E8M0 [a_count][ldsa], [E][N][ldsb]
    const int32_t *offsets;  // [E + 1]
    const int32_t *a_rows;   // [M] or null
    float alpha;
    int M, a_count, N, K, E;
    int KB;                  // K / 32 scale blocks
    int64_t ldd, lda_b, ldsa, ldb_b, ldsb;
    int64_t eb_b, esb;       // bytes from one expert's B, and scales, to the next's
    int tiles_n;             // column tiles
    int group_m;             // an expert's row tiles whose column tiles are taken together
    int d_vec, d_stage;      // 8-byte stores to D allowed; 16-byte ones
    int scale16;             // whole 16-block groups of scale bytes, rows 16-byte aligned
};
// Experts that the persistent tiled kernel keeps a table of in LDS.
constexpr int kGroupTable = 1024;
typedef void (*GroupedLaunchFn)(const GroupedArgs &, int64_t grid, hipStream_t);
struct GroupedTileKernel {
    int bm, bn;
    int min_rows[2];             // rows per expert from which it is taken: FP4 A, FP8 E4M3 A
    GroupedLaunchFn launch[2];   // FP4 A, FP8 E4M3 A (may be null)
    GroupedLaunchFn persist[2];  // persistent (may be null): 16-byte rows of D, N % 8 == 0, K >= 256, at most kGroupTable experts
};
const GroupedTileKernel *grouped_tile_kernels(int *count);
// Few rows per expert (mx_grouped.hip): groups of up to kStreamRows rows, and
// the most that M rows of E experts make
constexpr int kStreamRows = 16;
constexpr int grouped_stream_lines(int M, int E)
{
    const int some = E < M ? E : M;  // experts that can have rows
    return some + (M - some) / kStreamRows;
}
void launch_grouped_stream(bool fp8, const GroupedArgs &g, hipStream_t s);

}  // namespace mx
