// C-ABI entry points of the mixture-of-experts operators declared in
// libmxgemm.h: argument validation on the host, then one or two launches on
// the caller's stream.  Nothing here allocates or keeps state.
#include "libmxgemm.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdlib>
#include <cstring>

#include "mx_experts.hpp"
#include "mx_host.hpp"

namespace {

constexpr int kMaxK = 1 << 24;
constexpr int64_t kMaxInt = 0x7FFFFFFF;
constexpr int kMaxRows = 1 << 30;                  // of a grouped product: a tile past them still counts in an int
constexpr int kMaxSum = 1024;                      // rows that a token's weighted sum adds
constexpr int64_t kMaxThreads = (int64_t)1 << 32;  // of a launch, exclusive

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// width in bits of the formats an operator here takes (0: not one of them)
int elem_bits(int a_format)
{
    return a_format == MXGEMM_FMT_FP4 ? 4 : a_format == MXGEMM_FMT_FP8_E4M3 ? 8 : 0;
}

// Bytes of a row of lda elements, and whether they are a multiple of 16: no
// product that a stride of any size could overflow
int64_t row_bytes(int64_t lda, int bits) { return bits == 4 ? lda / 2 : lda; }
bool row_aligned(int64_t lda, int bits) { return lda % (128 / bits) == 0; }

// A quantized output (rows of lda elements): extents, then alignment
mxgemm_status check_quantized(const void *A, int K, int64_t lda, int64_t ldsa, int bits)
{
    if (lda < K || ldsa < K / 32)
        return MXGEMM_ERR_SHAPE;
    if (!aligned(A, 16) || !row_aligned(lda, bits))
        return MXGEMM_ERR_ALIGN;
    return MXGEMM_OK;
}

mxgemm_status launched() { return hipGetLastError() == hipSuccess ? MXGEMM_OK : MXGEMM_ERR_HIP; }

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Units of the selection per workgroup, and its workgroups
int route_units_per_block(int T, int unit) { return (int)cdiv(cdiv(T, unit), mx::kRouteMaxBlocks); }
int route_blocks(int T, int unit) { return (int)cdiv(cdiv(T, unit), route_units_per_block(T, unit)); }

// The grouped product's kernel: an index into the tiles, or -1 for streaming.
// The host knows the rows and experts, not how the rows are spread.
//   - Rows that make few tiles (16 an expert, and 128 columns of every expert
//     that can have rows on less than all compute units) are streamed.  Cold
//     weights, us, streaming / the 32-row tile, FP4 and FP8: 4 rows of 32 experts,
//     N = 4096, K = 2048, 8.1 / 9.3 and 8.6 / 9.7; 64 of 16, N = 1024, K = 4096,
//     12.7 / 18.6 and 13.7 / 19.4; 1024 of 64, N = 256, K = 2048, 8.8 / 10.6 and
//     10.5 / 11.2, all of one expert's 8.0 / 7.7 and 9.7 / 8.3.  It loses on short
//     K (K = 512 there 5.5 / 4.6 and 6.3 / 4.8) and, the most, where one of few
//     experts has all of many rows (128 of 8, N = 2880, K = 4096, 20.3 / 12.8 and
//     25.3 / 13.9; evenly spread 20.2 / 20.5 and 25.1 / 20.9): the host does not
//     know how they are spread.
//   - Else the first tile whose rows per expert are reached and whose tiles,
//     every expert's last one half filled, occupy 3/4 of the compute units
//     (8 experts of 128 rows, N = 2048, K = 4096, FP8: 21.1 us on 91 % of them
//     with 64 x 128, 26.3 us on half of them with 128 x 256).
// MXGEMM_GROUPED_TILE=<index> (-1: streaming) is the tests' choice instead.
int plan_grouped(int rows, int N, int groups, int bits, int num_cu)
{
    int n_tiles = 0;
    const mx::GroupedTileKernel *tiles = mx::grouped_tile_kernels(&n_tiles);
    if (const char *e = std::getenv("MXGEMM_GROUPED_TILE")) {
        const int k = std::atoi(e);
        if (k < n_tiles && (k < 0 || tiles[k].launch[bits == 8]))
            return k < 0 ? -1 : k;
    }
    const int64_t some = std::min(rows, groups);  // experts that can have rows
    if (rows <= 16 * some && some * cdiv(N, 128) < num_cu)
        return -1;
    for (int k = 0; k < n_tiles - 1; ++k) {
        const mx::GroupedTileKernel &t = tiles[k];
        if (t.launch[bits == 8] && rows >= (int64_t)t.min_rows[bits == 8] * groups &&
            4 * (rows / t.bm + (some + 1) / 2) * cdiv(N, t.bn) >= 3 * (int64_t)num_cu)
            return k;
    }
    return n_tiles - 1;
}

}  // namespace

extern "C" {

size_t mxgemm_route_workspace_bytes(int T, int E)
{
    if (T < 1 || E < 1 || E > mx::kRouteMaxExperts)
        return 0;
    // (room for four times as many workgroups of kRouteFew tokens, whose
    // counts are a byte each)
    const int blocks = route_blocks(T, mx::kRouteUnit);
    return blocks > 1 ? (size_t)blocks * E * 4 : 0;
}

mxgemm_status mxgemm_route(int32_t *ids, float *weights, int32_t *pos, int32_t *offsets, int32_t *rows,
                           const void *logits, int bf16, int T, int E, int top_k, int64_t ldl, int renorm,
                           void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    if (!ids || !weights || !pos || !offsets || !rows || !logits || (bf16 != 0 && bf16 != 1) ||
        (renorm != 0 && renorm != 1))
        return MXGEMM_ERR_INVALID_ARG;
    if (T < 1 || E < 1 || E > mx::kRouteMaxExperts || top_k < 1 || top_k > mx::kRouteMaxTopK || top_k > E || ldl < E ||
        (int64_t)T * top_k > kMaxInt)
        return MXGEMM_ERR_SHAPE;
    if (!aligned(ids, 4) || !aligned(weights, 4) || !aligned(pos, 4) || !aligned(offsets, 4) || !aligned(rows, 4) ||
        !aligned(logits, bf16 ? 2 : 4))
        return MXGEMM_ERR_ALIGN;
    const size_t need = mxgemm_route_workspace_bytes(T, E);
    if (need > 0) {
        if (!workspace || workspace_bytes < need)
            return MXGEMM_ERR_WORKSPACE;
        if (!aligned(workspace, 4))
            return MXGEMM_ERR_ALIGN;
    }
    mxgemm_status st = mx::check_device();
    if (st != MXGEMM_OK)
        return st;
    mx::RouteArgs r;
    r.logits = logits;
    r.ids = ids;
    r.weights = weights;
    r.pos = pos;
    r.offsets = offsets;
    r.rows = rows;
    r.counts = workspace;
    r.T = T;
    r.E = E;
    r.k = top_k;
    r.ldl = ldl;
    r.bf16 = bf16;
    r.renorm = renorm;
    r.unit = T > mx::kRouteUnit && T <= mx::kRouteFewTokens ? mx::kRouteFew : mx::kRouteUnit;
    r.units = route_units_per_block(T, r.unit);
    r.blocks = route_blocks(T, r.unit);
    mx::launch_route(r, stream);
    return launched();
}

mxgemm_status mxgemm_glu_quantize(void *A, void *scaleA, const void *X, const int32_t *live, int M, int K, int64_t ldx,
                                  int64_t lda, int64_t ldsa, int a_format, hipStream_t stream)
{
    const int bits = elem_bits(a_format);
    if (!A || !scaleA || !X || !bits)
        return MXGEMM_ERR_INVALID_ARG;
    if (M < 1 || K < 32 || K % 32 || K > kMaxK || ldx < 2 * (int64_t)K)
        return MXGEMM_ERR_SHAPE;
    mxgemm_status st = check_quantized(A, K, lda, ldsa, bits);
    if (st != MXGEMM_OK)
        return st;
    if (!aligned(X, 16) || ldx % 8 || !aligned(live, 4))
        return MXGEMM_ERR_ALIGN;
    const int64_t blocks = (int64_t)M * (K / 32);
    if (mx::glu_grid(blocks) * 256 >= kMaxThreads)
        return MXGEMM_ERR_SHAPE;
    st = mx::check_device();
    if (st != MXGEMM_OK)
        return st;
    mx::GluArgs q;
    q.X = (const uint16_t *)X;
    q.live = live;
    q.A = (uint8_t *)A;
    q.S = (uint8_t *)scaleA;
    q.M = M;
    q.K = K;
    q.ldx = ldx;
    q.lda_b = row_bytes(lda, bits);
    q.lds = ldsa;
    q.blocks = blocks;
    q.fp8 = bits == 8;
    mx::launch_glu(q, stream);
    return launched();
}

mxgemm_status mxgemm_norm_quantize(const mxgemm_norm *n, int T, int K, hipStream_t stream)
{
    if (!n || !n->Y || (!n->H && !n->Z && !n->A) || (n->A == nullptr) != (n->scaleA == nullptr) || n->top_k < 0 ||
        (n->top_k > 0) != (n->pos != nullptr) || (n->top_k > 0) != (n->weights != nullptr) || !(n->eps > 0.0f))
        return MXGEMM_ERR_INVALID_ARG;
    const int bits = elem_bits(n->a_format);
    if (!bits)
        return MXGEMM_ERR_INVALID_ARG;
    if (T < 1 || n->top_k > kMaxSum || K < 32 || K % 32 || K > mx::kNormMaxK || n->ldy < K || (n->top_k > 0 && n->y_rows < 1) ||
        (int64_t)T * mx::norm_threads(K) >= kMaxThreads || (n->X && n->ldx < K) || (n->gate && n->ldg != 0 && n->ldg < K) || (n->H && n->ldh < K) || (n->Z && n->ldz < K))
        return MXGEMM_ERR_SHAPE;
    if (n->A) {
        const mxgemm_status st = check_quantized(n->A, K, n->lda, n->ldsa, bits);
        if (st != MXGEMM_OK)
            return st;
    }
    const void *rows[] = {n->Y, n->X, n->gate, n->H, n->Z, n->w_post, n->w_pre};
    const int64_t ld[] = {n->ldy, n->X ? n->ldx : 0, n->gate ? n->ldg : 0, n->H ? n->ldh : 0, n->Z ? n->ldz : 0, 0, 0};
    for (int i = 0; i < 7; ++i)
        if (!aligned(rows[i], 16) || ld[i] % 8)
            return MXGEMM_ERR_ALIGN;
    if (!aligned(n->pos, 4) || !aligned(n->weights, 4))
        return MXGEMM_ERR_ALIGN;
    int cu = 0;
    const mxgemm_status st = mx::check_device(&cu);
    if (st != MXGEMM_OK)
        return st;
    mx::NormArgs a;
    a.Y = (const uint16_t *)n->Y;
    a.pos = n->pos;
    a.weights = n->weights;
    a.w_post = (const uint16_t *)n->w_post;
    a.gate = (const uint16_t *)n->gate;
    a.X = (const uint16_t *)n->X;
    a.w_pre = (const uint16_t *)n->w_pre;
    a.H = (uint16_t *)n->H;
    a.Z = (uint16_t *)n->Z;
    a.A = (uint8_t *)n->A;
    a.S = (uint8_t *)n->scaleA;
    a.T = T;
    a.K = K;
    a.top_k = n->top_k;
    a.y_rows = n->y_rows;
    a.ldy = n->ldy;
    a.ldg = n->ldg;
    a.ldx = n->ldx;
    a.ldh = n->ldh;
    a.ldz = n->ldz;
    a.lda_b = row_bytes(n->lda, bits);
    a.lds = n->ldsa;
    a.res_scale = n->res_scale;
    a.eps = n->eps;
    a.fp8 = bits == 8;
    mx::launch_norm(a, cu, stream);
    return launched();
}

mxgemm_status mxgemm_grouped_run(void *D, const void *A, const void *B, const void *scaleA, const void *scaleB,
                                 const int32_t *offsets, const int32_t *a_rows, float alpha, int rows, int a_count, int N,
                                 int K, int groups, const mxgemm_grouped *strides, hipStream_t stream)
{
    if (!D || !A || !B || !scaleA || !scaleB || !offsets)
        return MXGEMM_ERR_INVALID_ARG;
    mxgemm_grouped s = {N, K, K / 32, K, K / 32, (int64_t)N * K, (int64_t)N * (K / 32), MXGEMM_FMT_FP4};
    if (strides)
        s = *strides;
    const int bits = elem_bits(s.a_format);
    if (!bits)
        return MXGEMM_ERR_INVALID_ARG;
    if (rows < 1 || rows > kMaxRows || a_count < 1 || (!a_rows && a_count < rows) || N < 1 || K < 32 || K % 32 || K > kMaxK || groups < 1 ||
        groups > 65535 || s.ldd < N || s.lda < K || s.ldsa < K / 32 || s.ldb < K || s.ldsb < K / 32 || s.strideb < 0 ||
        s.strideb_scale < 0)
        return MXGEMM_ERR_SHAPE;
    if (s.lda % 2 || s.ldb % 2 || s.strideb % 2 || !aligned(A, 16) || !aligned(B, 16) || !row_aligned(s.lda, bits) ||
        (s.ldb / 2) % 16 || (s.strideb / 2) % 16 || !aligned(D, 2) || !aligned(offsets, 4) || !aligned(a_rows, 4))
        return MXGEMM_ERR_ALIGN;
    mx::GroupedArgs g = {};
    g.lda_b = row_bytes(s.lda, bits);
    g.ldb_b = s.ldb / 2;
    // the kernels address a tile's rows of B, and through a row list all of
    // A, with 32-bit offsets
    constexpr int64_t kSpan = (int64_t)1 << 31;
    const int64_t a_span = a_rows ? a_count : 256;
    if (g.lda_b >= kSpan / a_span || s.ldsa >= kSpan / a_span || g.ldb_b >= kSpan / 256 || s.ldsb >= kSpan / 256)
        return MXGEMM_ERR_SHAPE;
    g.D = (uint16_t *)D;
    g.A = (const uint8_t *)A;
    g.B = (const uint8_t *)B;
    g.SA = (const uint8_t *)scaleA;
    g.SB = (const uint8_t *)scaleB;
    g.offsets = offsets;
    g.a_rows = a_rows;
    g.alpha = alpha;
    g.M = rows;
    g.a_count = a_count;
    g.N = N;
    g.K = K;
    g.KB = K / 32;
    g.E = groups;
    g.ldd = s.ldd;
    g.ldsa = s.ldsa;
    g.ldsb = s.ldsb;
    g.eb_b = s.strideb / 2;
    g.esb = s.strideb_scale;
    g.d_vec = aligned(D, 8) && s.ldd % 4 == 0;
    g.d_stage = aligned(D, 16) && s.ldd % 8 == 0;
    auto scale_rows = [&](const void *p, int64_t ld, int64_t n) { return g.KB % n == 0 && aligned(p, n) && ld % n == 0; };
    g.scale16 = scale_rows(scaleA, s.ldsa, 16) && scale_rows(scaleB, s.ldsb, 16) && s.strideb_scale % 16 == 0;
    g.group_m = 8;

    int cu = 0;
    const mxgemm_status st = mx::check_device(&cu);
    if (st != MXGEMM_OK)
        return st;
    const int kernel = plan_grouped(rows, N, groups, bits, cu);
    if (kernel < 0) {
        if (cdiv(N, 32) * 256 >= kMaxThreads || mx::grouped_stream_lines(rows, groups) > 65535)
            return MXGEMM_ERR_SHAPE;
        mx::launch_grouped_stream(bits == 8, g, stream);
        return launched();
    }
    int n_tiles = 0;
    const mx::GroupedTileKernel &t = mx::grouped_tile_kernels(&n_tiles)[kernel];
    const int64_t some = std::min(rows, groups);
    const int64_t grid = ((rows - some) / t.bm + some) * cdiv(N, t.bn);
    if (grid * 512 >= kMaxThreads)  // (a tile's threads are 512 at most)
        return MXGEMM_ERR_SHAPE;
    g.tiles_n = (int)cdiv(N, t.bn);
    const char *e = std::getenv("MXGEMM_TILE_PERSIST");
    if (t.persist[bits == 8] && !(e && std::strcmp(e, "0") == 0) && grid > cu && g.d_stage && N % 8 == 0 &&
        K >= 256 && groups <= mx::kGroupTable && s.ldd < ((int64_t)1 << 21))
        t.persist[bits == 8](g, cu, stream);
    else
        t.launch[bits == 8](g, grid, stream);
    return launched();
}

}  // extern "C"
