// C-ABI entry points of the attention over a paged cache declared in
// libmxgemm.h: argument validation on the host, then one launch on the
// caller's stream.  Nothing here allocates or keeps state.
#include "libmxgemm.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>

#include "mx_attention.hpp"
#include "mx_host.hpp"

namespace {

constexpr int kMaxTokens = 1 << 24;
constexpr int kMaxSeqs = 1 << 16;
constexpr int64_t kMaxRows = (int64_t)1 << 30;  // T * heads of an attention
constexpr int64_t kMaxThreads = ((int64_t)1 << 32) - 1;  // of a launch
constexpr int kMaxHeads = 512;  // of queries, keys and values together
constexpr int64_t kMaxInt = 0x7FFFFFFF;

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
mxgemm_status launched() { return hipGetLastError() == hipSuccess ? MXGEMM_OK : MXGEMM_ERR_HIP; }

// The cache's own rules; pages: whether its keys and values are used
mxgemm_status check_cache(const mxgemm_kv_cache *c, bool pages, mx::CacheArgs &a)
{
    if (!c || !c->offsets || !c->lens || (pages && (!c->k || !c->v || !c->pages)) ||
        (c->format != MXGEMM_KV_BF16 && c->format != MXGEMM_KV_FP8_E4M3) ||
        (c->format == MXGEMM_KV_BF16 && (c->k_scale || c->v_scale)))
        return MXGEMM_ERR_INVALID_ARG;
    const int D = c->head_dim, P = c->page_size, width = c->format == MXGEMM_KV_BF16 ? 2 : 1;
    if (c->seqs < 1 || c->seqs > kMaxSeqs || c->kv_heads < 1 || c->kv_heads > kMaxHeads || D < 32 || D > 256 || D % 32 ||
        P < 16 || P > 65536 || (P & (P - 1)) || c->num_pages < 1 || c->max_pages < 1 || (int64_t)c->max_pages * P > kMaxInt ||
        c->ld_pages < c->max_pages || c->token_stride < D || c->head_stride < D || c->page_stride < D ||
        c->token_stride > kMaxInt / 2 / P || c->page_stride > ((int64_t)1 << 40) || c->head_stride > ((int64_t)1 << 40))
        return MXGEMM_ERR_SHAPE;
    const int64_t unit = 16 / width;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || c->token_stride % unit || c->head_stride % unit || c->page_stride % unit ||
        !aligned(c->pages, 4) || !aligned(c->offsets, 4) || !aligned(c->lens, 4) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return MXGEMM_ERR_ALIGN;
    a.k = (uint8_t *)c->k;
    a.v = (uint8_t *)c->v;
    a.page_b = c->page_stride * width;
    a.head_b = c->head_stride * width;
    a.token_b = c->token_stride * width;
    a.pages = c->pages;
    a.ld_pages = c->ld_pages;
    a.offsets = c->offsets;
    a.lens = c->lens;
    a.k_scale = c->k_scale;
    a.v_scale = c->v_scale;
    a.num_pages = c->num_pages;
    a.page_shift = __builtin_ctz((unsigned)P);
    a.seqs = c->seqs;
    a.max_pages = c->max_pages;
    a.kv_heads = c->kv_heads;
    a.D = D;
    return MXGEMM_OK;
}

// Tiles of `tile` rows over all sequences and key heads, at most
int64_t most_units(int64_t T, int seqs, int group, int kv_heads, int tile)
{
    return kv_heads * ((T * group + std::min<int64_t>(T, seqs) * (tile - 1)) / tile);
}

// 32-row parts of the partial results of a call's workgroups (twice as many
// have room: a workgroup may leave two)
int64_t most_parts(int D) { return D > 128 ? 1024 : 2048; }

bool attention_shape(int T, int seqs, int heads, int kv_heads, int D)
{
    return T >= 1 && T <= kMaxTokens && seqs >= 1 && seqs <= kMaxSeqs && kv_heads >= 1 && heads >= kv_heads &&
           heads + 2 * kv_heads <= kMaxHeads && heads % kv_heads == 0 && (int64_t)T * heads <= kMaxRows && D >= 32 && D <= 256 && D % 32 == 0;
}

// Which kernel, and how its work is handed out.
//   - Few rows of a sequence and key head: the waves of a workgroup share 32 or 64
//     rows and take keys in turn.  Up to 512 rows (256 where 64 do not fit the
//     registers) this also holds where all rows would fill tiles of the other
//     kernel for less than a fifth of the compute units, although keys are then
//     read once per 64 rows: us, keys / rows kernel, 8 key heads of 4 query heads,
//     D = 128: 64 tokens over 32768 68 / 104, 100 over 8192 41 / 55, 8 x 16 over
//     16384 87 / 96, 128 over 32768 110 / 119, 4 x 48 over 8192 (48 tiles) 64 / 64,
//     but 3 x 100 over 8192 (75) 97 / 64, 8 x 48 (96) 127 / 83, 16 x 20 over 4096
//     (80) 73 / 59.
//     64 rows read the keys half as often, but a tile of them that is cut into many
//     parts takes long to add up by one workgroup: us, 32 / 64 rows, 40 rows of 64
//     heads over 16384 in 8 bits 42 / 36, 192 rows of 8 heads over 32768 75 / 65, but
//     128 rows over 8192 23 / 37 and 64 over 32768 43 / 58 (16 and 32 parts).
//   - Else tiles of 128 rows, two workgroups on a compute unit, or of 256 where
//     sequences have many new tokens and room for long contexts: us, 128 / 256 rows,
//     32 query and 8 key heads of 128: 512 tokens over 8192 98 / 91, 2048 over 30720
//     in 8 bits 1155 / 999, a prompt of 8192 561 / 541, but 8 prompts of 500 47 / 53,
//     512 tokens in a batch of 32 decoding ones over 4096 95 / 126.  (D <= 64: 128
//     rows always, 8000 tokens of 16 heads 68 / 80; D > 128: 128 rows of 4 waves.)
// MXGEMM_ATTENTION_KERNEL (0: keys, 32 rows; 1: keys, 64 rows; 2, 3: rows, smaller
// and larger tiles) is the tests' choice instead.
constexpr int kKeysFewRows = 64;
constexpr int kKeysRows = 512;
constexpr int kWideParts = 12;    // that a tile of 64 rows is cut into, at most
constexpr int kLargeRows = 1024;  // of a sequence and key head, on average
constexpr int kLargeKeys = 2048;  // that a sequence has room for

struct AttnChoice {
    mx::AttnLaunchFn launch;
    int plan, grid;
};
AttnChoice choose_attention(int T, int seqs, int G, int Hk, int D, bool fp8, int max_new, int64_t groups, int cu)
{
    const int64_t most_rows = (int64_t)(max_new > 0 ? std::min(max_new, T) : T) * G;
    const mx::AttnKeysKernel keys = mx::attn_keys_kernel(D, fp8);
    bool small = (int64_t)T * G < (int64_t)kLargeRows * seqs || groups * mx::kAttnGroup <= kLargeKeys;
    bool wide = most_rows > mx::kAttnTile && (int64_t)T * G * Hk * kWideParts >= (int64_t)2 * mx::kAttnTile * cu;
    bool few = most_rows <= kKeysFewRows ||
               (most_rows <= (keys.launch[1] ? kKeysRows : kKeysRows / 2) &&
                5 * (int64_t)T * G * Hk <= (int64_t)cu * mx::attn_rows_kernel(D, fp8, small).tile);
    if (const char *e = std::getenv("MXGEMM_ATTENTION_KERNEL")) {
        const int k = std::atoi(e);
        few = k < 2;
        wide = k == 1;
        small = k == 2;
    }
    if (few) {
        wide = wide && keys.launch[1];
        const int64_t tiles = most_units(T, seqs, G, Hk, wide ? 2 * mx::kAttnTile : mx::kAttnTile);
        // few units: one workgroup a compute unit (fewer parts to add: one token over
        // 32768 in 8 bits 19.5 us, with two 24)
        const bool parts = 2 * tiles <= cu;
        const int64_t wgs = std::min<int64_t>((int64_t)cu * (parts ? 1 : keys.per_cu[wide]), mx::kAttnPieces);
        return {keys.launch[wide], parts ? mx::kPlanParts : mx::kPlanLine, (int)std::min(tiles * groups, wgs)};
    }
    const mx::AttnRowsKernel rows = mx::attn_rows_kernel(D, fp8, small);
    const int64_t tiles = most_units(T, seqs, G, Hk, rows.tile);
    const int64_t wgs = std::min<int64_t>({(int64_t)cu * rows.per_cu, mx::kAttnPieces, most_parts(D) / (rows.tile / 32)});
    // (every sequence and key head may have a tile that is partly filled: more
    // workgroups, of 64 threads a tile's 32 rows, than a launch can have go in line)
    if (tiles >= 2 * wgs && tiles * 2 * rows.tile <= kMaxThreads)
        return {rows.launch, mx::kPlanWhole, (int)tiles};
    return {rows.launch, mx::kPlanLine, (int)std::min(tiles * groups, wgs)};
}

}  // namespace

extern "C" {

mxgemm_status mxgemm_rope_frequencies(double *freq, int rot_dim, double base, double factor, double original, double low,
                                      double high)
{
    if (!freq || !(base > 0.0) || !(factor > 0.0) || !std::isfinite(base) || !std::isfinite(factor))
        return MXGEMM_ERR_INVALID_ARG;
    if (rot_dim < 2 || rot_dim % 2 || rot_dim > 256)
        return MXGEMM_ERR_SHAPE;
    const bool parts = low != 0.0 || high != 0.0;
    if (parts && (!(original > 0.0) || !(low >= 0.0) || !(high > low) || !std::isfinite(original) || !std::isfinite(high)))
        return MXGEMM_ERR_INVALID_ARG;
    for (int i = 0; i < rot_dim / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / rot_dim);
        const double turns = original * f / 6.283185307179586476925;  // over the original context
        const double keep = parts ? std::min(1.0, std::max(0.0, (turns - low) / (high - low))) : 0.0;
        freq[i] = f * (keep + (1.0 - keep) / factor);
    }
    return MXGEMM_OK;
}

mxgemm_status mxgemm_kv_append(const mxgemm_kv_cache *cache, const mxgemm_append *p, int T, hipStream_t stream)
{
    if (!p || (!p->Q && !p->K) || (p->Q == nullptr) != (p->Q_out == nullptr) || (p->K == nullptr) != (p->V == nullptr) ||
        (p->interleaved != 0 && p->interleaved != 1) || (p->rot_dim > 0 && !p->freq))
        return MXGEMM_ERR_INVALID_ARG;
    mx::AppendArgs a = {};
    mxgemm_status st = check_cache(cache, p->K != nullptr, a.c);
    if (st != MXGEMM_OK)
        return st;
    const int D = cache->head_dim, Hk = cache->kv_heads, H = p->Q ? p->heads : 0;
    if (T < 1 || T > kMaxTokens || (p->Q && H < 1) || H > kMaxHeads || H + 2 * Hk > kMaxHeads || p->rot_dim < 0 || p->rot_dim > D || p->rot_dim % 16 ||
        (p->Q && (p->ldq < (int64_t)H * D || p->ldqo < (int64_t)H * D || (p->Q == p->Q_out && p->ldq != p->ldqo))) ||
        (p->K && (p->ldk < (int64_t)Hk * D || p->ldv < (int64_t)Hk * D)))
        return MXGEMM_ERR_SHAPE;
    if (!aligned(p->Q, 16) || !aligned(p->Q_out, 16) || !aligned(p->K, 16) || !aligned(p->V, 16) ||
        (p->Q && (p->ldq % 8 || p->ldqo % 8)) || (p->K && (p->ldk % 8 || p->ldv % 8)) || !aligned(p->positions, 4) ||
        !aligned(p->freq, 8))
        return MXGEMM_ERR_ALIGN;
    int cu = 0;
    st = mx::check_device(&cu);
    if (st != MXGEMM_OK)
        return st;
    a.Q = (const uint16_t *)p->Q;
    a.K = (const uint16_t *)p->K;
    a.V = (const uint16_t *)p->V;
    a.QO = (uint16_t *)p->Q_out;
    a.ldq = p->ldq;
    a.ldk = p->ldk;
    a.ldv = p->ldv;
    a.ldqo = p->ldqo;
    a.positions = p->positions;
    a.freq = p->freq;
    a.factor = p->factor;
    a.T = T;
    a.heads = H;
    a.rot = p->rot_dim;
    a.interleaved = p->interleaved;
    a.fp8 = cache->format == MXGEMM_KV_FP8_E4M3;
    mx::launch_append(a, cu, stream);
    return launched();
}

size_t mxgemm_paged_attention_workspace_bytes(int T, int seqs, int heads, int kv_heads, int head_dim)
{
    if (!attention_shape(T, seqs, heads, kv_heads, head_dim))
        return 0;
    return (size_t)(mx::kAttnCounterBytes + 2 * most_parts(head_dim) * mx::attn_partial_floats(head_dim) * 4);
}

mxgemm_status mxgemm_paged_attention(const mxgemm_kv_cache *cache, const mxgemm_attention *p, int T, void *workspace,
                                     size_t workspace_bytes, hipStream_t stream)
{
    if (!p || !p->Q || (!p->O && !p->A) || (p->A == nullptr) != (p->scaleA == nullptr) || (p->causal != 0 && p->causal != 1) ||
        !std::isfinite(p->scale))
        return MXGEMM_ERR_INVALID_ARG;
    const int bits = p->a_format == MXGEMM_FMT_FP4 ? 4 : p->a_format == MXGEMM_FMT_FP8_E4M3 ? 8 : 0;
    if (!bits)
        return MXGEMM_ERR_INVALID_ARG;
    mx::AttnArgs a = {};
    mxgemm_status st = check_cache(cache, true, a.c);
    if (st != MXGEMM_OK)
        return st;
    const int D = cache->head_dim, Hk = cache->kv_heads, H = p->heads;
    if (!attention_shape(T, cache->seqs, H, Hk, D) || p->window < 0 || p->max_new < 0 || p->ldq < (int64_t)H * D ||
        (p->O && (p->ldo < (int64_t)H * D || (p->O == p->Q && p->ldo != p->ldq))) || (p->A && (p->lda < (int64_t)H * D || p->ldsa < H * D / 32)))
        return MXGEMM_ERR_SHAPE;
    if (!aligned(p->Q, 16) || p->ldq % 8 || !aligned(p->O, 16) || (p->O && p->ldo % 8) || !aligned(p->lse, 4) ||
        !aligned(p->sinks, 4) || !aligned(p->A, 16) || (p->A && p->lda % (128 / bits)))
        return MXGEMM_ERR_ALIGN;
    const int G = H / Hk;
    const int64_t units = most_units(T, cache->seqs, G, Hk, mx::kAttnTile);
    const int64_t groups = cdiv((int64_t)cache->max_pages * cache->page_size, mx::kAttnGroup);
    // (the plan rounds the steps of all units up to whole workgroups in 32 bits)
    if (units > (kMaxInt - mx::kAttnPieces) / (groups + mx::kAttnUnitSteps))
        return MXGEMM_ERR_SHAPE;
    const size_t need = mxgemm_paged_attention_workspace_bytes(T, cache->seqs, H, Hk, D);
    if (!workspace || workspace_bytes < need)
        return MXGEMM_ERR_WORKSPACE;
    if (!aligned(workspace, 16))
        return MXGEMM_ERR_ALIGN;
    int cu = 0;
    st = mx::check_device(&cu);
    if (st != MXGEMM_OK)
        return st;
    a.Q = (const uint16_t *)p->Q;
    a.O = (uint16_t *)p->O;
    a.lse = p->lse;
    a.A = (uint8_t *)p->A;
    a.S = (uint8_t *)p->scaleA;
    a.sinks = p->sinks;
    a.ldq = p->ldq;
    a.ldo = p->ldo;
    a.lda_b = bits == 4 ? p->lda / 2 : p->lda;
    a.lds = p->ldsa;
    a.scale = p->scale;
    a.T = T;
    a.heads = H;
    a.group = G;
    a.by_group = mx::divisor(G);
    a.by_kv_heads = mx::divisor(Hk);
    a.causal = p->causal;
    a.window = p->window;
    a.a_fp8 = bits == 8;
    a.counters = (int *)workspace;
    a.partials = (float *)((uint8_t *)workspace + mx::kAttnCounterBytes);
    const bool fp8 = cache->format == MXGEMM_KV_FP8_E4M3;
    const AttnChoice k = choose_attention(T, cache->seqs, G, Hk, D, fp8, p->max_new, groups, cu);
    k.launch(a, k.plan, k.grid, stream);
    return launched();
}

}  // extern "C"
