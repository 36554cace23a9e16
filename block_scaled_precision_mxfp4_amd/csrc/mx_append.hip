// Rotary positions and the append to a paged cache (gfx950): queries and keys
// of new tokens are turned to their positions, queries written out, keys and
// values written into their pages, each read once.  Bound by HBM: 16384 tokens of
// 32 + 2 x 8 heads of 128, 403 MB read and written: 92 us, 4.4 TB/s (a large copy:
// 4.7).  One token takes 3.4 us, 509 tokens 6.2: latency of the search of the
// offsets, the positions, the angles and the rows, one after another.
//
// A workgroup has a few tokens.  One wave per token finds its sequence (a
// 64-way search of the offsets), its position and its page; the angles, which
// all heads share, are reduced in 64 bits (pos * freq in turns, less the whole
// turns: at position 2^20 a 32-bit angle is off by up to 1/16) and their
// cosines and sines kept in LDS; then every thread takes 16-byte pieces (half
// layout: a piece and its partner half a turned part further, by the same
// thread, so that Q may be turned in place).
#include "mx_attention.hpp"
#include "mx_device.hpp"

namespace mx {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;  // of a workgroup

struct AppendGeo {
    int tokens;                    // of a workgroup
    int q_units, k_units, v_units; // pieces (or pairs of them) of a head
    int per_token;                 // of a token, all heads
    uint32_t m_token, m_q, m_k, m_v;  // 2^32 / per_token, ... rounded up
};

// n / d for n * d < 2^32, with m = ceil(2^32 / d); d == 1: m is 0
__device__ __forceinline__ int quotient(int n, uint32_t m) { return m ? (int)__umulhi((uint32_t)n, m) : n; }

__device__ __forceinline__ float e4m3_range(float x) { return x > 448.0f ? 448.0f : x < -448.0f ? -448.0f : x; }  // (a NaN stays)

__device__ __forceinline__ void unpack(v4i x, float (&f)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f[i] = bf16_to_f32(((uint32_t)x[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
}

__device__ __forceinline__ v4i pack_bf16(const float (&f)[8])
{
    v4i r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r[i] = (int)bf16x2_rne(f[2 * i], f[2 * i + 1]);
    return r;
}

// 8 values over the scale to E4M3 codes: the quotient in fp32, then one
// rounding to nearest even; what is beyond 448 saturates, a NaN stays one
__device__ __forceinline__ v2u pack_fp8(const float (&f)[8], float scale)
{
    v2u r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q[i] = e4m3_range(__fdiv_rn(f[4 * h + i], scale));
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
        r[h] = (uint32_t)w;
    }
    return r;
}

struct Token {
    int64_t at;    // byte offset of its row in a page, head 0; -1: not written
    int32_t seen;  // whether it belongs to a sequence
};

template <bool FP8, bool PAIRS>  // PAIRS: interleaved layout
__global__ void __launch_bounds__(kThreads) mx_append_kernel(AppendArgs a, AppendGeo geo)
{
    extern __shared__ __attribute__((aligned(16))) float s_angle[];  // [token][cosines rot/2, sines rot/2]
    __shared__ Token s_tok[kMaxTokens];
    __shared__ double s_pos[kMaxTokens];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int t0 = blockIdx.x * geo.tokens, n = min(geo.tokens, a.T - t0);
    const CacheArgs &c = a.c;

    for (int i = wave; i < n; i += kThreads / 64) {
        const int t = t0 + i;
        // the last s with offsets[s] <= t, among S + 1 entries: 64 at a time
        int lo = 0, step = c.seqs + 1;
        while (step > 0) {
            const int width = step;  // entries lo .. lo + width - 1 are left
            step = (width + 63) / 64;
            const int at = lo + lane * step;
            const bool below = lane * step < width && c.offsets[at] <= t;
            const int upto = __popcll(__builtin_amdgcn_ballot_w64(below));
            if (upto == 0) {
                lo = -1;
                break;
            }
            lo += (upto - 1) * step;
            if (step == 1)
                break;
            step = min(step, width - (upto - 1) * step);
        }
        int pos = 0;
        Token k = {-1, 0};
        if (lo >= 0 && lo < c.seqs) {
            const int o0 = c.offsets[lo], o1 = c.offsets[lo + 1];
            if (t >= max(o0, 0) && t < o1) {
                const int len = min(max(c.lens[lo], 0), c.max_pages << c.page_shift);
                const int in = len - (min(o1, a.T) - t);  // its position in the cache
                k.seen = 1;
                pos = a.positions ? a.positions[t] : in;
                if (a.K && in >= 0) {
                    const int page = c.pages[(int64_t)lo * c.ld_pages + (in >> c.page_shift)];
                    if ((uint32_t)page < (uint32_t)c.num_pages)
                        k.at = (int64_t)page * c.page_b + (int64_t)(in & ((1 << c.page_shift) - 1)) * c.token_b;
                }
            }
        }
        if (lane == 0) {
            s_tok[i] = k;
            s_pos[i] = (double)pos;
        }
    }
    __syncthreads();
    const int half = a.rot / 2;
    for (int i = threadIdx.x; i < n * half; i += kThreads) {
        const int k = i / half, j = i - k * half;
        constexpr double kTurn = 0.15915494309189533577;  // 1 / (2 pi)
        const double turns = s_pos[k] * (a.freq[j] * kTurn);
        float sn, cs;
        sincospif(2.0f * (float)(turns - rint(turns)), &sn, &cs);
        s_angle[k * a.rot + j] = cs * a.factor;
        s_angle[k * a.rot + half + j] = sn * a.factor;
    }
    __syncthreads();

    for (int i = threadIdx.x; i < n * geo.per_token; i += kThreads) {
        const int k = quotient(i, geo.m_token);
        int u = i - k * geo.per_token;
        const Token tok = s_tok[k];
        const int64_t t = t0 + k;
        const float *angle = s_angle + k * a.rot;
        // which head, and which of its pieces
        const uint16_t *src;
        uint16_t *dst = nullptr;  // a row of bf16, or a place in a page
        uint8_t *page = nullptr;
        float scale = 1.0f;
        int h;
        bool turn = true;
        if (u < a.heads * geo.q_units) {
            h = quotient(u, geo.m_q);
            u -= h * geo.q_units;
            src = a.Q + t * a.ldq + h * c.D;
            dst = a.QO + t * a.ldqo + h * c.D;
            if (!tok.seen)
                continue;
        } else {
            if (tok.at < 0)
                continue;
            u -= a.heads * geo.q_units;
            if (u < c.kv_heads * geo.k_units) {
                h = quotient(u, geo.m_k);
                u -= h * geo.k_units;
                src = a.K + t * a.ldk + h * c.D;
                page = c.k + tok.at + h * c.head_b;
                if (FP8 && c.k_scale)
                    scale = c.k_scale[h];
            } else {
                u -= c.kv_heads * geo.k_units;
                h = quotient(u, geo.m_v);
                u -= h * geo.v_units;
                src = a.V + t * a.ldv + h * c.D;
                page = c.v + tok.at + h * c.head_b;
                if (FP8 && c.v_scale)
                    scale = c.v_scale[h];
                turn = false;
            }
        }
        auto store = [&](int col, const float (&f)[8], v4i bits, bool same) __attribute__((always_inline)) {
            if (dst)
                *reinterpret_cast<v4i *>(dst + col) = same ? bits : pack_bf16(f);
            else if constexpr (FP8)
                *reinterpret_cast<v2u *>(page + col) = pack_fp8(f, scale);
            else
                *reinterpret_cast<v4i *>(page + 2 * col) = same ? bits : pack_bf16(f);
        };
        float x[8], y[8];
        if constexpr (PAIRS) {
            const int col = u * 8;
            const v4i w = *reinterpret_cast<const v4i *>(src + col);
            unpack(w, x);
            const bool turned = turn && col < a.rot;
            if (turned) {
                const v4f cs = *reinterpret_cast<const v4f *>(angle + col / 2);
                const v4f sn = *reinterpret_cast<const v4f *>(angle + half + col / 2);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[2 * e] = fmaf(x[2 * e], cs[e], -(x[2 * e + 1] * sn[e]));
                    y[2 * e + 1] = fmaf(x[2 * e + 1], cs[e], x[2 * e] * sn[e]);
                }
                store(col, y, w, false);
            } else {
                store(col, x, w, true);
            }
        } else {
            const int pairs = turn ? half / 8 : 0;
            if (u < pairs) {
                const int col = u * 8;
                const v4i w0 = *reinterpret_cast<const v4i *>(src + col), w1 = *reinterpret_cast<const v4i *>(src + half + col);
                unpack(w0, x);
                unpack(w1, y);
                float p[8], q[8];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const v4f cs = *reinterpret_cast<const v4f *>(angle + col + 4 * b);
                    const v4f sn = *reinterpret_cast<const v4f *>(angle + half + col + 4 * b);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        p[4 * b + e] = fmaf(x[4 * b + e], cs[e], -(y[4 * b + e] * sn[e]));
                        q[4 * b + e] = fmaf(y[4 * b + e], cs[e], x[4 * b + e] * sn[e]);
                    }
                }
                store(col, p, w0, false);
                store(half + col, q, w1, false);
            } else {
                const int col = (u + pairs) * 8;  // (behind the turned part: 2 * pairs pieces)
                const v4i w = *reinterpret_cast<const v4i *>(src + col);
                unpack(w, x);
                store(col, x, w, true);
            }
        }
    }
}

uint32_t magic(int d) { return d > 1 ? (uint32_t)((((uint64_t)1 << 32) + d - 1) / d) : 0; }

}  // namespace

void launch_append(const AppendArgs &a, int num_cu, hipStream_t s)
{
    AppendGeo g;
    g.v_units = a.c.D / 8;
    g.k_units = a.interleaved ? a.c.D / 8 : a.c.D / 8 - a.rot / 16;
    g.q_units = g.k_units;
    const int heads = a.Q ? a.heads : 0;
    g.per_token = heads * g.q_units + (a.K ? a.c.kv_heads * (g.k_units + g.v_units) : 0);
    g.tokens = a.T >= 8 * kMaxTokens * num_cu ? kMaxTokens : a.T >= 32 * num_cu ? 4 : a.T >= 8 * num_cu ? 2 : 1;
    g.m_token = magic(g.per_token);
    g.m_q = magic(g.q_units);
    g.m_k = magic(g.k_units);
    g.m_v = magic(g.v_units);
    AppendArgs b = a;
    b.heads = heads;
    const int grid = (a.T + g.tokens - 1) / g.tokens;
    const size_t lds = (size_t)g.tokens * a.rot * 4;
    if (a.interleaved)
        a.fp8 ? mx_append_kernel<true, true><<<grid, kThreads, lds, s>>>(b, g) : mx_append_kernel<false, true><<<grid, kThreads, lds, s>>>(b, g);
    else
        a.fp8 ? mx_append_kernel<true, false><<<grid, kThreads, lds, s>>>(b, g) : mx_append_kernel<false, false><<<grid, kThreads, lds, s>>>(b, g);
}

}  // namespace mx
