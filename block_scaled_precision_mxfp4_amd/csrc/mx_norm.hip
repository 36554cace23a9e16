// The norms around a block on gfx950, one workgroup per token, one pass over
// memory:
//   y = sum_j weight_j * Y[pos_j]            (the experts' rows, or row t of Y)
//   n = y * rsqrt(mean(y^2) + eps) * w_post  (or y)
//   h = bf16(x + res_scale * gate * n)
//   z = bf16(h * rsqrt(mean(h^2) + eps) * w_pre)  (or h)
// and z's 32-blocks in MXFP4 or MXFP8 (the next product's A).
//
// A thread keeps its 8 C elements of the token in registers from the first
// load to the last store; the two means are sums over the workgroup.  All
// arithmetic between the bf16 inputs and the bf16 results is in 64 bits
// (products of bf16 values are exact there, and the multiply-add runs at
// fp32's rate on this chip): h and z are the correctly rounded values up to
// 2^-45 or so, whatever the order of the sums, so codes and scales do not
// flip with it.
//
// Bound by HBM: 2 (top_k + 1) bytes read and 4 + 17/32 (FP4) or 33/32 (FP8)
// written per element with every output asked for.
#include "mx_device.hpp"
#include "mx_experts.hpp"
#include "mx_quantize_out.hpp"
#include "mx_rows16.hpp"

namespace mx {

__device__ __forceinline__ double bf16_at(v4i x, int i)
{
    return (double)bf16_to_f32(((uint32_t)x[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
}

__device__ __forceinline__ double dpp_f64(double v, int step)
{
    const uint64_t u = __double_as_longlong(v);
    const uint32_t lo = row_partner((uint32_t)u, step), hi = row_partner((uint32_t)(u >> 32), step);
    return __longlong_as_double((int64_t)(((uint64_t)hi << 32) | lo));
}

// Sum over a wave, the same bits in every lane: four steps inside 16 lanes by
// row permutes, then the four rows' sums in order.
__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v += dpp_f64(v, i);
    const uint64_t u = __double_as_longlong(v);
    double t = 0.0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)u, 16 * r);
        const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(u >> 32), 16 * r);
        t += __longlong_as_double((int64_t)(((uint64_t)hi << 32) | lo));
    }
    return t;
}

// Sum over the workgroup, the same bits in every thread; s: NW doubles of its
// own (two sums in a row use different ones).
template <int NW>
__device__ __forceinline__ double block_sum(double v, double *s)
{
    v = wave_sum(v);
    if constexpr (NW == 1)
        return v;
    if ((threadIdx.x & 63) == 0)
        s[threadIdx.x >> 6] = v;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < NW; ++w)
        t += s[w];
    return t;
}

template <int NT, int C, bool FP8>
__global__ void __launch_bounds__(NT) mx_norm_kernel(NormArgs a)
{
    __shared__ double s_sum[2][NT / 64];
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x;
    const v4i zero = {0, 0, 0, 0};
    int e[C];
    bool on[C];
    v4i x[C], gate[C], wpost[C], wpre[C];
    double y[C][8];
    auto load = [&](const uint16_t *p, int c) __attribute__((always_inline)) {
        return on[c] && p ? *reinterpret_cast<const v4i *>(p + e[c]) : zero;
    };
#pragma unroll
    for (int c = 0; c < C; ++c) {
        e[c] = (c * NT + tid) * 8;
        on[c] = e[c] < a.K;
        x[c] = load(a.X ? a.X + t * a.ldx : nullptr, c);
        gate[c] = load(a.gate ? a.gate + t * a.ldg : nullptr, c);
        wpost[c] = load(a.w_post, c);
        wpre[c] = load(a.w_pre, c);
    }
    if (a.pos) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                y[c][i] = 0.0;
        // U rows at a time, all of their loads in flight together.  A row
        // that is not there reads as zeros (row 0 is read in its place: what
        // it holds does not matter, also a NaN).
        constexpr int U = C == 1 ? 4 : 2;
        for (int j0 = 0; j0 < a.top_k; j0 += U) {
            v4i r[U][C];
            double w[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int64_t at = t * a.top_k + min(j0 + i, a.top_k - 1);
                const int p = a.pos[at];
                const bool ok = j0 + i < a.top_k && (uint32_t)p < (uint32_t)a.y_rows;
                w[i] = (double)a.weights[at];
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    r[i][c] = load(a.Y + (int64_t)(ok ? p : 0) * a.ldy, c);
                    if (!ok)
                        r[i][c] = zero;
                }
                w[i] = ok ? w[i] : 0.0;
            }
#pragma unroll
            for (int i = 0; i < U; ++i)
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int x8 = 0; x8 < 8; ++x8)
                        y[c][x8] = fma(w[i], bf16_at(r[i][c], x8), y[c][x8]);
        }
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const v4i r = load(a.Y + t * a.ldy, c);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                y[c][i] = bf16_at(r, i);
        }
    }
    if (a.w_post) {
        double q = 0.0;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                q = fma(y[c][i], y[c][i], q);
        const double inv = 1.0 / sqrt(block_sum<NT / 64>(q, s_sum[0]) / a.K + (double)a.eps);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                y[c][i] *= inv * bf16_at(wpost[c], i);
    }
    const double scale = (double)a.res_scale;
    double q = 0.0;
    v4i h[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            float f[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int i = 2 * w + b;
                double n = y[c][i];
                if (a.gate)
                    n *= bf16_at(gate[c], i);
                f[b] = f32_for_bf16(fma(scale, n, bf16_at(x[c], i)));
            }
            h[c][w] = (int)bf16x2_rne(f[0], f[1]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            q = fma(bf16_at(h[c], i), bf16_at(h[c], i), q);
        if (a.H && on[c])
            *reinterpret_cast<v4i *>(a.H + t * a.ldh + e[c]) = h[c];
    }
    if (!a.Z && !a.A)
        return;
    if (a.w_pre) {
        const double inv = 1.0 / sqrt(block_sum<NT / 64>(q, s_sum[1]) / a.K + (double)a.eps);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float lo = f32_for_bf16(bf16_at(h[c], 2 * w) * inv * bf16_at(wpre[c], 2 * w));
                const float hi = f32_for_bf16(bf16_at(h[c], 2 * w + 1) * inv * bf16_at(wpre[c], 2 * w + 1));
                h[c][w] = (int)bf16x2_rne(lo, hi);
            }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (a.Z && on[c])
            *reinterpret_cast<v4i *>(a.Z + t * a.ldz + e[c]) = h[c];
        if (a.A)
            quantize_store<FP8>(h[c], a.A + t * a.lda_b, a.S + t * a.lds, e[c], on[c]);
    }
}

template <int NT, int C>
static void launch_norm_as(const NormArgs &n, hipStream_t s)
{
    if (n.fp8)
        hipLaunchKernelGGL((mx_norm_kernel<NT, C, true>), dim3((unsigned)n.T), dim3(NT), 0, s, n);
    else
        hipLaunchKernelGGL((mx_norm_kernel<NT, C, false>), dim3((unsigned)n.T), dim3(NT), 0, s, n);
}

int norm_threads(int K) { return K <= 512 ? 64 : K <= 4096 ? 256 : K <= 8192 ? 512 : 1024; }

// Up to one token per compute unit a workgroup twice as wide, 8 elements a
// thread: its latency is what counts (1 x 4096, top 4: 4.6 against 5.6 us). For
// more tokens 16 a thread (8192 x 4096: 96.9 us with top 4, 5.2 TB/s, and 58.3
// without, against 101.4 and 64.8 us; 32 a thread: 124.6 and 73.7).
void launch_norm(const NormArgs &n, int num_cu, hipStream_t s)
{
    const bool wide = n.T <= num_cu;
    if (n.K <= 512)
        launch_norm_as<64, 1>(n, s);
    else if (n.K <= 2048)
        launch_norm_as<256, 1>(n, s);
    else if (n.K <= 4096)
        wide ? launch_norm_as<512, 1>(n, s) : launch_norm_as<256, 2>(n, s);
    else if (n.K <= 8192)
        wide ? launch_norm_as<1024, 1>(n, s) : launch_norm_as<512, 2>(n, s);
    else
        launch_norm_as<1024, 2>(n, s);
}

}  // namespace mx
