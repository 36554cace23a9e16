// Gated activation and quantizer on gfx950: v = bf16(silu(gate) * up) from
// rows [gate 0..K-1 | up K..2K-1] in bf16, and v's 32-blocks in MXFP4 or
// MXFP8, in one pass: v itself never reaches memory.
//
// silu(g) u = g u / (1 + e^-g).  v is that in 64 bits, rounded once to bf16, so
// that codes and scales do not depend on how the exponential was computed: it
// is evaluated in fp32, and again in 64 bits only where fp32's error leaves
// the bf16 rounding open (1 element in 4000) or its range does not carry it.
// (64 bits round as the exact value does, but where they leave 1 + e^-g at 1 or
// 2, g > 36 or |g| < 2^-50, and g u or g u / 2 is a tie between bf16 values.)
//
// Bound by HBM: 4 bytes read and 17/32 (FP4) or 33/32 (FP8) byte written per
// element, each once.  Four lanes share a block and hold 8 elements each.
#include "mx_device.hpp"
#include "mx_experts.hpp"
#include "mx_quantize_out.hpp"

namespace mx {

// The value in 64 bits.  Zeros of finite factors are what they are.
__device__ __noinline__ float glu_f64(float g, float u, float v)
{
    if (v == 0.0f && (g == 0.0f || u == 0.0f))
        return v;
    return f32_for_bf16((double)g / (1.0 + exp(-(double)g)) * (double)u);
}

// 8 values of a lane.  fp32's error: the argument of the exponential is kept
// to twice fp32's bits (hi + lo = -g log2 e), exp2 and rcp are within one unit
// in the last place, the five roundings around them half a unit each, so v is
// within 6 units.  `open`: the low 16 bits are within 8 units of a half, or |g|
// is above 64 (the exponential may overflow), or |g| or |v| below 2^-98 (fp32
// may lose bits on the way; for |g| <= 64 silu(g) is no smaller than |g| / 2 or
// 2^-87).  Infinite or NaN products are the same in both.  The 8 tests are
// made as one first: 1 group of 8 in 500 fails it.
__device__ __forceinline__ v4i glu_8(v4i xg, v4i xu)
{
    const float c = -1.44269504088896341f, c_lo = -1.92596299112661746887e-8f;
    constexpr uint32_t kNear = 16u << 16;
    float g[8], u[8], v[8];
    uint32_t near = 0xFFFFFFFFu;
    float most = 0.0f, least = 1.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t g2 = (uint32_t)xg[i >> 1], u2 = (uint32_t)xu[i >> 1];
        g[i] = __uint_as_float(i & 1 ? g2 & 0xFFFF0000u : g2 << 16);
        u[i] = __uint_as_float(i & 1 ? u2 & 0xFFFF0000u : u2 << 16);
        const float hi = g[i] * c;
        const float lo = fmaf(g[i], c_lo, fmaf(g[i], c, -hi));
        float e = __builtin_amdgcn_exp2f(hi);
        e = fmaf(e, lo * 0.69314718055994531f, e);
        v[i] = g[i] * __builtin_amdgcn_rcpf(1.0f + e) * u[i];
        near = min(near, (__float_as_uint(v[i]) - 0x7FF8u) << 16);
        most = fmaxf(most, fabsf(g[i]));
        least = fminf(least, fminf(fabsf(g[i]), fabsf(v[i])));
    }
    if (near <= kNear || most > 64.0f || least < 0x1p-98f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool open = (__float_as_uint(v[i]) - 0x7FF8u) << 16 <= kNear || !(fabsf(g[i]) <= 64.0f) ||
                              !(fminf(fabsf(g[i]), fabsf(v[i])) >= 0x1p-98f);
            if (open)
                v[i] = glu_f64(g[i], u[i], v[i]);
        }
    }
    v4i out;
#pragma unroll
    for (int w = 0; w < 4; ++w)
        out[w] = (int)bf16x2_rne(v[2 * w], v[2 * w + 1]);
    return out;
}

// A workgroup takes 64 blocks, one for each four lanes.  One block a lane
// group and a workgroup per 64, against 2 and 4 blocks: 32768 x 2048 67.3 us
// against 69.3 and 71.2 (FP4; 4.2 TB/s), 65.1 against 71.5 and 74.0 (FP8), 256 x
// 2048 4.4 against 6.1 and 9.6.
template <bool FP8>
__global__ void __launch_bounds__(256) mx_glu_kernel(GluArgs q)
{
    const int j = threadIdx.x & 3;
    const int64_t b = (int64_t)blockIdx.x * 64 + (threadIdx.x >> 2);
    const int kbn = q.K >> 5;
    const int64_t live_rows = q.live ? min((int64_t)max(*q.live, 0), (int64_t)q.M) : q.M;
    const int64_t row = (uint32_t)b / (uint32_t)kbn;  // (blocks: below 2^30)
    const int elem = (int)(b - row * kbn) * 32 + j * 8;
    const bool on = row < live_rows;
    v4i xg = {0, 0, 0, 0}, xu = xg;
    if (on) {
        const uint16_t *p = q.X + row * q.ldx + elem;
        xg = __builtin_nontemporal_load(reinterpret_cast<const v4i *>(p));
        xu = __builtin_nontemporal_load(reinterpret_cast<const v4i *>(p + q.K));
    }
    const int64_t r = on ? row : 0;  // (a dead row's addresses are not used)
    quantize_store<FP8>(glu_8(xg, xu), q.A + r * q.lda_b, q.S + r * q.lds, elem, on);
}

int64_t glu_grid(int64_t blocks) { return (blocks + 63) / 64; }

void launch_glu(const GluArgs &g, hipStream_t s)
{
    const dim3 grid((unsigned)glu_grid(g.blocks));
    if (g.fp8)
        hipLaunchKernelGGL(mx_glu_kernel<true>, grid, dim3(256), 0, s, g);
    else
        hipLaunchKernelGGL(mx_glu_kernel<false>, grid, dim3(256), 0, s, g);
}

}  // namespace mx
