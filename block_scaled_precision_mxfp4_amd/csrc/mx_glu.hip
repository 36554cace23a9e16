// Gated activation and quantizer on gfx950: v = bf16(silu(gate) * up) from
// rows [gate 0..K-1 | up K..2K-1] in bf16, and v's 32-blocks in MXFP4 or
// MXFP8, in one pass: v itself never reaches memory.
//
// silu(g) u = g u / (1 + e^-g).  v is the correctly rounded bf16 value, so
// that codes and scales do not depend on how the exponential was computed:
// the fp32 evaluation is within 6 units in its last place, and only where
// that leaves the bf16 rounding open (its low 16 bits within 8 of a half, 1
// element in 4000), or where its range does not carry it, the element is
// evaluated again in 64 bits.
//
// Bound by HBM: 4 bytes read and 17/32 (FP4) or 33/32 (FP8) byte written per
// element, each once.  Four lanes share a block and hold 8 elements each.
#include "mx_device.hpp"
#include "mx_experts.hpp"
#include "mx_quantize.hpp"

namespace mx {

__device__ __noinline__ float glu_f64(float g, float u)
{
    return f32_for_bf16((double)g / (1.0 + exp(-(double)g)) * (double)u);
}

__device__ __forceinline__ float glu_f32(float g, float u)
{
    // e^-g = 2^hi * (1 + lo ln 2): hi + lo = -g log2 e to twice fp32's bits
    const float c = -1.44269504088896341f, c_lo = -1.92596299112661746887e-8f;
    const float hi = g * c;
    const float lo = fmaf(g, c_lo, fmaf(g, c, -hi));
    float e = __builtin_amdgcn_exp2f(hi);
    e = fmaf(e, lo * 0.69314718055994531f, e);
    const float s = g * __builtin_amdgcn_rcpf(1.0f + e);
    const float v = s * u;
    const uint32_t low = __float_as_uint(v) & 0xFFFFu;
    // beyond |g| = 64 or below 2^-100 (also infinities and NaN) fp32 may lose
    // the value on the way
    const bool tiny = !(fabsf(s) >= 0x1p-100f) || !(fabsf(v) >= 0x1p-120f);
    const bool zero = v == 0.0f && (g == 0.0f || u == 0.0f);
    const bool open = low - 0x7FF8u <= 16u || !(fabsf(g) <= 64.0f) || (tiny && !zero);
    return open ? glu_f64(g, u) : v;
}

template <int U, bool FP8>
__global__ void __launch_bounds__(256) mx_glu_kernel(GluArgs q)
{
    const int j = threadIdx.x & 3, grp = threadIdx.x >> 2;
    const int kbn = q.K >> 5;
    const int64_t b0 = (int64_t)blockIdx.x * (64 * U) + grp;
    const int64_t live_rows = q.live ? min((int64_t)max(*q.live, 0), (int64_t)q.M) : q.M;
    int64_t row = b0 / kbn;
    int col = (int)(b0 - row * kbn);
    const int drow = 64 / kbn, dcol = 64 % kbn;
    v4i xg[U], xu[U];
    int64_t r[U];
    int kb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const bool on = row < live_rows;
        r[u] = on ? row : -1;
        kb[u] = col;
        const uint16_t *p = q.X + row * q.ldx + col * 32 + j * 8;
        xg[u] = on ? __builtin_nontemporal_load(reinterpret_cast<const v4i *>(p)) : v4i{0, 0, 0, 0};
        xu[u] = on ? __builtin_nontemporal_load(reinterpret_cast<const v4i *>(p + q.K)) : v4i{0, 0, 0, 0};
        row += drow;
        col += dcol;
        if (col >= kbn) {
            col -= kbn;
            ++row;
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        v4i v;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t g2 = (uint32_t)xg[u][w], u2 = (uint32_t)xu[u][w];
            const float lo = glu_f32(bf16_to_f32(g2 & 0xFFFFu), bf16_to_f32(u2 & 0xFFFFu));
            const float hi = glu_f32(bf16_to_f32(g2 >> 16), bf16_to_f32(u2 >> 16));
            v[w] = (int)bf16x2_rne(lo, hi);
        }
        // (a dead row's addresses are not used)
        const int64_t rr = r[u] < 0 ? 0 : r[u];
        quantize_store<FP8>(v, q.A + rr * q.lda_b, q.S + rr * q.lds, kb[u] * 32 + j * 8, r[u] >= 0);
    }
}

constexpr int kGluU = 2;
int64_t glu_grid(int64_t blocks) { return (blocks + 64 * kGluU - 1) / (64 * kGluU); }

void launch_glu(const GluArgs &g, hipStream_t s)
{
    const dim3 grid((unsigned)glu_grid(g.blocks));
    if (g.fp8)
        hipLaunchKernelGGL((mx_glu_kernel<kGluU, true>), grid, dim3(256), 0, s, g);
    else
        hipLaunchKernelGGL((mx_glu_kernel<kGluU, false>), grid, dim3(256), 0, s, g);
}

}  // namespace mx
