// Quantized outputs of the mixture-of-experts kernels: MXFP4 by the activation
// quantizer's routine (mx_quantize.hpp) or MXFP8, from values that are rounded
// to bf16 first.
#pragma once

#include "mx_quantize.hpp"

namespace mx {

// quantize_quarter's block to MXFP8 (E4M3 codes, four a word): the largest E4M3 exponent
// is 8, so X = floor(log2 max|v|) - 8, and v / 2^X lies below 512; beyond 448
// it saturates.  The scaling is exact (a power of two of a normal float; what
// underflows rounds to zero in E4M3 anyway) and the conversion rounds once,
// to nearest even.
__device__ __forceinline__ void quantize_quarter_fp8(v4i x, v2u &words, uint8_t &scale)
{
    uint32_t amag = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w)
        amag = max(amag, max((uint32_t)x[w] & 0x7FFFu, ((uint32_t)x[w] >> 16) & 0x7FFFu));
    amag = max(amag, (uint32_t)__builtin_amdgcn_mov_dpp((int)amag, 0xB1, 0xF, 0xF, true));
    amag = max(amag, (uint32_t)__builtin_amdgcn_mov_dpp((int)amag, 0x4E, 0xF, 0xF, true));
    const bool special = amag >= 0x7F80u;  // the largest magnitude is an infinity or a NaN
    int xs = -127;
    if (amag != 0) {
        const int ef = (int)(amag >> 7);
        const int fl = ef > 0 ? ef - 127 : -133 + (31 - __builtin_clz(amag & 0x7Fu));
        xs = max(-127, fl - 8);
    }
    const float inv = __uint_as_float((uint32_t)(127 - xs) << 23);  // 2^-xs, -127 <= xs <= 119
    words = v2u{0, 0};
    if (!special) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t hb = ((uint32_t)x[2 * h + (i >> 1)] >> (16 * (i & 1))) & 0xFFFFu;
                f[i] = fminf(fmaxf(bf16_to_f32(hb) * inv, -448.0f), 448.0f);
            }
            int w = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
            w = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], w, true);
            words[h] = (uint32_t)w;
        }
    }
    scale = special ? (uint8_t)0xFF : (uint8_t)(xs + 127);
}

// 8 bf16 (a lane's quarter of a block) to codes at A + elem (FP4: elem / 2)
// and, from the first lane of the four, the scale at S + elem / 32.
template <bool FP8>
__device__ __forceinline__ void quantize_store(v4i x, uint8_t *A, uint8_t *S, int elem, bool live)
{
    uint8_t scale;
    if constexpr (FP8) {
        v2u w;
        quantize_quarter_fp8(x, w, scale);
        if (live)
            __builtin_nontemporal_store(w, reinterpret_cast<v2u *>(A + elem));
    } else {
        uint32_t w;
        quantize_quarter(x, w, scale);
        if (live)
            __builtin_nontemporal_store(w, reinterpret_cast<uint32_t *>(A + elem / 2));
    }
    if (live && (elem & 24) == 0)
        S[elem / 32] = scale;
}

// A value in 64 bits to fp32 such that a following rounding to bf16 is the
// value's own: fp32's rounding may land exactly halfway between two bf16
// values, where the tie rule would decide what the value's lower bits should.
__device__ __forceinline__ float f32_for_bf16(double d)
{
    const float f = (float)d;
    uint32_t u = __float_as_uint(f);
    if ((u & 0xFFFFu) == 0x8000u && (double)f != d)
        u += fabs(d) > fabs((double)f) ? 1u : 0xFFFFFFFFu;
    return __uint_as_float(u);
}

}  // namespace mx
