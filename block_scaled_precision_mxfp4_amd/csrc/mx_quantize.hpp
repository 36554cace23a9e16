// One 32-element block of a bf16 row -> MXFP4 (E2M1 codes + E8M0 scale),
// shared by the activation quantizer and the GEMV that quantizes its single
// A row on load.  The rule (OCP Microscaling Formats v1.0, section 6.3):
// scale exponent X = floor(log2 max|v|) - 2 clamped to [-127, 127]; each
// element v / 2^X rounded to the nearest E2M1 value, ties to the even
// mantissa, saturating at 6, sign kept; a block holding a NaN or an infinity
// gets scale 0xFF and codes 0.
#pragma once

#include "mx_device.hpp"

namespace mx {

// Encode one 32-block: x holds this lane's 8 bf16 (a quarter of the block);
// the four lanes of the block combine their maximum and NaN/inf flag.
__device__ __forceinline__ void quantize_quarter(v4i x, uint32_t &word, uint8_t &scale)
{
    // bf16 magnitude bits order like the values for finite inputs; an
    // all-ones exponent field is an infinity or a NaN
    uint32_t amag = 0, special = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t hb = ((uint32_t)x[w] >> (16 * h)) & 0xFFFFu;
            special |= (hb & 0x7F80u) == 0x7F80u;
            amag = max(amag, hb & 0x7FFFu);
        }
    }
    // the block's four lanes are one aligned quad: quad permutes (lane ^ 1,
    // lane ^ 2) exchange within it without going through LDS
    amag = max(amag, (uint32_t)__builtin_amdgcn_mov_dpp((int)amag, 0xB1, 0xF, 0xF, true));
    amag = max(amag, (uint32_t)__builtin_amdgcn_mov_dpp((int)amag, 0x4E, 0xF, 0xF, true));
    special |= (uint32_t)__builtin_amdgcn_mov_dpp((int)special, 0xB1, 0xF, 0xF, true);
    special |= (uint32_t)__builtin_amdgcn_mov_dpp((int)special, 0x4E, 0xF, 0xF, true);

    // floor(log2 amax) from the bf16 fields (subnormal: from the top set
    // mantissa bit), then the scale exponent
    int xs = -127;
    if (amag != 0) {
        const int ef = (int)(amag >> 7);
        const int fl = ef > 0 ? ef - 127 : -133 + (31 - __builtin_clz(amag & 0x7Fu));
        xs = min(127, max(-127, fl - 2));
    }
    word = 0;
    if (!special && xs > -127) {
        // v_cvt_scalef32_pk_fp4_bf16: two bf16 divided by the scale, rounded
        // to nearest even E2M1 with saturation at 6, sign kept -- the rule
        // above, measured equal on every finite input tried; one instruction
        // per pair, byte w of the word holds elements 2w (low nibble), 2w+1
        // (the pairs are formed from the whole 16 bytes viewed as eight
        // bf16: a bit cast of single extracted words was folded onto word 0)
        typedef __bf16 v2bf_t __attribute__((ext_vector_type(2)));
        typedef __bf16 v8bf_t __attribute__((ext_vector_type(8)));
        const v8bf_t e = __builtin_bit_cast(v8bf_t, x);
        const float sc = __uint_as_float((uint32_t)(xs + 127) << 23);  // 2^xs, a normal float
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(word, v2bf_t{e[0], e[1]}, sc, 0);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(word, v2bf_t{e[2], e[3]}, sc, 1);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(word, v2bf_t{e[4], e[5]}, sc, 2);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(word, v2bf_t{e[6], e[7]}, sc, 3);
    } else if (!special) {
        // scale 2^-127 is not a normal float: encode in software
#pragma unroll
        for (int w = 0; w < 4; ++w) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t hb = ((uint32_t)x[w] >> (16 * h)) & 0xFFFFu;
                const float s = ldexpf(__uint_as_float(hb << 16), -xs);  // exact scaling
                const float m = fabsf(s);
                uint32_t c;
                if (m >= 6.0f)
                    c = 7u;  // saturate (no E2M1 value above 6)
                else if (m < 2.0f)
                    c = (uint32_t)rintf(m * 2.0f);  // steps of 1/2: codes 0..4
                else if (m < 4.0f)
                    c = (uint32_t)rintf(m) + 2u;  // 2, 3, 4 -> codes 4, 5, 6
                else
                    c = (uint32_t)rintf(m * 0.5f) + 4u;  // 4, 6 -> codes 6, 7
                c |= (hb >> 12) & 8u;  // sign bit of the input
                word |= c << (4 * (2 * w + h));
            }
        }
    }
    scale = special ? (uint8_t)0xFF : (uint8_t)(xs + 127);
}

// The same block to MXFP8 (E4M3 codes, four a word): the largest E4M3 exponent
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
