// Device code that the attention kernels share: a sequence's extents, keys and
// values from pages into LDS, the products with a block of 32 keys, the
// running softmax, and what is done with a finished row.
//
// One wave holds 32 rows of queries (a row is one new token and one of the
// query heads that share a key head) and takes 32 keys at a time:
//
//   S^T[key][row] = K Q^T     v_mfma_f32_32x32x16_bf16, K first, Q second
//   O^T[d][row]  += V^T P^T   the same, V^T first, P^T second
//
// Both products have the row in the lane: lane l holds row l % 32, and of a
// block's 32 keys those with (key / 4) % 2 = l / 32 (accumulator g: key
// 8 (g / 4) + 4 (l / 32) + g % 4).  So the softmax of a row needs one exchange
// (the two lanes of a row), its maximum and sum are one register each, and P
// is the second product's operand where it stands: the order of the keys
// within a product's 16 is free as long as both operands have it, and V^T is
// read from LDS in P's order (transposed reads, whose rows each lane names).
//
// The scores are scaled by c = scale * k_scale * log2(e), p = 2^(c s - m).
// P is rounded to bf16 for the second product (up to 2^-8 of each p, which leaves
// the result about as far off as its own rounding to bf16 does: measured 0.0022 of
// the exact result's norm with both, 0.0017 with the last alone); the sum adds
// the unrounded p in fp32.  The running maximum is raised only where it grows
// by more than 8 (p up to 2^8): all of O would have to be rescaled otherwise.
#pragma once

#include "mx_attention.hpp"
#include "mx_pipe.hpp"
#include "mx_quantize_out.hpp"

namespace mx {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kNegInf = -__builtin_inff();
constexpr float kRaise = 8.0f;

template <int N>
__device__ __forceinline__ void attn_wait_vm()
{
    static_assert(N >= 0 && N < 64, "vmcnt range");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

template <int OFF>
__device__ __forceinline__ v2u lds_read_tr16(uint32_t base)
{
    static_assert(OFF >= 0 && OFF < 65536, "ds offset field");
    v2u r;
    asm volatile("ds_read_b64_tr_b16 %0, %1 offset:%2" : "=v"(r) : "v"(base), "n"(OFF) : "memory");
    return r;
}

template <int OFF>
__device__ __forceinline__ v2u lds_read_tr8(uint32_t base)
{
    static_assert(OFF >= 0 && OFF < 65536, "ds offset field");
    v2u r;
    asm volatile("ds_read_b64_tr_b8 %0, %1 offset:%2" : "=v"(r) : "v"(base), "n"(OFF) : "memory");
    return r;
}

__device__ __forceinline__ v16f mfma32(v4i a, v4i b, v16f c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// 8 E4M3 codes to 8 bf16 (exact)
__device__ __forceinline__ v4i bf16_of_fp8(v2u w)
{
    v4i r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r[i] = __builtin_bit_cast(int, (i & 1) ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i >> 1], 1.0f, true)
                                               : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i >> 1], 1.0f, false));
    return r;
}

// A value of the two lanes of a row combined
__device__ __forceinline__ float row_max(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float row_sum(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Read-only data at a wave-uniform address: scalar loads, also after asm that
// the compiler takes for a store.
__device__ __forceinline__ int load_uniform(const int32_t *p)
{
    return *(const __attribute__((address_space(4))) int32_t *)(uintptr_t)p;
}
__device__ __forceinline__ float load_uniform(const float *p)
{
    return *(const __attribute__((address_space(4))) float *)(uintptr_t)p;
}

__device__ __forceinline__ int quotient(int n, Divisor d) { return d.m ? (int)(__umulhi((uint32_t)n, d.m) >> d.shift) : n; }

// A row of a sequence: its new token, its query head
struct AttnRow {
    int token, head;
};
__device__ __forceinline__ AttnRow attn_row(const AttnArgs &a, int r, int kv_head)
{
    const int t = quotient(r, a.by_group);
    return {t, kv_head * a.group + (r - t * a.group)};
}

// ---- sequences

struct AttnSeq {
    int t0, n, len;  // first new token, new tokens, keys (whatever the arrays hold: within T and the page table)
};

__device__ __forceinline__ AttnSeq seq_from(const CacheArgs &c, int T, int o0, int o1, int len)
{
    o0 = min(max(o0, 0), T);
    o1 = min(max(o1, 0), T);
    return {o0, max(o1 - o0, 0), min(max(len, 0), c.max_pages << c.page_shift)};
}

// s wave-uniform
__device__ __forceinline__ AttnSeq load_seq(const CacheArgs &c, int T, int s)
{
    return seq_from(c, T, load_uniform(c.offsets + s), load_uniform(c.offsets + s + 1), load_uniform(c.lens + s));
}

// Blocks of `size` that hold n keys: a length may be as close to 2^31 as 16
__device__ __forceinline__ int key_blocks(int n, int size) { return (int)(((uint32_t)n + (uint32_t)(size - 1)) / (uint32_t)size); }

// Rows of a sequence, in tiles of `tile`; and the 128-key groups that a tile
// can need (an upper bound where a window moves with the tokens)
__device__ __forceinline__ int seq_tiles(const AttnSeq &q, int group, int tile) { return (q.n * group + tile - 1) / tile; }
__device__ __forceinline__ int seq_groups(const AttnArgs &a, const AttnSeq &q, int tile)
{
    int n = key_blocks(q.len, kAttnGroup);
    if (a.window > 0 && a.causal) {
        const int64_t most = (int64_t)a.window + tile / a.group + 1;
        n = (int)min((int64_t)n, (most + kAttnGroup - 1) / kAttnGroup + 1);
    }
    return max(n, 1);
}

// The first key that a token at position p sees (a window may be as long as an
// int is: p - window alone would wrap below 0, and so would a limit below 0 less
// the first key of a block)
__device__ __forceinline__ int first_key(const AttnArgs &a, int p)
{
    const int before = a.window > 0 ? a.window - 1 : 0x7FFFFFFF;  // keys before p that it sees
    return max(p, before) - before;
}

// Keys [lo, hi) that the tokens i0 .. i1 of a sequence can see between them
__device__ __forceinline__ void tile_keys(const AttnArgs &a, const AttnSeq &q, int i0, int i1, int &lo, int &hi)
{
    const int p0 = q.len - q.n + i0, p1 = q.len - q.n + i1;
    hi = a.causal ? min(max(p1 + 1, 0), q.len) : (p1 < 0 ? 0 : q.len);
    lo = min(first_key(a, p0), hi);
}

// ---- keys and values in LDS
//
// A row of DP elements is ROWB bytes of 16-byte chunks; load instructions fill
// 1 KiB, whole rows, so a chunk's place within its row is chosen by which
// chunk a lane loads.  K rows: chunk c at c ^ kswz(row): the 16 rows that a
// 16-byte read serves in one cycle fall on different banks.  V rows: 64-byte
// (bf16) or 32-byte (8 bits) pieces, piece p at p ^ vswz(row): a transposed
// read serves 4 rows x 64 bytes, or 8 rows x 32 bytes, at a time.
template <int DP, bool FP8>
struct AttnLds {
    static constexpr int ROWB = DP * (FP8 ? 1 : 2);
    static constexpr int CH = ROWB / 16;       // chunks of a row
    static constexpr int RPI = 1024 / ROWB;    // rows of a load instruction
    static constexpr int NIH = 16 / RPI;       // load instructions of 16 keys
    static constexpr int BLOCK = 32 * ROWB;    // 32 keys
    static constexpr int NS = DP / 16;         // products over d
    static constexpr int ND = DP / 32;         // blocks of O's columns
    static_assert(RPI >= 1 && NIH >= 1, "rows of 64 to 512 bytes");

    static __device__ __forceinline__ int kswz(int r)
    {
        return ROWB >= 256 ? r & 15 : ROWB == 128 ? (r >> 1) & 7 : (r >> 2) & 3;
    }
    static __device__ __forceinline__ int vswz(int r)
    {
        if constexpr (FP8)
            return ROWB >= 256 ? (r & 3) | ((r >> 1) & 4) : ROWB == 128 ? ((r >> 1) & 1) | ((r >> 2) & 2) : (r >> 3) & 1;
        else
            return ROWB >= 256 ? r & 3 : (r >> 1) & 1;
    }
    // chunk that stands at place c of row r
    static __device__ __forceinline__ int k_chunk(int r, int c) { return c ^ kswz(r); }
    static __device__ __forceinline__ int v_chunk(int r, int c) { return c ^ (vswz(r) * (FP8 ? 2 : 4)); }

    // this lane's byte offsets in 16 rows of the cache, by load instruction
    // (columns from D on lie outside every page: zeros)
    static __device__ __forceinline__ void load_offsets(const CacheArgs &c, int lane, uint32_t (&ko)[NIH], uint32_t (&vo)[NIH])
    {
        const int place = lane % CH;
#pragma unroll
        for (int j = 0; j < NIH; ++j) {
            const int r = j * RPI + lane / CH;
            const int kc = k_chunk(r, place) * 16, vc = v_chunk(r, place) * 16;
            const int row = c.D * (FP8 ? 1 : 2);
            ko[j] = kc < row ? (uint32_t)(r * c.token_b + kc) : kOOB;
            vo[j] = vc < row ? (uint32_t)(r * c.token_b + vc) : kOOB;
        }
    }

    // LDS addresses of this lane's K fragments of a block (bf16: product s,
    // columns 16 s + 8 (lane / 32) + 0..7; 8 bits: products 2 p and 2 p + 1,
    // columns 16 (2 p + lane / 32) + 0..7 and + 8..15): fragment s is at the
    // first one's address, its bits from 32 on changed by s
    static constexpr int KF = FP8 ? NS / 2 : NS;
    static __device__ __forceinline__ uint32_t k_first(uint32_t base, int lane)
    {
        const int r = lane & 31, h = lane >> 5;
        return base + r * ROWB + (h ^ kswz(r)) * 16;
    }
    static __device__ __forceinline__ uint32_t k_at(uint32_t first, int s) { return first ^ (uint32_t)(s * 32); }
    // ... and of its V^T fragments, likewise by block of 32 columns
    static __device__ __forceinline__ uint32_t v_first(uint32_t base, int lane)
    {
        const int h = lane >> 5, grp = (lane >> 4) & 1, q = lane & 15;
        if constexpr (FP8) {
            const int i = q >> 1, r = (i >> 2) * 8 + 4 * h + (i & 3);
            return base + r * ROWB + vswz(r) * 32 + grp * 16 + (q & 1) * 8;
        } else {
            const int r = 4 * h + (q >> 2);
            return base + r * ROWB + vswz(r) * 64 + grp * 32 + (q & 3) * 8;
        }
    }
    static __device__ __forceinline__ uint32_t v_at(uint32_t first, int d) { return first ^ (uint32_t)(d * (FP8 ? 32 : 64)); }
    // columns of this lane's Q fragment s
    static __device__ __forceinline__ int q_col(int s, int lane)
    {
        const int h = lane >> 5;
        return FP8 ? 16 * (2 * (s >> 1) + h) + 8 * (s & 1) : 16 * s + 8 * h;
    }
};

// 16 keys from key0 on: descriptors of K's and V's rows that exist (the others
// read as zeros).  k, v: the key head's rows in page 0.  page: as the table has it.
// Loads ahead of the last key may be past 2^31: they name key0 as the length too.
struct AttnRows {
    __amdgpu_buffer_rsrc_t k, v;
};
__device__ __forceinline__ AttnRows attn_rows(const CacheArgs &c, const uint8_t *k, const uint8_t *v, int page, uint32_t key0, uint32_t len)
{
    const bool there = (uint32_t)page < (uint32_t)c.num_pages;
    const int rows = there ? min(max((int)(len - key0), 0), 16) : 0;
    const int64_t at = (int64_t)(there ? page : 0) * c.page_b + (key0 & ((1u << c.page_shift) - 1)) * (uint32_t)c.token_b;
    const uint32_t bytes = (uint32_t)rows * (uint32_t)c.token_b;
    return {make_rsrc_u(k + at, bytes), make_rsrc_u(v + at, bytes)};
}

// A sequence's page table, 64 entries at a time in LDS (128 of a wave's own: the
// next 64 are on their way).  Loads into registers would be waited for with every
// load behind them still in flight; a scalar load is waited for with the LDS
// reads behind it.
struct AttnPages {
    static constexpr int LDS = 512;  // bytes
    __amdgpu_buffer_rsrc_t table;
    uint8_t *lds;
    int base, first;     // entry at lds[0]; first entry of the present 64
    __device__ __forceinline__ void load(int at, int lane)
    {
        load4_to_lds(table, (lds_void *)(lds + ((at - base) & 64) * 4), (uint32_t)(at + lane) * 4);
    }
    // (waits for every load of the wave); at: wave-uniform
    __device__ __forceinline__ void open(const CacheArgs &c, int s, int at, uint8_t *mine, int lane)
    {
        table = make_rsrc_u(c.pages + (int64_t)s * c.ld_pages, (uint32_t)c.max_pages * 4);  // (behind it: page 0)
        lds = mine;
        base = first = at;
        load(at, lane);
        load(at + 64, lane);
        attn_wait_vm<0>();
    }
    // Entries a and b >= a (both less than 64 behind the ones before); the read and
    // its wait are one piece, so that no value in flight is ever in a register
    __device__ __forceinline__ void get(int a, int b, int lane, int &page_a, int &page_b)
    {
        if (a >= first + 64) {
            first += 64;
            load(first + 64, lane);
        }
        const uint32_t at = lds_addr(lds), x = at + ((a - base) & 127) * 4, y = at + ((b - base) & 127) * 4;
        uint32_t r, s;
        asm volatile("ds_read_b32 %0, %2\n\tds_read_b32 %1, %3\n\ts_waitcnt lgkmcnt(0)"
                     : "=&v"(r), "=&v"(s)
                     : "v"(x), "v"(y)
                     : "memory");
        page_a = __builtin_amdgcn_readfirstlane((int)r);
        page_b = __builtin_amdgcn_readfirstlane((int)s);
    }
};

// x, as a value that is new here: what is computed from it is not moved out of
// the loop over units (the addresses of a unit's end, 70 registers, would be).
__device__ __forceinline__ int anew(int x)
{
    asm volatile("" : "+v"(x));
    return x;
}

// The kernel's arguments read again: fields that only the end of a unit needs
// would else be kept in scalar registers over its loop (100 of them spilled).
__device__ __forceinline__ AttnArgs args_again()
{
    const __attribute__((address_space(4))) AttnArgs *p =
        (const __attribute__((address_space(4))) AttnArgs *)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    AttnArgs a;
    __builtin_memcpy(&a, (const AttnArgs *)p, sizeof a);
    return a;
}

// ---- products and softmax

// This lane's Q fragments (its row's columns); zeros for rows and columns that
// do not exist.
template <int DP, bool FP8>
__device__ __forceinline__ void load_q(const AttnArgs &a, const uint16_t *row, bool live, int lane, v4i (&q)[DP / 16])
{
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) {
        const int col = AttnLds<DP, FP8>::q_col(s, lane);
        q[s] = v4i{0, 0, 0, 0};
        if (live && col < a.c.D)
            q[s] = *reinterpret_cast<const v4i *>(row + col);
    }
}
// Negated, where the scores' scale is negative
template <int NS>
__device__ __forceinline__ void negate_q(v4i (&q)[NS], bool negate)
{
    if (negate)
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                q[s][i] ^= (int)0x80008000;
}

// S^T of one block of 32 keys in LDS, for NT tiles of 32 rows
template <int DP, bool FP8, int NT>
__device__ __forceinline__ void scores(uint32_t ka, const v4i (&q)[NT][DP / 16],
                                       v16f (&s)[NT])
{
    using L = AttnLds<DP, FP8>;
#pragma unroll
    for (int n = 0; n < NT; ++n)
        s[n] = v16f{};
    constexpr int B = L::KF < 8 ? L::KF : 8;  // fragments read together
    static_for<L::KF / B>([&](auto bc) {
        v4i f[B];
#pragma unroll
        for (int i = 0; i < B; ++i)
            f[i] = lds_read16<0>(L::k_at(ka, bc.value * B + i));
        static_for<B / 2>([&](auto ic) {
            constexpr int I = 2 * ic.value;
            lds_wait_n<B - I - 2>(f[I], f[I + 1]);
#pragma unroll
            for (int i = I; i < I + 2; ++i) {
                const int k = bc.value * B + i;
                if constexpr (FP8) {
                    const v4i lo = bf16_of_fp8(v2u{(uint32_t)f[i][0], (uint32_t)f[i][1]});
                    const v4i hi = bf16_of_fp8(v2u{(uint32_t)f[i][2], (uint32_t)f[i][3]});
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        s[n] = mfma32(lo, q[n][2 * k], s[n]);
                        s[n] = mfma32(hi, q[n][2 * k + 1], s[n]);
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        s[n] = mfma32(f[i], q[n][k], s[n]);
                }
            }
        });
    });
}

// The running softmax's state of this lane's row
template <int ND>
struct AttnState {
    float m, l;  // maximum so far (of both lanes of the row), sum (this lane's keys)
    v16f o[ND];
    __device__ __forceinline__ void reset()
    {
        m = kNegInf;
        l = 0.0f;
#pragma unroll
        for (int d = 0; d < ND; ++d)
            o[d] = v16f{};
    }
};

// The running maximum raised to x (the scores' maximum over this lane's keys)
// where it has to be
template <int ND>
__device__ __forceinline__ void raise_to(AttnState<ND> &t, float x, float c)
{
    x = row_max(x) * c;
    if (__builtin_amdgcn_ballot_w64(x > t.m + kRaise)) {
        const float m = fmaxf(t.m, x);
        const float w = m == kNegInf ? 1.0f : exp2_fast(t.m - m);
        t.m = m;
        t.l *= w;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int g = 0; g < 16; ++g)
                t.o[d][g] *= w;
    }
}
template <int ND>
__device__ __forceinline__ void raise_max(AttnState<ND> &t, const v16f &s, float c)
{
    float x = s[0];
#pragma unroll
    for (int g = 1; g < 16; ++g)
        x = fmaxf(x, s[g]);
    raise_to(t, x, c);
}

// What p = 2^(c s - m) subtracts; a row that has seen no key yet: every score
// is -inf, p = 0
__device__ __forceinline__ float less_max(float m) { return m == kNegInf ? 0.0f : -m; }

// Scores 2 i and 2 i + 1 of a block to P (bf16 pairs, the second product's
// operands for its two steps of 16 keys), and to the sum.  (The results stay
// where they are written: the compiler would put them off until P is needed.)
template <int ND>
__device__ __forceinline__ void exponential_pair(AttnState<ND> &t, const v16f &s, int i, float c, float less, v4i (&p)[2])
{
    const float e0 = exp2_fast(fmaf(s[2 * i], c, less)), e1 = exp2_fast(fmaf(s[2 * i + 1], c, less));
    int w = (int)bf16x2_rne(e0, e1);
    t.l += e0 + e1;
    asm volatile("" : "+v"(w), "+v"(t.l));
    p[i >> 2][i & 3] = w;
}
template <int ND>
__device__ __forceinline__ void exponentials(AttnState<ND> &t, const v16f &s, float c, v4i (&p)[2])
{
    const float less = less_max(t.m);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        exponential_pair(t, s, i, c, less, p);
}

// V^T fragments of columns 32 d .. 32 d + 31, keys' step s (16 keys)
template <int DP, bool FP8>
struct AttnV {
    using L = AttnLds<DP, FP8>;
    v2u r[FP8 ? 1 : 2];
    template <int S>
    __device__ __forceinline__ void read(uint32_t at)
    {
        if constexpr (FP8) {
            r[0] = lds_read_tr8<S * 16 * L::ROWB>(at);
        } else {
            r[0] = lds_read_tr16<S * 16 * L::ROWB>(at);
            r[1] = lds_read_tr16<(S * 16 + 8) * L::ROWB>(at);
        }
    }
    static constexpr int N = FP8 ? 1 : 2;  // reads
    __device__ __forceinline__ v4i frag() const
    {
        if constexpr (FP8)
            return bf16_of_fp8(r[0]);
        else
            return v4i{(int)r[0][0], (int)r[0][1], (int)r[1][0], (int)r[1][1]};
    }
};

// whether a pair of bf16 holds an infinity or a NaN
__device__ __forceinline__ bool special_pair(int w)
{
    return (w & 0x7F80) == 0x7F80 || (w & 0x7F800000) == 0x7F800000;
}

// The products with V^T where it holds infinities or NaN and some rows do not
// see all keys: key by key, added to the rows that see it (0 times an infinity
// is a NaN: a p of 0 does not keep it out).
__device__ __forceinline__ void values_apart(const v4i (&w)[2], const v4i (&p)[2], int lo, int hi, int lane, v16f &o)
{
#pragma unroll 1
    for (int key = 0; key < 32; ++key) {
        // the key's slot: step key / 16, lane half (key / 4) % 2, element 4 ((key / 8) % 2) + key % 4
        const int e = 4 * ((key >> 3) & 1) + (key & 3);
        const int keep = ((key >> 2) & 1) == (lane >> 5) ? 0xFFFF << (16 * (e & 1)) : 0;
        v4i w1, p1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = i == (e >> 1) ? keep : 0;
            w1[i] = (key < 16 ? w[0][i] : w[1][i]) & k;
            p1[i] = (key < 16 ? p[0][i] : p[1][i]) & k;
        }
        const v16f x = mfma32(w1, p1, v16f{});
        const bool sees = key >= lo && key < hi;
#pragma unroll
        for (int g = 0; g < 16; ++g)
            o[g] += sees ? x[g] : 0.0f;
    }
}

// O^T += V^T P^T of one block, for NT tiles of 32 rows.  masked (wave-uniform):
// some rows do not see some of its keys; lo, hi: keys of the block that this
// lane's row of a tile sees.
template <int DP, bool FP8, int NT>
__device__ __forceinline__ void values(uint32_t va, const v4i (&p)[NT][2],
                                       AttnState<AttnLds<DP, FP8>::ND> (&t)[NT], bool masked, const int (&lo)[NT],
                                       const int (&hi)[NT], int lane)
{
    using L = AttnLds<DP, FP8>;
    using V = AttnV<DP, FP8>;
    constexpr int B = 2;  // blocks of columns read together
    static_for<L::ND / B>([&](auto bc) {
        constexpr int D0 = bc.value * B;
        V f[B][2];
#pragma unroll
        for (int i = 0; i < B; ++i) {
            f[i][0].template read<0>(L::v_at(va, D0 + i));
            f[i][1].template read<1>(L::v_at(va, D0 + i));
        }
        static_for<B>([&](auto ic) {
            constexpr int I = ic.value;
            lds_wait_n<(B - 1 - I) * 2 * V::N>(f[I][0].r, f[I][1].r);
            v4i w[2] = {f[I][0].frag(), f[I][1].frag()};
            if (masked) {
                bool special = false;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    special |= special_pair(w[e >> 2][e & 3]);
                if (__builtin_amdgcn_ballot_w64(special)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        values_apart(w, p[n], lo[n], hi[n], lane, t[n].o[D0 + I]);
                    w[0] = w[1] = v4i{0, 0, 0, 0};
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                t[n].o[D0 + I] = mfma32(w[0], p[n][0], t[n].o[D0 + I]);
                t[n].o[D0 + I] = mfma32(w[1], p[n][1], t[n].o[D0 + I]);
            }
        });
    });
}

// The scores of one block for one tile of 32 rows
template <int DP>
__device__ __forceinline__ v16f scores_one(uint32_t ka, const v4i (&q)[DP / 16])
{
    v16f s[1];
    scores<DP, false, 1>(ka, reinterpret_cast<const v4i (&)[1][DP / 16]>(q), s);
    return s[0];
}

// Scores outside a row's keys to -inf.  lo, hi: relative to the block.
__device__ __forceinline__ void mask_scores(v16f &s, int lo, int hi, int lane)
{
    const int h = 4 * (lane >> 5);
    lo -= h;  // (the limits are moved, not the keys: these stay constants)
    hi -= h;
#pragma unroll
    for (int g = 0; g < 16; ++g)
        s[g] = 8 * (g >> 2) + (g & 3) >= lo && 8 * (g >> 2) + (g & 3) < hi ? s[g] : kNegInf;
}

// The scale of a key head's scores, as a positive factor (in powers of two),
// whether Q is to be negated for it, and whether it is 0 (Q is then taken as
// 0 with a factor of 1: masked scores, -inf, must not meet a factor of 0).
struct AttnScale {
    float c;
    bool negate, zero;
};
__device__ __forceinline__ AttnScale attn_scale(const AttnArgs &a, int head)
{
    const float c = a.scale * kLog2e * (a.c.k_scale ? load_uniform(a.c.k_scale + head) : 1.0f);
    return {c == 0.0f ? 1.0f : fabsf(c), c < 0.0f, c == 0.0f};
}

// A finished row's 8 columns from col on: o relative to 2^m, l the sum; the
// sink's share joins the sum.  Every lane of a quad has the same row.
struct RowEnd {
    float f;    // O's factor
    float lse;
};
__device__ __forceinline__ RowEnd end_row(const AttnArgs &a, int kv_head, int head, float m, float l)
{
    float w = 1.0f;
    if (a.sinks) {
        const float k = a.sinks[head] * kLog2e, n = fmaxf(m, k);
        if (n != kNegInf || k != k) {  // (a NaN sink: NaN, also where no key is seen)
            w = exp2_fast(m - n);
            l = l * w + exp2_fast(k - n);
            m = n;
        }
    }
    const float vs = a.c.v_scale ? a.c.v_scale[kv_head] : 1.0f;
    return {l == 0.0f ? 0.0f : w / l * vs, l == 0.0f ? kNegInf : (m + __builtin_amdgcn_logf(l)) * kLn2};
}
__device__ __forceinline__ void store_row(const AttnArgs &a, int token, int head, int col, v4i x, bool live)
{
    if (live && a.O)
        *reinterpret_cast<v4i *>(a.O + (int64_t)token * a.ldo + head * a.c.D + col) = x;
    if (a.A) {
        uint8_t *A = a.A + (int64_t)token * a.lda_b, *S = a.S + (int64_t)token * a.lds;
        if (a.a_fp8)
            quantize_store<true>(x, A, S, head * a.c.D + col, live);
        else
            quantize_store<false>(x, A, S, head * a.c.D + col, live);
    }
}
template <typename F>
__device__ __forceinline__ void finish_row(const AttnArgs &a, int kv_head, int token, int head, int col, float m, float l,
                                           F &&o, bool live)
{
    const RowEnd e = end_row(a, kv_head, head, m, l);
    v4i x;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = (int)bf16x2_rne(o(2 * i) * e.f, o(2 * i + 1) * e.f);
    if (live && a.lse && col == 0)
        a.lse[(int64_t)token * a.heads + head] = e.lse;
    store_row(a, token, head, col, x, live);
}

// A wave's 32 finished rows from its registers, through `lds` (32 * DP * 2
// bytes of its own).  r0: the first row's number among the sequence's rows;
// rows: how many there are (at most 32); m, l of this lane's row, l of all its keys.
template <int DP>
__device__ __forceinline__ void finish_tile(const AttnArgs &a, const AttnSeq &q, int kv_head, int r0, int rows, float m,
                                            float l, const v16f (&o)[DP / 32], uint8_t *lds, int lane)
{
    constexpr int CH = DP / 8;  // 16-byte chunks of a row
    const int row = lane & 31, rr = r0 + min(row, rows - 1);
    const AttnRow at = attn_row(a, rr, kv_head);
    const int token = q.t0 + at.token, head = at.head;
    const RowEnd e = end_row(a, kv_head, head, m, l);
    if (a.lse && lane < rows)
        a.lse[(int64_t)token * a.heads + head] = e.lse;
    auto swz = [](int r) { return CH >= 16 ? r & 15 : (r >> 1) & 7; };
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int g = 0; g < 16; g += 4) {
            const int c = d * 4 + (g >> 2);
            v2u x;
            x[0] = bf16x2_rne(o[d][g] * e.f, o[d][g + 1] * e.f);
            x[1] = bf16x2_rne(o[d][g + 2] * e.f, o[d][g + 3] * e.f);
            *reinterpret_cast<v2u *>(lds + row * (DP * 2) + ((c ^ swz(row)) * 16) + (lane >> 5) * 8) = x;
        }
#pragma unroll
    for (int i = 0; i < 32 * CH / 64; ++i) {
        const int r = (i * 64 + lane) / CH, c = lane % CH;
        const v4i x = *reinterpret_cast<const v4i *>(lds + r * (DP * 2) + ((c ^ swz(r)) * 16));
        const AttnRow to = attn_row(a, r0 + min(r, rows - 1), kv_head);
        store_row(a, q.t0 + to.token, to.head, c * 8, x, r < rows && c * 8 < a.c.D);
    }
}

}  // namespace mx
