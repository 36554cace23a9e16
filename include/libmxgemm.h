/*
 * libmxgemm — MXFP4 block-scaled GEMM for AMD Instinct MI355X (gfx950).
 *
 *     D[M,N] = bf16( alpha * A[M,K] * B[N,K]^T + beta * C[M,N] )
 *
 * A and B hold OCP E2M1 (fp4) codes packed two per byte; every run of 32
 * consecutive K elements of a row carries one E8M0 scale byte.  This is the
 * problem the asm_f4gemm README ("asm_f4gemm -- driving aiter's gfx950
 * MXFP4 GEMM code objects") states at its top; operand formats follow its
 * section "Data layouts":
 *
 *   A      [M][lda/2] bytes, row-major.  Byte i of a row holds element 2i in
 *          its low nibble and element 2i+1 in its high nibble.  A code's
 *          value is one of {0, .5, 1, 1.5, 2, 3, 4, 6}, sign in bit 3.
 *   B      [N][ldb/2] bytes, same encoding (B is used transposed: D = A B^T).
 *   scaleA [M][ldsa] bytes: scaleA[i][k/32] is the E8M0 scale of A[i][k];
 *          its value is 2^(e-127) (0xFF is NaN).
 *   scaleB [N][ldsb] bytes, likewise for B.
 *   C, D   [M][ldc], [M][ldd] bf16, row-major.
 *
 * Arithmetic: the scaled products are accumulated in fp32 by the CDNA4
 * scaled matrix instructions ("CDNA4 dense MFMA builtins", section
 * "Mixed-precision with scaling"), partial sums of a split K are added in
 * fp32 in a fixed order, and the epilogue forms alpha*acc + beta*C in fp32
 * and rounds once to bf16 (nearest, ties to even).  When beta == 0, C is not
 * read (it may be NULL and may hold NaNs).
 *
 * Every pointer passed to libmxgemm is a DEVICE pointer on the current HIP
 * device, owned by the caller; the library never frees, retains or
 * reallocates caller memory.  All calls are asynchronous on `stream` (NULL
 * means the null stream) and return after enqueueing.  No call throws or
 * aborts: every failure is a negative status code.  Argument validation
 * happens on the host before any HIP call is made.
 */
#ifndef LIBMXGEMM_H
#define LIBMXGEMM_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ------------------------------------------------------- */

typedef int mxgemm_status;

#define MXGEMM_OK                      0
#define MXGEMM_ERR_INVALID_ARG        -1  /* NULL pointer, bad split_k, C == NULL with beta != 0, ... */
#define MXGEMM_ERR_SHAPE              -2  /* M, N < 1; K < 32; K % 32 != 0; K > 2^24; stride < extent */
#define MXGEMM_ERR_ALIGN              -3  /* A/B base not 16-byte aligned, or row pitch lda/2, ldb/2 not a multiple of 16 bytes */
#define MXGEMM_ERR_UNSUPPORTED_DEVICE -4  /* current device is not gfx950 */
#define MXGEMM_ERR_HIP                -5  /* a HIP runtime call failed (launch, allocation) */
#define MXGEMM_ERR_WORKSPACE          -6  /* caller workspace smaller than mxgemm_query's workspace_bytes */
#define MXGEMM_ERR_SCRATCH            -7  /* mxgemm_run_noalloc: the plan needs more than its fixed scratch */

/* Static string naming a status code (never NULL). */
const char *mxgemm_status_string(mxgemm_status status);

/* ---- strides and options --------------------------------------------------- */

/*
 * Row strides of the operands.  Passing NULL for the whole struct means
 * dense rows: ldd = ldc = N, lda = ldb = K, ldsa = ldsb = K/32, b_packed = 0,
 * library-owned workspace.
 *
 * The fully packed form (b_packed = sa_packed = 1: pre-shuffled B, shuffled
 * scaleA and scaleB, row-major A) is the operand set of the asm_f4gemm
 * README's pre-shuffled kernels ("Data layouts") and the fastest one: the
 * kernels read every shuffled scale word with contiguous loads.
 *
 * Units follow the asm_f4gemm README ("Kernel ABI", kernarg notes): A and B
 * strides count fp4 ELEMENTS (twice the byte pitch) and must be even; scale
 * strides count bytes; C and D strides count elements of their type.  ldc
 * and ldd are honoured separately, so D may alias C (in place) when ldc ==
 * ldd and C is bf16.
 *
 * The option fields at the end default to 0 (a zeroed struct):
 *   a_format   A's element format, MXGEMM_FMT_*: FP4 E2M1 (the default),
 *              FP8 E4M3, BF8 E5M2, FP6 E2M3 or FP6 E3M2 -- the inputs of the
 *              scaled matrix instructions ("CDNA4 dense MFMA builtins",
 *              "Mixed-precision with scaling"; encodings per the OCP MX
 *              v1.0 specification).  B stays FP4.  A row is a little-endian
 *              bit stream of the format's w-bit codes (element k at bits
 *              k*w .. k*w+w-1; for FP4 the low-nibble-first bytes), one E8M0
 *              scale per 32 elements as for FP4.  lda counts elements of
 *              A's format; the byte pitch lda*w/8 must be a whole multiple of
 *              16 (of 8 for the FP6 formats, whose dense rows are 24 bytes
 *              per 32 elements).  Kernels: for M == 1 the GEMV where it
 *              applies (kernel family 4), else for M <= 16 the
 *              skinny kernel, and for 16 < M <= 64 the rows kernel (all at
 *              the speed of
 *              the FP4 case; FP6 on the rows kernel needs an even K/32);
 *              otherwise, for M > 16, the 8-bit formats run on the tiled
 *              kernel with 8-bit A tiles, and FP6 A is first re-laid,
 *              codes unchanged, in a library-owned buffer per (device,
 *              stream), allocated on first use like the split-K buffers
 *              and freed by mxgemm_release_workspaces: on large shapes
 *              into the scaled instruction's operand order (24 bytes per
 *              lane, 1536 bytes per 16 rows and 128 K; its A scales
 *              shuffled beside it, and a row-major B and its scales packed
 *              as mxgemm_pack_b packs them) for a 256 x 256 FP6 tile,
 *              otherwise into 32-byte slots per 32-element block (rows of
 *              K bytes rounded up to 128) for the 8-bit tiles; both pass
 *              the FP6 operand format to the instruction, which runs it at
 *              its FP4 rate (when 256 re-laid rows reach 2^31 bytes, once
 *              per 16 rows on the skinny kernel instead).  Needs
 *              sa_packed = 0 and split_mode = MXGEMM_SPLIT_FP32 (else
 *              MXGEMM_ERR_INVALID_ARG); size a caller workspace with
 *              mxgemm_query_ex.
 *   c_f32      C is float32 instead of bf16.  The README's "C / bias" note
 *              says aiter documents its bias operand as f32; with c_f32 = 1
 *              the epilogue reads that type (D stays bf16; one rounding of
 *              alpha*acc + beta*C, computed in fp32).
 *   split_mode MXGEMM_SPLIT_FP32: split-K partials are fp32 sums added in a
 *              fixed order (deterministic; the default).
 *              MXGEMM_SPLIT_BF16_ATOMIC: each K chunk adds bf16(alpha *
 *              partial) into D with packed bf16 atomic adds, onto D first
 *              set to bf16(beta * C), the reduction the README's kernels use
 *              ("Verification": split-K accumulates in bf16).  Offered only
 *              to measure that reduction's error against the fp32 one: the
 *              result is rounded once per chunk and its bits depend on the
 *              order the chunks arrive in.  It runs on the tiled kernel
 *              (the skinny kernels are never chosen), needs D 4-byte
 *              aligned, ldd and N even (else MXGEMM_ERR_ALIGN), and D must
 *              not alias C.  With split 1 it is the ordinary path.
 *   b_layout   MXGEMM_B_NK: B as above ([N][ldb/2] rows, or mxgemm_pack_b's
 *              layout with b_packed = 1).  MXGEMM_B_KN: B's codes are
 *              stored MN-major, [K][ldb/2] bytes: row k holds the codes of
 *              the N columns at that k, element n in the low nibble of byte
 *              n/2 when n is even (a weight kept as W[K][N]).  ldb then
 *              counts fp4 elements between K-rows: ldb >= N, even, ldb/2 a
 *              multiple of 16 bytes.  scaleB stays one byte per column and
 *              32-block of k: [N][ldsb] with b_packed = 0, or
 *              mxgemm_pack_scales' shuffle of it over the N rows with
 *              b_packed = 1 (the codes are never pre-shuffled in this
 *              layout).  The tiled kernel reads such a B from LDS with the
 *              4-bit transposed loads of "CDNA4 MFMA transpose load
 *              builtins" (ds_read_tr4_b64, two per 16 x 128 operand, K
 *              split as that page's "Hardware constraints" table gives),
 *              for every M.  Needs a_format = MXGEMM_FMT_FP4 (else
 *              MXGEMM_ERR_INVALID_ARG); mxgemm_run_bf16a then quantizes
 *              first also at M = 1.
 */
#define MXGEMM_SPLIT_FP32        0
#define MXGEMM_SPLIT_BF16_ATOMIC 1

#define MXGEMM_B_NK 0  /* B [N][ldb/2]: row n holds its K codes (K-major) */
#define MXGEMM_B_KN 1  /* B [K][ldb/2]: row k holds the N columns' codes (MN-major) */

#define MXGEMM_FMT_FP4      0  /* E2M1, 4 bits */
#define MXGEMM_FMT_FP8_E4M3 1  /* 8 bits */
#define MXGEMM_FMT_FP8_E5M2 2  /* 8 bits */
#define MXGEMM_FMT_FP6_E2M3 3  /* 6 bits */
#define MXGEMM_FMT_FP6_E3M2 4  /* 6 bits */

typedef struct mxgemm_strides {
    int64_t ldd;      /* bf16 elements between rows of D, >= N */
    int64_t ldc;      /* elements between rows of C, >= N (ignored if beta == 0) */
    int64_t lda;      /* elements between rows of A (fp4 unless a_format says otherwise), >= K */
    int64_t ldb;      /* fp4 elements between rows of B, >= K (>= N for MXGEMM_B_KN), even
                         (ignored if b_packed with MXGEMM_B_NK) */
    int64_t ldsa;     /* bytes between rows of scaleA, >= K/32 */
    int64_t ldsb;     /* bytes between rows of scaleB, >= K/32 (ignored if b_packed) */
    int32_t b_packed; /* 0: B, scaleB row-major as above; 1: outputs of mxgemm_pack_b */
    int32_t sa_packed; /* 0: scaleA row-major as above; 1: output of mxgemm_pack_scales
                          for the M rows of A (ldsa ignored; needs b_packed = 1) */
    void *workspace;  /* optional device buffer for split-K partials; NULL = library-owned */
    size_t workspace_bytes;
    int32_t c_f32;      /* 0: C is bf16; 1: C is float32 */
    int32_t split_mode; /* MXGEMM_SPLIT_FP32 or MXGEMM_SPLIT_BF16_ATOMIC */
    int32_t a_format;   /* MXGEMM_FMT_* */
    int32_t b_layout;   /* MXGEMM_B_NK (B's rows hold K) or MXGEMM_B_KN (B's rows hold N) */
    int32_t a_packed;   /* 0: A and scaleA as above; 1: an FP6 A (a_format MXGEMM_FMT_FP6_*)
                           and its scales as mxgemm_pack_a wrote them (lda, ldsa and
                           sa_packed ignored; M > 64, where the dense FP6 tile runs; not
                           with mxgemm_run_bf16a): the call skips its re-layout of A */
} mxgemm_strides;

/* ---- the GEMM ------------------------------------------------------------- */

/*
 * D = bf16(alpha * A * B^T + beta * C).  Enqueued on `stream`.
 *
 * split_k: 0 or -1 lets the library choose (the "-1 lets the heuristic try"
 *          convention of the asm_f4gemm CLI, section "Build and run");
 *          1 = no split; 2, 4, 8 or 16 = split the K range into that many
 *          chunks whose fp32 partial sums are added in a fixed order (the
 *          result is bitwise reproducible run to run).  Other values:
 *          MXGEMM_ERR_INVALID_ARG.  Chunks are whole units of 256 K (tiled
 *          kernel, M > 64) or 512 K (skinny kernels, M <= 64); a split that
 *          needs smaller chunks is reduced to the number of such units
 *          (mxgemm_query reports the split used).
 *
 * Shapes: M, N >= 1; K >= 32, K % 32 == 0, K <= 2^24.  M and N need not be
 * multiples of any tile size and K need not be a multiple of 128: edges are
 * handled inside the kernels (no caller padding as in the asm_f4gemm README's
 * "D -- output" note).
 *
 * Alignment: A and B base addresses 16-byte aligned and lda/2, ldb/2 (the
 * byte pitches) multiples of 16.  Scales, C and D need only natural
 * alignment (D and a bf16 C: 2 bytes; an f32 C: 4 bytes).
 *
 * Split-K (split_k > 1, chosen or forced) keeps fp32 partial sums in a
 * workspace of mxgemm_query(...).workspace_bytes.  With strides->workspace
 * == NULL the library allocates one per (device, stream) on first use and
 * keeps it until mxgemm_release_workspaces(); a caller workspace must be at
 * least that size and must not be used by two calls that can run
 * concurrently.  The per-tile arrival counters of split-K are always
 * library-owned: one zeroed buffer per (device, stream), allocated on first
 * use and returned to all-zero by every call.  The first call with a new
 * (device, stream) or a larger need therefore allocates; calls on one
 * stream are ordered, calls on different streams use separate buffers.
 */
mxgemm_status mxgemm_run(void *D, const void *C, const void *A, const void *B,
                         const void *scaleA, const void *scaleB,
                         float alpha, float beta, int M, int N, int K,
                         const mxgemm_strides *strides, int split_k,
                         hipStream_t stream);

/* ---- allocation-free GEMM ------------------------------------------------------ */

/*
 * For callers that cannot allocate device memory: code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc.
 *
 * mxgemm_run with every library-owned buffer taken from one fixed device
 * array per GPU of MXGEMM_NOALLOC_SCRATCH_BYTES (32 MiB), which the library
 * holds from load until the process ends: the split-K arrival counters
 * (first 64 KiB: 4 bytes per output tile of a split plan), the split-K fp32
 * partials unless strides->workspace brings them, and the re-laid copy of
 * an FP6 A on the tiled kernels (M * K bytes, K rounded up to 128, on the
 * 8-bit tiles; about 3/4 of that plus M * K / 32 scale bytes on the FP6
 * tile, plus N * K * 17/32 bytes when B is row-major).  Same
 * arguments, plans, kernels and results as
 * mxgemm_run, bit for bit.  Never calls hipMalloc or hipFree (the first call
 * on a device looks up that device's array once).  A plan that needs more
 * than the array holds returns MXGEMM_ERR_SCRATCH before any launch;
 * mxgemm_query_ex gives the plan's workspace_bytes.
 *
 * Every call on one GPU shares that GPU's array, which keeps the last call's
 * contents; each call clears the counters it uses (with a kernel on
 * `stream`) before its GEMM.  Calls that can overlap on one GPU (on
 * different streams, or from host threads without ordering) race on the
 * array and must not be issued; calls ordered on one stream are safe.
 */
#define MXGEMM_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)

mxgemm_status mxgemm_run_noalloc(void *D, const void *C, const void *A, const void *B,
                                 const void *scaleA, const void *scaleB,
                                 float alpha, float beta, int M, int N, int K,
                                 const mxgemm_strides *strides, int split_k,
                                 hipStream_t stream);

/* ---- B pre-shuffle ----------------------------------------------------------- */

/*
 * Rewrite B [N][ldb/2] and scaleB [N][ldsb] into the layout the kernels read
 * directly (b_packed = 1).  The byte permutation is the "16x16
 * tile-transposed" B shuffle of the asm_f4gemm README ("Data layouts", B):
 *
 *   B[n0*16 + n1][k-byte k0*32 + k1*16 + k2]
 *       -> Bp[(((n0 * Kp/32 + k0) * 2 + k1) * 16 + n1) * 16 + k2],
 *
 * with Kp = (K rounded up to 128)/2 bytes and N rounded up to 16 rows, so
 * that every 1 KiB of Bp is one matrix-instruction operand (16 rows x 128
 * K), and the scale shuffle of the same section (its "A_scale / B_scale"
 * part), over scaleB padded to [N rounded up to 32][K/32 rounded up to 8]:
 *
 *   scaleB[d0*32 + d1*16 + d2][d3*8 + d4*4 + d5]
 *       -> SBp[((((d0 * sn/8 + d3) * 4 + d5) * 16 + d2) * 2 + d4) * 2 + d1],
 *
 * sn = padded K/32.  Padding bytes are code 0 for Bp and 0x7F (2^0) for SBp.
 * Bp and SBp are caller buffers of mxgemm_query's packed_b_bytes and
 * packed_sb_bytes; they must not overlap B or scaleB.  Bp 16-byte aligned,
 * SBp 4-byte aligned, B as for mxgemm_run.  Same shape rules as mxgemm_run.
 */
mxgemm_status mxgemm_pack_b(void *Bp, void *SBp, const void *B, const void *scaleB,
                            int N, int K, int64_t ldb, int64_t ldsb,
                            hipStream_t stream);

/*
 * Shuffle a [rows][K/32] E8M0 scale matrix (row pitch lds bytes) into the
 * layout of the asm_f4gemm README's "A_scale / B_scale" part of "Data
 * layouts" -- the same transform mxgemm_pack_b applies to scaleB -- for use
 * as scaleA with sa_packed = 1 (rows = M).  Sp is a caller buffer of
 * ceil(rows/32)*32 * ceil(K/256)*8 bytes (mxgemm_info.packed_sa_bytes for
 * rows = M), 4-byte aligned, not overlapping S; padding bytes are 0x7F.
 * Shape rules as mxgemm_run with rows in place of M.
 */
mxgemm_status mxgemm_pack_scales(void *Sp, const void *S, int rows, int K, int64_t lds,
                                 hipStream_t stream);

/*
 * An FP6 A (a_format MXGEMM_FMT_FP6_E2M3 or _E3M2; the layout does not depend
 * on which) and its scales, put once into the order the dense FP6 tile reads:
 * what mxgemm_run does to a row-major FP6 A on every call with M > 64
 * (for an A used in several calls, or written that way by its producer).
 * Codes: per 16-row group of A and 128-K step, 1536 bytes in the scaled
 * matrix instruction's operand order ("CDNA4 dense MFMA builtins",
 * "Mixed-precision with scaling": lane l holds row l%16, K-block l/16 of the
 * step, 24 bytes of FP6 codes, unchanged), steps padded to an even count,
 * groups in order; rows past M and blocks past K/32 are code 0.  Scales:
 * mxgemm_pack_scales' shuffle of scaleA (padding 0x7F).  A: [M][lda] FP6
 * elements (byte pitch lda*6/8 a multiple of 8; A 16-byte aligned);
 * scaleA: [M][ldsa] bytes.  Ap: mxgemm_pack_a_bytes(M, K) bytes, 16-byte
 * aligned; SAp: ceil(M/32)*32 * ceil(K/256)*8 bytes (packed_sa_bytes),
 * 4-byte aligned; neither overlaps A or scaleA.  Pass Ap as A and SAp as
 * scaleA to mxgemm_run with a_packed = 1.  Asynchronous on `stream`; errors
 * as mxgemm_run (MXGEMM_ERR_INVALID_ARG for another a_format).
 */
mxgemm_status mxgemm_pack_a(void *Ap, void *SAp, const void *A, const void *scaleA, int M, int K,
                            int64_t lda, int64_t ldsa, int a_format, hipStream_t stream);

/* Bytes of mxgemm_pack_a's Ap for an M x K FP6 A (0 for an invalid shape). */
size_t mxgemm_pack_a_bytes(int M, int K);

/* ---- activation quantizer -------------------------------------------------------- */

/*
 * Quantize a bf16 matrix X [M][ldx] (row-major, ldx in bf16 elements) to the
 * operand format of A: packed E2M1 codes A [M][lda/2] bytes (lda in fp4
 * elements, element 2i in the low nibble of byte i) and E8M0 scales
 * scaleA [M][ldsa] bytes, one per 32 consecutive K elements (asm_f4gemm
 * README, "Data layouts").  The outputs can be passed to mxgemm_run as A and
 * scaleA.
 *
 * The pages fix the encodings but not how a scale is chosen for real input;
 * the conversion follows the OCP Microscaling Formats v1.0 specification,
 * section 6.3: per 32-block, scale = 2^X with X = floor(log2 max|x|) - 2
 * clamped to [-127, 127]; each element is x / 2^X rounded to the nearest
 * E2M1 value (ties to the even mantissa), magnitudes beyond 6 saturate to 6,
 * the sign is kept (a negative value rounding to zero gives code 0x8).  A
 * block holding a NaN or an infinity gets scale 0xFF and codes 0; an all-zero
 * block gets scale 0x00 and codes 0.  The result is exact (deterministic and
 * independent of launch shape): every decision is taken on exactly scaled
 * values.
 *
 * Shapes: M >= 1; K >= 32, K % 32 == 0, K <= 2^24; ldx >= K, lda >= K,
 * ldsa >= K/32 (else MXGEMM_ERR_SHAPE).  Alignment (else MXGEMM_ERR_ALIGN):
 * X 16-byte aligned with ldx % 8 == 0; A 16-byte aligned with lda even and
 * lda/2 a multiple of 16 (the rule mxgemm_run applies to A); scaleA any.
 * X must not overlap A or scaleA.  Only the first K elements of each X row
 * are read and only the first K/2 bytes of each A row and K/32 bytes of each
 * scaleA row are written.  Asynchronous on `stream`; allocates nothing.
 */
mxgemm_status mxgemm_quantize(void *A, void *scaleA, const void *X, int M, int K,
                              int64_t ldx, int64_t lda, int64_t ldsa, hipStream_t stream);

/*
 * D = bf16(alpha * Q(X) * B^T + beta * C), where X is a bf16 activation
 * matrix [M][ldx] (row-major, ldx in bf16 elements, 16-byte aligned rows:
 * ldx % 8 == 0, X 16-byte aligned, ldx >= K) and Q is mxgemm_quantize's
 * encoding -- the activation-side quantizer in front of the GEMM.  B,
 * scaleB, C, D, strides (ldd, ldc, ldb, ldsb, b_packed, c_f32, workspace)
 * and split_k as for mxgemm_run; strides->lda / ldsa are ignored, and
 * a_format, sa_packed and split_mode must be 0 (else
 * MXGEMM_ERR_INVALID_ARG).
 *   M == 1 (decode), K-major B: one launch.  The skinny kernel loads the
 *     bf16 row and quantizes each 32-block in registers with the quantizer's
 *     rule, so D is bit for bit what mxgemm_quantize followed by mxgemm_run
 *     gives where mxgemm_run plans the skinny kernel too; where it plans the
 *     single-row GEMV (kernel family 4, another K order) the two agree
 *     within the fp32 accumulation's rounding.
 *   M > 1, or an MN-major B (b_layout = MXGEMM_B_KN): mxgemm_quantize into a library-owned buffer of
 *     M*K/2 + M*K/32 bytes per (device, stream) (allocated on first use like
 *     the split-K buffers, freed by mxgemm_release_workspaces), then
 *     mxgemm_run on it, both on `stream`.
 * Asynchronous on `stream`; errors as mxgemm_run.
 */
mxgemm_status mxgemm_run_bf16a(void *D, const void *C, const void *X, const void *B, const void *scaleB,
                               float alpha, float beta, int M, int N, int K, int64_t ldx,
                               const mxgemm_strides *strides, int split_k, hipStream_t stream);

/* ---- FP16 GEMM with transposed LDS reads ---------------------------------- */

/*
 * C = A * B with A [M, K] fp16 row-major, B [K, N] fp16 row-major (K-major:
 * row k holds the N columns of that k) and C [M, N] fp32: the FP16 GEMM of
 * "CDNA4 MFMA transpose load builtins" ("FP16 GEMM example"), whose B
 * fragments are read from LDS with ds_read_tr16_b64 (a hardware 16-bit
 * transpose) because B is stored K-major.  Products are exact in fp32 and
 * accumulate in fp32 inside the v_mfma_f32_16x16x32_f16 instructions.
 *
 * Strides count elements: lda >= K, ldb >= N, ldc >= N.  Shapes: M, N, K
 * >= 1, K and N multiples of 8 (whole 16-byte chunks of the rows of A and
 * B), 256 * lda * 2 and K * ldb * 2 below 2^31 bytes.  A, B base 16-byte
 * aligned, lda and ldb multiples of 8; C 4-byte aligned.  Errors:
 * MXGEMM_ERR_INVALID_ARG (NULL pointer), MXGEMM_ERR_SHAPE, MXGEMM_ERR_ALIGN,
 * all before any HIP call.  Asynchronous on `stream`; allocates nothing.
 */
mxgemm_status mxgemm_f16_run(void *C, const void *A, const void *B, int M, int N, int K,
                             int64_t lda, int64_t ldb, int64_t ldc, hipStream_t stream);

/* ---- mixture of experts ------------------------------------------------------- */

/*
 * The feed-forward of a mixture of experts over MXFP4 weights, in four
 * operators that hand their device buffers on without a host copy:
 *
 *   mxgemm_route           router logits -> experts, weights, rows by expert
 *   mxgemm_grouped_run     each expert's rows times its B (gate and up)
 *   mxgemm_glu_quantize    silu(gate) * up -> the next product's A
 *   mxgemm_grouped_run     each expert's rows times its B (down)
 *   mxgemm_norm_quantize   weighted sum of a token's expert rows, norms around
 *                          the block, gate, residual -> the next block's A
 *
 * Forward only, like the rest of the library (4-bit weights for serving).
 * None of them allocates, reads back or keeps anything: all can be captured
 * into a graph, and calls that share no output or workspace can overlap.
 * Quantized outputs are MXFP4 (a_format MXGEMM_FMT_FP4, mxgemm_quantize's
 * rule) or MXFP8 (MXGEMM_FMT_FP8_E4M3: X = floor(log2 max|x|) - 8 clamped to
 * [-127, 127], elements to the nearest E4M3 value, ties to even, saturating
 * at 448; the special blocks as for MXFP4): rows of lda elements of the
 * format, the byte pitch a multiple of 16, and ldsa scale bytes, as
 * mxgemm_run takes them.  Another a_format: MXGEMM_ERR_INVALID_ARG.
 */

/*
 * The router's choice.  logits [T][ldl] (float32, or bf16 with bf16 = 1), E
 * experts, 1 <= E <= 1024, 1 <= top_k <= min(E, 16); T * top_k < 2^31.
 *
 *   ids [T][top_k]      the experts of the top_k largest logits, largest
 *                       first, equal logits by the lower expert.  A logit of
 *                       -inf or NaN is never chosen; slots left over: -1.
 *   weights [T][top_k]  exp(l - max) / sum in float32, the sum over the
 *                       token's chosen experts (renorm = 1) or over all its
 *                       logits that may be chosen (renorm = 0).  A logit of
 *                       +inf shares the token's weight with its equals.
 *                       Slots left over: 0.
 *   offsets [E + 1]     expert e's rows are offsets[e] .. offsets[e+1] - 1;
 *                       offsets[E] counts the routed (token, slot) pairs.
 *   rows [T * top_k]    rows[i] = the token of row i; an expert's rows are in
 *                       the order of their tokens.  From offsets[E] on: -1.
 *   pos [T][top_k]      the row of (token, slot): rows[pos[t][j]] = t; -1 for
 *                       slots left over.
 *
 * workspace: mxgemm_route_workspace_bytes(T, E) bytes (0 for T <= 64: it may
 * be NULL), 4-byte aligned, not shared by calls that can overlap; at most
 * 4 * E * ceil(T / 64).  The outputs do not overlap each other or the logits.
 * Deterministic.  Errors: MXGEMM_ERR_INVALID_ARG (NULL, a flag that is not 0
 * or 1), MXGEMM_ERR_SHAPE, MXGEMM_ERR_ALIGN (natural alignment),
 * MXGEMM_ERR_WORKSPACE, all before any HIP call.
 */
mxgemm_status mxgemm_route(int32_t *ids, float *weights, int32_t *pos, int32_t *offsets, int32_t *rows,
                           const void *logits, int bf16, int T, int E, int top_k, int64_t ldl, int renorm,
                           void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Bytes of mxgemm_route's workspace (0: none needed, or an invalid shape). */
size_t mxgemm_route_workspace_bytes(int T, int E);

/* Row strides and options of mxgemm_grouped_run, units as in mxgemm_strides.
 * NULL for the whole struct: dense rows, ldd = N, lda = ldb = K, ldsa = ldsb =
 * K/32, strideb = N * K, strideb_scale = N * K/32, FP4 A. */
typedef struct mxgemm_grouped {
    int64_t ldd;           /* bf16 elements between rows of D, >= N */
    int64_t lda;           /* elements between rows of A (of a_format), >= K */
    int64_t ldsa;          /* bytes between rows of scaleA, >= K/32 */
    int64_t ldb;           /* fp4 elements between rows of an expert's B, >= K */
    int64_t ldsb;          /* bytes between rows of an expert's scaleB, >= K/32 */
    int64_t strideb;       /* fp4 elements from one expert's B to the next's, >= 0 (0: one B for all) */
    int64_t strideb_scale; /* bytes from one expert's scaleB to the next's, >= 0 */
    int32_t a_format;      /* MXGEMM_FMT_FP4 or MXGEMM_FMT_FP8_E4M3 */
} mxgemm_grouped;

/*
 * The product grouped by expert, in one launch: for every expert e and every
 * row i with offsets[e] <= i < offsets[e+1],
 *
 *     D[i][n] = bf16( alpha * sum_k A[r(i)][k] * B[e][n][k] ),
 *
 * r(i) = a_rows[i] with a row list (mxgemm_route's rows: the tokens' A is read
 * in place, no copy is made per expert), else i.  offsets [groups + 1] and
 * a_rows [rows] are device arrays of int32; the host knows only rows, the
 * rows of D (an upper bound of offsets[groups]).  Rows of D that no expert
 * has, those from offsets[groups] on among them, are not written.  Experts
 * without rows cost nothing.  Sums are in fp32 inside the scaled matrix
 * instructions (with an 8-bit A these first add 8 products, aligned to the
 * largest and kept to 13 bits below its exponent); deterministic.
 *
 * Operands as for mxgemm_run: A [a_count][lda] MXFP4 or MXFP8 E4M3 with
 * scaleA, B [groups][N][ldb] MXFP4 with scaleB, row-major.  a_count: the rows
 * of A (>= rows without a row list).  offsets have to ascend; whatever they
 * hold, no address outside the buffers is formed (they are clamped to [0,
 * rows]), and a row index outside [0, a_count) reads as a row of zeros.
 *
 * Shapes: rows, a_count, N >= 1; rows <= 2^30; 1 <= groups <= 65535; K >= 32,
 * K % 32 == 0, K <= 2^24; 256 rows of A, of B and of a scale matrix, and with a
 * row list all of A and of scaleA, below 2^31 bytes; fewer than 2^23 tiles, the
 * smallest of 32 x 128 elements of D (else MXGEMM_ERR_SHAPE).  Alignment: A, B
 * 16-byte aligned, the byte pitches of A, B and strideb multiples of 16; D 2
 * bytes, offsets and a_rows 4 bytes.  D must not overlap an input.
 * Asynchronous on `stream`; errors as mxgemm_run.
 */
mxgemm_status mxgemm_grouped_run(void *D, const void *A, const void *B, const void *scaleA, const void *scaleB,
                                 const int32_t *offsets, const int32_t *a_rows, float alpha, int rows, int a_count,
                                 int N, int K, int groups, const mxgemm_grouped *strides, hipStream_t stream);

/*
 * Gated activation and quantizer in one pass: X [M][ldx] bf16 holds a row's
 * gate values in columns 0 .. K-1 and its up values in K .. 2K-1 (the output
 * of a product with both weights, N = 2K);
 *
 *     v = bf16( gate / (1 + e^-gate) * up ),    (A, scaleA) = quantized v,
 *
 * v rounded once from 64 bits, to nearest even, so that the result does not
 * depend on the launch's shape or on how the exponential was computed.  That
 * is the exact value's rounding but for one case: where 64 bits leave 1 +
 * e^-gate at 1 or 2 (gates above 36, or nearer to 0 than 2^-50) and gate * up, or
 * half of it, lies in the middle between two bf16 values, the tie may decide
 * instead of what the exact value is beside it.  A gate or up that is infinite
 * or NaN makes v what IEEE arithmetic makes it (-inf / inf: NaN); its block then
 * has scale 0xFF and codes 0.
 *
 * live: NULL, or a device int32 (offsets + groups, say): only rows below *live
 * (clamped to [0, M]) are read and written.  Shapes: M >= 1, K >= 32, K % 32
 * == 0, K <= 2^24, M * K < 2^35, ldx >= 2K.  X 16-byte aligned, ldx % 8 == 0; live 4-byte
 * aligned.  X must not overlap the outputs.  Asynchronous on `stream`.
 */
mxgemm_status mxgemm_glu_quantize(void *A, void *scaleA, const void *X, const int32_t *live, int M, int K, int64_t ldx,
                                  int64_t lda, int64_t ldsa, int a_format, hipStream_t stream);

/*
 * The norms around a block: per token t
 *
 *     y = sum_j weights[t][j] * Y[pos[t][j]]       (top_k > 0; else row t of Y)
 *     n = y * w_post / sqrt(mean(y^2) + eps)       (w_post NULL: n = y)
 *     h = bf16( X[t] + res_scale * gate * n )
 *     z = bf16( h * w_pre / sqrt(mean(h^2) + eps) )  (w_pre NULL: z = h)
 *
 * to H (the residual stream), Z and, quantized, A with scaleA; each of the
 * three may be NULL, not all.  The arithmetic between the bf16 inputs and the
 * two roundings is in 64 bits.  pos entries outside [0, y_rows) add nothing
 * (mxgemm_route's -1), whatever their weights and Y hold: a token that no
 * expert took has y = 0.
 */
typedef struct mxgemm_norm {
    const void *Y;        /* bf16 [y_rows][ldy] (top_k > 0) or [T][ldy] */
    int64_t ldy;
    const int32_t *pos;   /* [T][top_k], dense; NULL with top_k == 0 */
    const float *weights; /* [T][top_k], dense; NULL with top_k == 0 */
    int32_t top_k;        /* rows of Y summed per token, at most 1024; 0: row t of Y itself */
    int32_t y_rows;       /* rows of Y (used with top_k > 0) */
    const void *w_post;   /* bf16 [K] or NULL */
    const void *gate;     /* bf16 [T][ldg], or one row for all with ldg == 0; NULL: 1 */
    int64_t ldg;
    const void *X;        /* residual, bf16 [T][ldx]; NULL: 0 */
    int64_t ldx;
    float res_scale;
    float eps;            /* > 0 */
    void *H;              /* bf16 [T][ldh] or NULL; may be X (ldh == ldx), or Y with top_k == 0 (ldh == ldy) */
    int64_t ldh;
    const void *w_pre;    /* bf16 [K] or NULL */
    void *Z;              /* bf16 [T][ldz] or NULL; may be Y with top_k == 0 (ldz == ldy) */
    int64_t ldz;
    void *A;              /* [T][lda] codes or NULL */
    void *scaleA;         /* [T][ldsa] scale bytes; NULL with A */
    int64_t lda, ldsa;
    int32_t a_format;     /* MXGEMM_FMT_FP4 or MXGEMM_FMT_FP8_E4M3 */
} mxgemm_norm;

/*
 * T >= 1 tokens of K elements, K % 32 == 0, 32 <= K <= 16384 (a token is kept
 * in one workgroup's registers), T below 2^22 (K <= 512: 2^26, K <= 4096:
 * 2^24, K <= 8192: 2^23).  bf16 pointers 16-byte aligned, their
 * strides multiples of 8; A as in mxgemm_glu_quantize.  Apart from the places
 * named above no output overlaps an input or another output.  Errors:
 * MXGEMM_ERR_INVALID_ARG (NULL n or Y, no output, A without scaleA or the
 * other way round, pos or weights without top_k or the other way round, eps
 * not above 0, another a_format), MXGEMM_ERR_SHAPE, MXGEMM_ERR_ALIGN, all
 * before any HIP call.  Asynchronous on `stream`.
 */
mxgemm_status mxgemm_norm_quantize(const mxgemm_norm *n, int T, int K, hipStream_t stream);

/* ---- attention over a paged cache ---------------------------------------------- */

/*
 * What stands between a layer's QKV product and its output product when a
 * model is served, in two operators that hand their device buffers on without
 * a host copy:
 *
 *   mxgemm_run              activations -> queries, keys and values (bf16)
 *   mxgemm_kv_append        queries and keys turned to their positions; keys
 *                           and values into the cache's pages
 *   mxgemm_paged_attention  attention of the new tokens over the pages -> bf16
 *                           rows and / or the output product's quantized A
 *   mxgemm_run              the output product
 *
 * Forward only, like the rest of the library.  Neither allocates, reads back
 * or keeps anything: both can be captured into a graph, and calls that share
 * no output, cache or workspace can overlap.
 */
#define MXGEMM_KV_BF16     0
#define MXGEMM_KV_FP8_E4M3 1

/*
 * A paged cache and the batch of sequences that uses it.
 *
 * Token i of sequence s is row i % page_size of page pages[s][i / page_size];
 * key head h of that row stands at
 *
 *     k + page * page_stride + h * head_stride + row * token_stride
 *
 * (strides in elements of the format), v likewise.  Elements are bf16, or E4M3
 * codes worth code * k_scale[h] (v_scale[h]); NULL scales are 1.
 *
 * The batch's new tokens are rows of its activations: those of sequence s are
 * rows offsets[s] .. offsets[s + 1] - 1 (none: the sequence is left out).
 * lens[s] counts the tokens of s with the new ones, so that a new token's
 * position is lens[s] - (offsets[s + 1] - row).
 *
 * offsets, lens and pages are device arrays of int32.  offsets have to ascend;
 * whatever the three hold, no address outside the buffers is formed: offsets
 * are clamped to [0, T], lens to [0, max_pages * page_size], nothing is written
 * to a page outside [0, num_pages) and it reads as zeros.  Rows of outputs that
 * no sequence has are left as they were.
 *
 * Limits: head_dim a multiple of 32 up to 256; page_size a power of two from 16
 * to 65536; seqs <= 65536; max_pages * page_size < 2^31; token_stride *
 * page_size < 2^30; query, key and value heads together at most 512 (else
 * MXGEMM_ERR_SHAPE).  k and v 16-byte aligned, strides whole 16 bytes, arrays
 * 4-byte aligned (else MXGEMM_ERR_ALIGN).
 */
typedef struct mxgemm_kv_cache {
    void *k, *v;
    int64_t page_stride, head_stride, token_stride; /* elements, of both k and v */
    const int32_t *pages;   /* [seqs][ld_pages] */
    int64_t ld_pages;       /* >= max_pages */
    const int32_t *offsets; /* [seqs + 1] */
    const int32_t *lens;    /* [seqs] */
    const float *k_scale;   /* [kv_heads] or NULL (NULL with bf16) */
    const float *v_scale;
    int32_t num_pages;      /* pages there are */
    int32_t page_size;      /* tokens of a page */
    int32_t seqs;
    int32_t max_pages;      /* pages of a sequence, at most */
    int32_t kv_heads;
    int32_t head_dim;
    int32_t format;         /* MXGEMM_KV_BF16 or MXGEMM_KV_FP8_E4M3 */
} mxgemm_kv_cache;

/*
 * Rotary positions and the append.  Of every head of Q and K the first rot_dim
 * elements are turned in pairs p = 0 .. rot_dim / 2 - 1 (elements p and p +
 * rot_dim / 2, or 2p and 2p + 1 with interleaved = 1) by the angle a =
 * position * freq[p]:
 *
 *     x' = factor * (x cos a - y sin a),   y' = factor * (y cos a + x sin a)
 *
 * and the others are copied.  Q goes to Q_out; K and V, which is not turned, go
 * to the new tokens' rows of the cache.  Angles are reduced in 64 bits, the rest
 * is in fp32 with one rounding to the output's type; an E4M3 code is the fp32
 * quotient by the head's scale, to nearest even, saturating at 448 (a NaN stays
 * one).  A token without a place in the cache (a negative position, a page
 * outside the cache) has its Q turned and nothing written.  Two new tokens must
 * not have the same place.
 */
typedef struct mxgemm_append {
    const void *Q;            /* bf16 [T][ldq], head h from column h * head_dim; NULL: no queries */
    void *Q_out;              /* bf16 [T][ldqo]; may be Q (ldqo == ldq); NULL with Q */
    const void *K, *V;        /* bf16 [T][ldk], [T][ldv]; both NULL: only Q is turned (k, v, pages unused) */
    int64_t ldq, ldqo, ldk, ldv;
    const int32_t *positions; /* [T] positions to turn by, or NULL: the tokens' places in the cache */
    const double *freq;       /* device, [rot_dim / 2], radians a position (mxgemm_rope_frequencies) */
    float factor;             /* of the turned elements; 1 unless a long context's scaling has one */
    int32_t heads;            /* query heads */
    int32_t rot_dim;          /* a multiple of 16 up to head_dim; 0: nothing is turned */
    int32_t interleaved;
} mxgemm_append;

/*
 * 1 <= T <= 2^24.  bf16 pointers 16-byte aligned, their strides multiples of 8
 * and at least heads * head_dim (kv_heads * head_dim).  Q, K and V may be
 * columns of one matrix.  Apart from Q_out no output overlaps an input.  Errors:
 * MXGEMM_ERR_INVALID_ARG (NULL or half a pair, a flag that is not 0 or 1,
 * another format, scales with bf16), MXGEMM_ERR_SHAPE, MXGEMM_ERR_ALIGN, all
 * before any HIP call.  Asynchronous on `stream`.
 */
mxgemm_status mxgemm_kv_append(const mxgemm_kv_cache *cache, const mxgemm_append *p, int T, hipStream_t stream);

/*
 * Frequencies for mxgemm_kv_append, computed on the host into host memory:
 * freq[p] = base^(-2 p / rot_dim), scaled for contexts `factor` times as long as
 * the `original` one the model was trained on: with low = high = 0 all divided
 * by factor (1: as they are); else a pair that turns at least `high` times over
 * the original context keeps its frequency, one that turns at most `low` times
 * has it divided by factor, and between them the kept share grows linearly with
 * the turns.  rot_dim even, 2 .. 256; base, factor > 0; 0 <= low < high and
 * original > 0 where they are used.  No HIP call is made.
 */
mxgemm_status mxgemm_rope_frequencies(double *freq, int rot_dim, double base, double factor, double original, double low,
                                      double high);

/*
 * Attention of the new tokens over the cache, which holds their own keys and
 * values already.  Query head h uses key head h / (heads / kv_heads).  A token
 * at position p sees the keys j < lens[s] with j <= p (causal = 1) and j > p -
 * window (window > 0), none if p < 0:
 *
 *     O[t][h] = sum_j e^(x_j) v_j / (sum_j e^(x_j) + e^sinks[h]),  x_j = scale * q . k_j
 *     lse[t][h] = log(sum_j e^(x_j) + e^sinks[h])
 *
 * (without sinks the last terms are absent; a row without a key is 0, its lse
 * -inf or the sink; a sink of +inf or NaN makes the rows of its head NaN).  Keys
 * that a row does not see do not reach it, whatever they or their values hold.
 * O is rounded once to bf16; A with scaleA are those bf16 values quantized
 * (mxgemm_quantize's rule, or MXFP8 as in "mixture of experts"), blocks of 32
 * columns of a row.  Products are of bf16 (E4M3 codes as they are), sums in
 * fp32; e^x is rounded to bf16 for the product with v.
 */
typedef struct mxgemm_attention {
    const void *Q;      /* bf16 [T][ldq], head h from column h * head_dim */
    void *O;            /* bf16 [T][ldo] or NULL; may be Q (ldo == ldq) */
    float *lse;         /* [T][heads], dense, or NULL */
    const float *sinks; /* [heads] or NULL */
    void *A;            /* [T][lda] codes or NULL (O or A) */
    void *scaleA;       /* [T][ldsa] scale bytes; NULL with A */
    int64_t ldq, ldo, lda, ldsa;
    float scale;        /* finite */
    int32_t heads;      /* a multiple of kv_heads */
    int32_t causal;
    int32_t window;     /* 0: none */
    int32_t max_new;    /* the most new tokens of a sequence, which chooses the kernel; 0: not known (any value gives the same results but for the order of sums) */
    int32_t a_format;   /* MXGEMM_FMT_FP4 or MXGEMM_FMT_FP8_E4M3 */
} mxgemm_attention;

/*
 * workspace: mxgemm_paged_attention_workspace_bytes(...) device bytes or more,
 * 16-byte aligned, ZEROED once before its first use and not shared by calls that
 * can overlap.  Its first 4 KiB are counters, which every call leaves zero
 * again; the rest needs no clearing, so that calls of any sizes can use one
 * workspace in turn.  Deterministic: the same call gives the same bits.
 * 1 <= T <= 2^24, T * heads <= 2^30, and U * (ceil(max_pages * page_size / 128) + 2)
 * < 2^31 - 512, where U = kv_heads * floor((T * heads / kv_heads + 31 * min(T,
 * seqs)) / 32) (else MXGEMM_ERR_SHAPE); bf16 pointers 16-byte aligned, their
 * strides multiples of 8; A as in mxgemm_quantize.  But for O no output overlaps an
 * input or another output.  Errors:
 * MXGEMM_ERR_INVALID_ARG, MXGEMM_ERR_SHAPE, MXGEMM_ERR_ALIGN,
 * MXGEMM_ERR_WORKSPACE, all before any HIP call.  Asynchronous on `stream`.
 */
mxgemm_status mxgemm_paged_attention(const mxgemm_kv_cache *cache, const mxgemm_attention *p, int T, void *workspace,
                                     size_t workspace_bytes, hipStream_t stream);

/* Bytes of mxgemm_paged_attention's workspace (0: an invalid shape). */
size_t mxgemm_paged_attention_workspace_bytes(int T, int seqs, int heads, int kv_heads, int head_dim);

/* ---- plan / query ------------------------------------------------------------- */

typedef struct mxgemm_info {
    int32_t kernel;          /* kernel family: 0 = tiled (LDS, M > 64); 1 = skinny (M <= 16,
                                streams B); 2 = skinny rows (16 < M <= 64, streams B, A
                                shared through LDS); 3 = tiled with an FP8/FP6 A; 4 =
                                GEMV (M == 1, or 2 <= M <= 8 with FP4 A; row-major B,
                                K % 2048 == 0, N >= 4 x num_cu, unsplit; 4 rows of B per
                                workgroup; with 16-byte aligned scale rows, else the skinny
                                kernel) */
    int32_t tile_m, tile_n;  /* output tile per workgroup */
    int32_t split_k;         /* K chunks the plan uses */
    int64_t grid;            /* workgroups launched */
    size_t workspace_bytes;  /* split-K fp32 partials workspace needed (0 if split_k == 1) */
    size_t packed_b_bytes;   /* size of mxgemm_pack_b's Bp for this N, K */
    size_t packed_sb_bytes;  /* size of mxgemm_pack_b's SBp for this N, K */
    size_t packed_sa_bytes;  /* size of mxgemm_pack_scales' output for the M rows of scaleA */
    int32_t num_cu;          /* compute units the plan assumed */
    int32_t persist_grid;    /* > 0: the tiled kernel runs persistent, this many workgroups
                                (one per CU) walking the `grid` tiles in the same order;
                                assumes beta == 0 and 16-byte aligned pointers, as the
                                persistent form needs (else mxgemm_run uses the plain grid) */
    char kernel_name[64];
    char arch[32];           /* device architecture (mxgemm_query only) */
    double peak_flops;       /* dense MXFP4 matrix peak, flop/s, from the device clock and CU count */
    double clock_hz;         /* peak engine clock used for peak_flops */
} mxgemm_info;

/*
 * Plan for the current device: the kernel, tile and split mxgemm_run would
 * use for these arguments, and the buffer sizes it needs.  The plan follows
 * the asm_f4gemm README's "Tile selection heuristic" (count the rounds of
 * workgroups the compute units need per tile shape, prefer fewer rounds of
 * larger tiles, iterate candidates in a fixed order), weighted by a per-tile
 * cost that also prices split-K.  Returns MXGEMM_ERR_UNSUPPORTED_DEVICE
 * unless the current device is gfx950.  split_k as for mxgemm_run.
 */
mxgemm_status mxgemm_query(int M, int N, int K, int b_packed, int split_k,
                           mxgemm_info *out);

/*
 * The same plan for a device with num_cu compute units, computed on the
 * host without touching any device (arch, peak_flops, clock_hz left 0).
 */
mxgemm_status mxgemm_plan(int M, int N, int K, int b_packed, int split_k, int num_cu,
                          mxgemm_info *out);

/* mxgemm_plan / mxgemm_query for the exact path mxgemm_run takes with these
 * strides and options (a_format, split_mode, b_packed; NULL = defaults):
 * with a wider A format or the bf16-atomic split the kernel and the
 * workspace differ from the FP4 plan, and a caller workspace must be sized
 * from this call.  kernel = 3 is the tiled kernel with 8-bit A.  Same
 * errors as mxgemm_plan / mxgemm_query, plus MXGEMM_ERR_INVALID_ARG for
 * option values mxgemm_run rejects. */
mxgemm_status mxgemm_plan_ex(int M, int N, int K, const mxgemm_strides *strides, int split_k, int num_cu,
                             mxgemm_info *out);
mxgemm_status mxgemm_query_ex(int M, int N, int K, const mxgemm_strides *strides, int split_k,
                              mxgemm_info *out);

/* ---- measurement ------------------------------------------------------------ */

/*
 * Read `bytes` of device memory at src once, with the 16-byte non-temporal
 * loads the skinny kernels stream B with, and nothing else (sink, a 4-byte
 * device word, is written only if the XOR of everything read equals a fixed
 * constant).  A kernel whose minimum DRAM traffic is `bytes` cannot finish
 * faster on this chip ("Optimizing GEMM in HIP", background: the GEMM's
 * arithmetic intensity against its minimum required traffic), so its time
 * is the achievable ceiling the benchmark reports next to the published HBM
 * bandwidth.  bytes: a multiple of 16, below 2^31 (else
 * MXGEMM_ERR_SHAPE); src 16-byte and sink 4-byte aligned (else
 * MXGEMM_ERR_ALIGN).  Asynchronous on `stream`; allocates nothing.
 */
mxgemm_status mxgemm_stream_read(const void *src, size_t bytes, void *sink, hipStream_t stream);

/* Free the library-owned split-K workspaces (after synchronizing their
 * streams).  Later calls allocate again. */
mxgemm_status mxgemm_release_workspaces(void);

#ifdef __cplusplus
}
#endif

#endif /* LIBMXGEMM_H */
