"""Python binding of libmxgemm (MXFP4 block-scaled GEMM for gfx950).

Argument marshalling only: every function below calls the C-ABI entry point
of the same name in libmxgemm.so (declared in include/libmxgemm.h) and every
step of the computation runs in the library's HIP kernels.  Tensors may be
passed as torch tensors (their data_ptr() is used) or as raw device
addresses (int).  The stream defaults to torch's current stream.

There is no fallback: if libmxgemm.so is missing or fails to load, every
call raises MxGemmError.
"""
from __future__ import annotations

import ctypes
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmxgemm.so")

# C-ABI entry points declared in include/libmxgemm.h
EXPORTS = ("mxgemm_status_string", "mxgemm_run", "mxgemm_run_noalloc", "mxgemm_run_bf16a", "mxgemm_pack_b", "mxgemm_pack_scales", "mxgemm_pack_a",
           "mxgemm_pack_a_bytes", "mxgemm_quantize",
           "mxgemm_f16_run", "mxgemm_route", "mxgemm_route_workspace_bytes", "mxgemm_grouped_run", "mxgemm_glu_quantize",
           "mxgemm_norm_quantize", "mxgemm_kv_append", "mxgemm_rope_frequencies", "mxgemm_paged_attention",
           "mxgemm_paged_attention_workspace_bytes", "mxgemm_query", "mxgemm_plan", "mxgemm_query_ex", "mxgemm_plan_ex",
           "mxgemm_stream_read", "mxgemm_release_workspaces")

STATUS = {0: "MXGEMM_OK", -1: "MXGEMM_ERR_INVALID_ARG", -2: "MXGEMM_ERR_SHAPE",
          -3: "MXGEMM_ERR_ALIGN", -4: "MXGEMM_ERR_UNSUPPORTED_DEVICE", -5: "MXGEMM_ERR_HIP",
          -6: "MXGEMM_ERR_WORKSPACE", -7: "MXGEMM_ERR_SCRATCH"}


class MxGemmError(RuntimeError):
    def __init__(self, status, where=""):
        self.status = status
        name = STATUS.get(status, str(status))
        super().__init__("%s failed: %s (%s)" % (where, name, _status_text(status)))


class Strides(ctypes.Structure):
    _fields_ = [("ldd", ctypes.c_int64), ("ldc", ctypes.c_int64), ("lda", ctypes.c_int64),
                ("ldb", ctypes.c_int64), ("ldsa", ctypes.c_int64), ("ldsb", ctypes.c_int64),
                ("b_packed", ctypes.c_int32), ("sa_packed", ctypes.c_int32),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
                ("c_f32", ctypes.c_int32), ("split_mode", ctypes.c_int32),
                ("a_format", ctypes.c_int32), ("b_layout", ctypes.c_int32), ("a_packed", ctypes.c_int32)]


SPLIT_FP32 = 0         # MXGEMM_SPLIT_FP32
SPLIT_BF16_ATOMIC = 1  # MXGEMM_SPLIT_BF16_ATOMIC
# MXGEMM_FMT_*: A's element format
FMT_FP4, FMT_FP8_E4M3, FMT_FP8_E5M2, FMT_FP6_E2M3, FMT_FP6_E3M2 = 0, 1, 2, 3, 4
FORMAT_BITS = (4, 8, 8, 6, 6)
B_NK, B_KN = 0, 1  # MXGEMM_B_NK, MXGEMM_B_KN
KV_BF16, KV_FP8_E4M3 = 0, 1  # MXGEMM_KV_*: a cache's element format
NOALLOC_SCRATCH_BYTES = 32 << 20  # MXGEMM_NOALLOC_SCRATCH_BYTES


class Info(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int32), ("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32),
                ("split_k", ctypes.c_int32), ("grid", ctypes.c_int64),
                ("workspace_bytes", ctypes.c_size_t), ("packed_b_bytes", ctypes.c_size_t),
                ("packed_sb_bytes", ctypes.c_size_t), ("packed_sa_bytes", ctypes.c_size_t),
                ("num_cu", ctypes.c_int32),
                ("persist_grid", ctypes.c_int32), ("kernel_name", ctypes.c_char * 64),
                ("arch", ctypes.c_char * 32), ("peak_flops", ctypes.c_double),
                ("clock_hz", ctypes.c_double)]

    def as_dict(self):
        d = {f: getattr(self, f) for f, _ in self._fields_}
        d["kernel_name"] = self.kernel_name.decode()
        d["arch"] = self.arch.decode()
        return d


# (the functions below pass these two packed, in a fifth of a Structure's time;
# lib()'s entry points take either: a byref, or the bytes)
class Grouped(ctypes.Structure):
    _fields_ = [("ldd", ctypes.c_int64), ("lda", ctypes.c_int64), ("ldsa", ctypes.c_int64), ("ldb", ctypes.c_int64),
                ("ldsb", ctypes.c_int64), ("strideb", ctypes.c_int64), ("strideb_scale", ctypes.c_int64),
                ("a_format", ctypes.c_int32)]


class Norm(ctypes.Structure):
    _fields_ = [("Y", ctypes.c_void_p), ("ldy", ctypes.c_int64), ("pos", ctypes.c_void_p), ("weights", ctypes.c_void_p),
                ("top_k", ctypes.c_int32), ("y_rows", ctypes.c_int32), ("w_post", ctypes.c_void_p),
                ("gate", ctypes.c_void_p), ("ldg", ctypes.c_int64), ("X", ctypes.c_void_p), ("ldx", ctypes.c_int64),
                ("res_scale", ctypes.c_float), ("eps", ctypes.c_float), ("H", ctypes.c_void_p), ("ldh", ctypes.c_int64),
                ("w_pre", ctypes.c_void_p), ("Z", ctypes.c_void_p), ("ldz", ctypes.c_int64), ("A", ctypes.c_void_p),
                ("scaleA", ctypes.c_void_p), ("lda", ctypes.c_int64), ("ldsa", ctypes.c_int64),
                ("a_format", ctypes.c_int32)]


class KvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64), ("pages", ctypes.c_void_p),
                ("ld_pages", ctypes.c_int64), ("offsets", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("format", ctypes.c_int32)]


class Append(ctypes.Structure):
    _fields_ = [("Q", ctypes.c_void_p), ("Q_out", ctypes.c_void_p), ("K", ctypes.c_void_p), ("V", ctypes.c_void_p),
                ("ldq", ctypes.c_int64), ("ldqo", ctypes.c_int64), ("ldk", ctypes.c_int64), ("ldv", ctypes.c_int64),
                ("positions", ctypes.c_void_p), ("freq", ctypes.c_void_p), ("factor", ctypes.c_float),
                ("heads", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


class Attention(ctypes.Structure):
    _fields_ = [("Q", ctypes.c_void_p), ("O", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("sinks", ctypes.c_void_p),
                ("A", ctypes.c_void_p), ("scaleA", ctypes.c_void_p), ("ldq", ctypes.c_int64), ("ldo", ctypes.c_int64),
                ("lda", ctypes.c_int64), ("ldsa", ctypes.c_int64), ("scale", ctypes.c_float), ("heads", ctypes.c_int32),
                ("causal", ctypes.c_int32), ("window", ctypes.c_int32), ("max_new", ctypes.c_int32),
                ("a_format", ctypes.c_int32)]


_pack_grouped = struct.Struct("@7qi4x").pack
_pack_norm = struct.Struct("@PqPPiiPPqPqffPqPPqPPqqi4x").pack
_pack_cache = struct.Struct("@PPqqqPqPPPPiiiiiii4x").pack
_pack_append = struct.Struct("@PPPPqqqqPPfiii").pack
_pack_attention = struct.Struct("@PPPPPPqqqqfiiiii").pack

_lib = None


def lib():
    """The loaded libmxgemm.so (raises MxGemmError if it is not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise MxGemmError(-5, "loading %s (not built; run __graft_entry__.build())" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        L.mxgemm_status_string.argtypes = [i32]
        L.mxgemm_status_string.restype = ctypes.c_char_p
        L.mxgemm_run.argtypes = [vp, vp, vp, vp, vp, vp, ctypes.c_float, ctypes.c_float, i32, i32, i32,
                                 ctypes.POINTER(Strides), i32, vp]
        L.mxgemm_run.restype = i32
        L.mxgemm_run_noalloc.argtypes = L.mxgemm_run.argtypes
        L.mxgemm_run_noalloc.restype = i32
        L.mxgemm_run_bf16a.argtypes = [vp, vp, vp, vp, vp, ctypes.c_float, ctypes.c_float, i32, i32, i32, i64,
                                       ctypes.POINTER(Strides), i32, vp]
        L.mxgemm_run_bf16a.restype = i32
        L.mxgemm_pack_b.argtypes = [vp, vp, vp, vp, i32, i32, i64, i64, vp]
        L.mxgemm_pack_b.restype = i32
        L.mxgemm_pack_scales.argtypes = [vp, vp, i32, i32, i64, vp]
        L.mxgemm_pack_scales.restype = i32
        L.mxgemm_pack_a.argtypes = [vp, vp, vp, vp, i32, i32, i64, i64, i32, vp]
        L.mxgemm_pack_a.restype = i32
        L.mxgemm_pack_a_bytes.argtypes = [i32, i32]
        L.mxgemm_pack_a_bytes.restype = ctypes.c_size_t
        L.mxgemm_quantize.argtypes = [vp, vp, vp, i32, i32, i64, i64, i64, vp]
        L.mxgemm_quantize.restype = i32
        L.mxgemm_f16_run.argtypes = [vp, vp, vp, i32, i32, i32, i64, i64, i64, vp]
        L.mxgemm_f16_run.restype = i32
        L.mxgemm_route.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i64, i32, vp, ctypes.c_size_t, vp]
        L.mxgemm_route.restype = i32
        L.mxgemm_route_workspace_bytes.argtypes = [i32, i32]
        L.mxgemm_route_workspace_bytes.restype = ctypes.c_size_t
        L.mxgemm_grouped_run.argtypes = [vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, i32, i32, i32, i32, i32,
                                         vp, vp]
        L.mxgemm_grouped_run.restype = i32
        L.mxgemm_glu_quantize.argtypes = [vp, vp, vp, vp, i32, i32, i64, i64, i64, i32, vp]
        L.mxgemm_glu_quantize.restype = i32
        L.mxgemm_norm_quantize.argtypes = [vp, i32, i32, vp]
        L.mxgemm_norm_quantize.restype = i32
        L.mxgemm_kv_append.argtypes = [vp, vp, i32, vp]
        L.mxgemm_kv_append.restype = i32
        L.mxgemm_rope_frequencies.argtypes = [vp, i32] + [ctypes.c_double] * 5
        L.mxgemm_rope_frequencies.restype = i32
        L.mxgemm_paged_attention.argtypes = [vp, vp, i32, vp, ctypes.c_size_t, vp]
        L.mxgemm_paged_attention.restype = i32
        L.mxgemm_paged_attention_workspace_bytes.argtypes = [i32] * 5
        L.mxgemm_paged_attention_workspace_bytes.restype = ctypes.c_size_t
        L.mxgemm_query.argtypes = [i32, i32, i32, i32, i32, ctypes.POINTER(Info)]
        L.mxgemm_query.restype = i32
        L.mxgemm_plan.argtypes = [i32, i32, i32, i32, i32, i32, ctypes.POINTER(Info)]
        L.mxgemm_plan.restype = i32
        L.mxgemm_query_ex.argtypes = [i32, i32, i32, ctypes.POINTER(Strides), i32, ctypes.POINTER(Info)]
        L.mxgemm_query_ex.restype = i32
        L.mxgemm_plan_ex.argtypes = [i32, i32, i32, ctypes.POINTER(Strides), i32, i32, ctypes.POINTER(Info)]
        L.mxgemm_plan_ex.restype = i32
        L.mxgemm_stream_read.argtypes = [vp, ctypes.c_size_t, vp, vp]
        L.mxgemm_stream_read.restype = i32
        L.mxgemm_release_workspaces.argtypes = []
        L.mxgemm_release_workspaces.restype = i32
        _lib = L
    return _lib


def _status_text(status):
    try:
        return lib().mxgemm_status_string(status).decode()
    except Exception:
        return "?"


def _ptr(x):
    return x if x is None or isinstance(x, int) else x.data_ptr()


def _stream(stream):
    if stream is None:
        # torch.cuda.current_stream().cuda_stream, where torch has it without
        # building the Stream object (0.3 against 2.8 us, as much as the launch)
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        return torch.cuda.current_stream().cuda_stream if raw is None else raw(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status, where):
    if status != 0:
        raise MxGemmError(status, where)


def make_strides(*, ldd, ldc, lda, ldb, ldsa, ldsb, b_packed=0, sa_packed=0, workspace=None,
                 workspace_bytes=0, c_f32=0, split_mode=SPLIT_FP32, a_format=FMT_FP4, b_layout=B_NK, a_packed=0):
    return Strides(ldd, ldc, lda, ldb, ldsa, ldsb, b_packed, sa_packed, _ptr(workspace), workspace_bytes,
                   c_f32, split_mode, a_format, b_layout, a_packed)


def mxgemm_status_string(status: int) -> str:
    return lib().mxgemm_status_string(status).decode()


def mxgemm_run(D, C, A, B, scaleA, scaleB, alpha, beta, M, N, K, strides=None, split_k=-1,
               stream=None, check=True):
    """D = bf16(alpha * A * B^T + beta * C) on `stream` (asynchronous)."""
    sp = ctypes.byref(strides) if strides is not None else None
    st = lib().mxgemm_run(_ptr(D), _ptr(C), _ptr(A), _ptr(B), _ptr(scaleA), _ptr(scaleB),
                          float(alpha), float(beta), int(M), int(N), int(K), sp, int(split_k),
                          _stream(stream))
    if check:
        _check(st, "mxgemm_run")
    return st


def mxgemm_run_noalloc(D, C, A, B, scaleA, scaleB, alpha, beta, M, N, K, strides=None, split_k=-1,
                       stream=None, check=True):
    """mxgemm_run with the library's buffers in its fixed device scratch (no allocation)."""
    sp = ctypes.byref(strides) if strides is not None else None
    st = lib().mxgemm_run_noalloc(_ptr(D), _ptr(C), _ptr(A), _ptr(B), _ptr(scaleA), _ptr(scaleB),
                                  float(alpha), float(beta), int(M), int(N), int(K), sp, int(split_k),
                                  _stream(stream))
    if check:
        _check(st, "mxgemm_run_noalloc")
    return st


def mxgemm_pack_b(Bp, SBp, B, scaleB, N, K, ldb=None, ldsb=None, stream=None, check=True):
    """Pre-shuffle B and its scales into the kernels' layout (asynchronous)."""
    ldb = K if ldb is None else ldb
    ldsb = K // 32 if ldsb is None else ldsb
    st = lib().mxgemm_pack_b(_ptr(Bp), _ptr(SBp), _ptr(B), _ptr(scaleB), int(N), int(K),
                             int(ldb), int(ldsb), _stream(stream))
    if check:
        _check(st, "mxgemm_pack_b")
    return st


def mxgemm_pack_scales(Sp, S, rows, K, lds=None, stream=None, check=True):
    """Shuffle a [rows][K/32] scale matrix into the packed scale layout
    (scaleA for sa_packed = 1; asynchronous)."""
    lds = K // 32 if lds is None else lds
    st = lib().mxgemm_pack_scales(_ptr(Sp), _ptr(S), int(rows), int(K), int(lds), _stream(stream))
    if check:
        _check(st, "mxgemm_pack_scales")
    return st


def mxgemm_pack_a(Ap, SAp, A, scaleA, M, K, a_format, lda=None, ldsa=None, stream=None, check=True):
    """Put an FP6 A and its scales into the dense FP6 tile's order, for
    mxgemm_run with a_packed = 1 (asynchronous)."""
    lda = K if lda is None else lda
    ldsa = K // 32 if ldsa is None else ldsa
    st = lib().mxgemm_pack_a(_ptr(Ap), _ptr(SAp), _ptr(A), _ptr(scaleA), int(M), int(K), int(lda), int(ldsa),
                             int(a_format), _stream(stream))
    if check:
        _check(st, "mxgemm_pack_a")
    return st


def mxgemm_pack_a_bytes(M, K) -> int:
    return int(lib().mxgemm_pack_a_bytes(int(M), int(K)))


def mxgemm_run_bf16a(D, C, X, B, scaleB, alpha, beta, M, N, K, ldx=None, strides=None, split_k=-1,
                     stream=None, check=True):
    """D = bf16(alpha * quantize(X) * B^T + beta * C) on `stream` (asynchronous);
    X is a bf16 [M, ldx] activation (one fused launch at M = 1)."""
    sp = ctypes.byref(strides) if strides is not None else None
    st = lib().mxgemm_run_bf16a(_ptr(D), _ptr(C), _ptr(X), _ptr(B), _ptr(scaleB), float(alpha), float(beta),
                                int(M), int(N), int(K), int(K if ldx is None else ldx), sp, int(split_k),
                                _stream(stream))
    if check:
        _check(st, "mxgemm_run_bf16a")
    return st


def mxgemm_quantize(A, SA, X, M, K, ldx=None, lda=None, ldsa=None, stream=None, check=True):
    """bf16 X [M][ldx] -> packed E2M1 A [M][lda/2] bytes and E8M0 scales
    SA [M][ldsa] (asynchronous; strides default to dense rows)."""
    ldx = K if ldx is None else ldx
    lda = K if lda is None else lda
    ldsa = K // 32 if ldsa is None else ldsa
    st = lib().mxgemm_quantize(_ptr(A), _ptr(SA), _ptr(X), int(M), int(K), int(ldx), int(lda),
                               int(ldsa), _stream(stream))
    if check:
        _check(st, "mxgemm_quantize")
    return st


def mxgemm_f16_run(C, A, B, M, N, K, lda=None, ldb=None, ldc=None, stream=None, check=True):
    """fp32 C [M][ldc] = fp16 A [M][lda] x fp16 B [K][ldb] (asynchronous;
    strides in elements, default dense)."""
    lda = K if lda is None else lda
    ldb = N if ldb is None else ldb
    ldc = N if ldc is None else ldc
    st = lib().mxgemm_f16_run(_ptr(C), _ptr(A), _ptr(B), int(M), int(N), int(K), int(lda), int(ldb), int(ldc),
                              _stream(stream))
    if check:
        _check(st, "mxgemm_f16_run")
    return st


def mxgemm_route(ids, weights, pos, offsets, rows, logits, T, E, top_k, ldl=None, bf16=False, renorm=True,
                 workspace=None, workspace_bytes=0, stream=None, check=True):
    """Router logits -> each token's top_k experts and weights, and the rows
    ordered by expert (asynchronous; workspace: mxgemm_route_workspace_bytes)."""
    st = lib().mxgemm_route(_ptr(ids), _ptr(weights), _ptr(pos), _ptr(offsets), _ptr(rows), _ptr(logits), int(bf16),
                            int(T), int(E), int(top_k), int(E if ldl is None else ldl), int(renorm), _ptr(workspace),
                            int(workspace_bytes), _stream(stream))
    if check:
        _check(st, "mxgemm_route")
    return st


def mxgemm_route_workspace_bytes(T, E) -> int:
    return int(lib().mxgemm_route_workspace_bytes(int(T), int(E)))


def mxgemm_grouped_run(D, A, B, scaleA, scaleB, offsets, rows, N, K, groups, a_rows=None, a_count=None, alpha=1.0,
                       a_format=FMT_FP4, ldd=None, lda=None, ldsa=None, ldb=None, ldsb=None, strideb=None,
                       strideb_scale=None, stream=None, check=True):
    """D[i] = bf16(alpha * A[a_rows[i]] * B[e]^T) for the rows i of each
    expert e (offsets; asynchronous; strides default to dense)."""
    KB = K // 32
    ldb = K if ldb is None else ldb
    ldsb = KB if ldsb is None else ldsb
    g = _pack_grouped(N if ldd is None else ldd, K if lda is None else lda, KB if ldsa is None else ldsa, ldb, ldsb,
                      N * ldb if strideb is None else strideb, N * ldsb if strideb_scale is None else strideb_scale, a_format)
    st = lib().mxgemm_grouped_run(_ptr(D), _ptr(A), _ptr(B), _ptr(scaleA), _ptr(scaleB), _ptr(offsets), _ptr(a_rows),
                                  float(alpha), int(rows), int(rows if a_count is None else a_count), int(N), int(K),
                                  int(groups), g, _stream(stream))
    if check:
        _check(st, "mxgemm_grouped_run")
    return st


def mxgemm_glu_quantize(A, scaleA, X, M, K, live=None, ldx=None, lda=None, ldsa=None, a_format=FMT_FP4, stream=None,
                        check=True):
    """bf16 X [M][gate K | up K] -> quantized silu(gate) * up (asynchronous;
    rows from *live on are left; strides default to dense rows)."""
    st = lib().mxgemm_glu_quantize(_ptr(A), _ptr(scaleA), _ptr(X), _ptr(live), int(M), int(K),
                                   int(2 * K if ldx is None else ldx), int(K if lda is None else lda),
                                   int(K // 32 if ldsa is None else ldsa), int(a_format), _stream(stream))
    if check:
        _check(st, "mxgemm_glu_quantize")
    return st


def mxgemm_norm_quantize(T, K, Y, X=None, H=None, Z=None, A=None, scaleA=None, pos=None, weights=None, top_k=0, y_rows=0,
                         w_post=None, gate=None, res_scale=1.0, w_pre=None, eps=1e-6, a_format=FMT_FP4, ldy=None,
                         ldg=None, ldx=None, ldh=None, ldz=None, lda=None, ldsa=None, stream=None, check=True):
    """Weighted sum of a token's rows of Y, norm, gate, residual -> H; its
    norm -> Z and, quantized, A and scaleA (asynchronous; strides default to
    dense rows; a gate of one row for all tokens: ldg=0)."""
    n = _pack_norm(_ptr(Y) or 0, K if ldy is None else ldy, _ptr(pos) or 0, _ptr(weights) or 0, top_k, y_rows,
                   _ptr(w_post) or 0, _ptr(gate) or 0, K if ldg is None else ldg, _ptr(X) or 0, K if ldx is None else ldx,
                   res_scale, eps, _ptr(H) or 0, K if ldh is None else ldh, _ptr(w_pre) or 0, _ptr(Z) or 0,
                   K if ldz is None else ldz, _ptr(A) or 0, _ptr(scaleA) or 0, K if lda is None else lda,
                   K // 32 if ldsa is None else ldsa, a_format)
    st = lib().mxgemm_norm_quantize(n, int(T), int(K), _stream(stream))
    if check:
        _check(st, "mxgemm_norm_quantize")
    return st


def make_kv_cache(k, v, pages, offsets, lens, *, seqs, num_pages, page_size, max_pages, kv_heads, head_dim, fp8=False,
                  k_scale=None, v_scale=None, ld_pages=None, page_stride=None, head_stride=None, token_stride=None):
    """A paged cache and its batch for the calls below, as bytes that hold the
    tensors' addresses (keep the tensors); strides in elements, by default pages
    of [kv_heads][page_size][head_dim]."""
    token = head_dim if token_stride is None else token_stride
    head = page_size * token if head_stride is None else head_stride
    return _pack_cache(_ptr(k) or 0, _ptr(v) or 0, kv_heads * head if page_stride is None else page_stride, head, token,
                       _ptr(pages) or 0, max_pages if ld_pages is None else ld_pages, _ptr(offsets) or 0, _ptr(lens) or 0,
                       _ptr(k_scale) or 0, _ptr(v_scale) or 0, num_pages, page_size, seqs, max_pages, kv_heads, head_dim,
                       KV_FP8_E4M3 if fp8 else KV_BF16)


def mxgemm_kv_append(cache, T, Q=None, K=None, V=None, Q_out=None, heads=0, ldq=0, ldk=0, ldv=0, ldqo=0, positions=None,
                     freq=None, rot_dim=0, interleaved=False, factor=1.0, stream=None, check=True):
    """Turn the new tokens' queries and keys to their positions, Q to Q_out, K
    and V to the cache's pages (asynchronous; cache: make_kv_cache)."""
    p = _pack_append(_ptr(Q) or 0, _ptr(Q_out) or 0, _ptr(K) or 0, _ptr(V) or 0, ldq, ldqo, ldk, ldv, _ptr(positions) or 0,
                     _ptr(freq) or 0, factor, heads, rot_dim, interleaved)
    st = lib().mxgemm_kv_append(cache, p, int(T), _stream(stream))
    if check:
        _check(st, "mxgemm_kv_append")
    return st


def mxgemm_rope_frequencies(rot_dim, base=10000.0, factor=1.0, original=0.0, low=0.0, high=0.0) -> list:
    """The rot_dim / 2 frequencies of mxgemm_kv_append, float64 values on the host."""
    freq = (ctypes.c_double * max(rot_dim // 2, 1))()
    _check(lib().mxgemm_rope_frequencies(freq, int(rot_dim), float(base), float(factor), float(original), float(low),
                                         float(high)), "mxgemm_rope_frequencies")
    return list(freq)


def mxgemm_paged_attention(cache, T, Q, O=None, *, heads, scale, workspace, workspace_bytes, lse=None, sinks=None, A=None,
                           scaleA=None, ldq=0, ldo=0, lda=0, ldsa=0, causal=True, window=0, max_new=0, a_format=FMT_FP4,
                           stream=None, check=True):
    """Attention of the new tokens' Q over the cache (asynchronous; bf16 O and /
    or the quantized A and scaleA; workspace: zeroed once,
    mxgemm_paged_attention_workspace_bytes)."""
    p = _pack_attention(_ptr(Q) or 0, _ptr(O) or 0, _ptr(lse) or 0, _ptr(sinks) or 0, _ptr(A) or 0, _ptr(scaleA) or 0, ldq,
                        ldo, lda, ldsa, scale, heads, causal, window, max_new, a_format)
    st = lib().mxgemm_paged_attention(cache, p, int(T), _ptr(workspace), int(workspace_bytes), _stream(stream))
    if check:
        _check(st, "mxgemm_paged_attention")
    return st


def mxgemm_paged_attention_workspace_bytes(T, seqs, heads, kv_heads, head_dim) -> int:
    return int(lib().mxgemm_paged_attention_workspace_bytes(int(T), int(seqs), int(heads), int(kv_heads), int(head_dim)))


def mxgemm_query(M, N, K, b_packed=0, split_k=-1) -> dict:
    info = Info()
    _check(lib().mxgemm_query(int(M), int(N), int(K), int(b_packed), int(split_k),
                              ctypes.byref(info)), "mxgemm_query")
    return info.as_dict()


def mxgemm_query_ex(M, N, K, strides=None, split_k=-1) -> dict:
    """mxgemm_query for the path mxgemm_run takes with these strides/options."""
    info = Info()
    sp = ctypes.byref(strides) if strides is not None else None
    _check(lib().mxgemm_query_ex(int(M), int(N), int(K), sp, int(split_k), ctypes.byref(info)), "mxgemm_query_ex")
    return info.as_dict()


def mxgemm_plan_ex(M, N, K, strides=None, split_k=-1, num_cu=256) -> dict:
    """mxgemm_plan for the path mxgemm_run takes with these strides/options."""
    info = Info()
    sp = ctypes.byref(strides) if strides is not None else None
    _check(lib().mxgemm_plan_ex(int(M), int(N), int(K), sp, int(split_k), int(num_cu), ctypes.byref(info)),
           "mxgemm_plan_ex")
    return info.as_dict()


def mxgemm_plan(M, N, K, b_packed=0, split_k=-1, num_cu=256) -> dict:
    info = Info()
    _check(lib().mxgemm_plan(int(M), int(N), int(K), int(b_packed), int(split_k), int(num_cu),
                             ctypes.byref(info)), "mxgemm_plan")
    return info.as_dict()


def mxgemm_stream_read(src, nbytes, sink, stream=None, check=True):
    """Streaming read of nbytes at src (the achievable-bandwidth reference)."""
    st = lib().mxgemm_stream_read(_ptr(src), int(nbytes), _ptr(sink), _stream(stream))
    if check:
        _check(st, "mxgemm_stream_read")
    return st


def mxgemm_release_workspaces():
    _check(lib().mxgemm_release_workspaces(), "mxgemm_release_workspaces")
