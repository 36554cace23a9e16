"""Host-side checks of the mixture-of-experts entry points (no GPU): every
refusal comes before any HIP call, struct layouts match the header, and the
64-bit implementations the GPU tests compare with are checked themselves."""
import ctypes
import decimal
import math
import os
import shutil
import subprocess
import tempfile
from fractions import Fraction

import numpy as np
import pytest

import block_scaled_precision_mxfp4_amd as mx
import experts_ref as ref
import oracle
from block_scaled_precision_mxfp4_amd import build as mxbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    if mxbuild.is_stale():
        mxbuild.build()


def test_struct_layouts_match_the_header():
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    lines, want = [], []
    for cname, cls in {"mxgemm_grouped": mx.Grouped, "mxgemm_norm": mx.Norm}.items():
        lines.append('printf("%%zu\\n", sizeof(%s));' % cname)
        want.append(ctypes.sizeof(cls))
        for f, _ in cls._fields_:
            lines.append('printf("%%zu\\n", offsetof(%s, %s));' % (cname, f))
            want.append(getattr(cls, f).offset)
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "libmxgemm.h"\nint main(void){%s return 0;}\n' % " ".join(lines)
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "l.c"), os.path.join(d, "l")
        open(c, "w").write(src)
        subprocess.run([cc, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"), c,
                        "-o", exe], check=True)
        got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == want


def test_packed_structs_are_the_structs():
    rng = np.random.default_rng(1)
    for pack, cls in ((mx._pack_grouped, mx.Grouped), (mx._pack_norm, mx.Norm)):
        v = [float(np.float32(rng.random())) if t is ctypes.c_float else int(rng.integers(1, 1 << 30)) for _, t in cls._fields_]
        assert pack(*v) == bytes(cls(*v))


def test_structs_pass_to_the_library():
    """A caller's own structs, by reference, by pointer, packed, or none."""
    L = mx.lib()
    g = mx.Grouped(256, 512, 16, 512, 16, 256 * 512, 256 * 16, 0)
    n = mx.Norm(Y=0x1000, ldy=64, H=0x3000, ldh=64, eps=1e-6)

    def grouped(p):
        return L.mxgemm_grouped_run(0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000, None, 1.0, 64, 64, 256, 512, 8, p, 0)
    for way in (ctypes.byref, ctypes.pointer, bytes):
        g.ldd, g.a_format, n.ldy, n.eps = 255, 0, 64, 0.0
        assert grouped(way(g)) == -2 and L.mxgemm_norm_quantize(way(n), 4, 64, 0) == -1
        g.ldd, g.a_format, n.ldy, n.eps = 256, 2, 32, 1e-6
        assert grouped(way(g)) == -1 and L.mxgemm_norm_quantize(way(n), 4, 64, 0) == -2
    assert L.mxgemm_norm_quantize(None, 4, 64, 0) == -1
    assert L.mxgemm_grouped_run(0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000, None, 1.0, 64, 64, 256, 48, 8, None, 0) == -2


def test_current_stream_without_torchs_raw_getter(monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: type("S", (), {"cuda_stream": 0x1230}))
    assert mx._stream(None) == 0x1230 and mx._stream(7) == 7


def _route(**kw):
    a = dict(ids=0x1000, weights=0x2000, pos=0x3000, offsets=0x4000, rows=0x5000, logits=0x6000, T=64, E=32, top_k=4,
             workspace=None, workspace_bytes=0, stream=0)
    a.update(kw)
    return mx.mxgemm_route(**a, check=False)


@pytest.mark.parametrize("kw,code", [
    (dict(ids=None), -1), (dict(weights=None), -1), (dict(pos=None), -1), (dict(offsets=None), -1), (dict(rows=None), -1),
    (dict(logits=None), -1), (dict(bf16=2), -1), (dict(renorm=-1), -1),
    (dict(T=0), -2), (dict(E=0), -2), (dict(E=1025, ldl=1025), -2), (dict(top_k=0), -2), (dict(top_k=17), -2),
    (dict(E=3), -2), (dict(ldl=31), -2), (dict(T=1 << 29, top_k=4), -2),
    (dict(ids=0x1002), -3), (dict(weights=0x2001), -3), (dict(pos=0x3002), -3), (dict(offsets=0x4002), -3),
    (dict(rows=0x5002), -3), (dict(logits=0x6002), -3), (dict(logits=0x6001, bf16=True), -3),
    (dict(T=65), -6), (dict(T=65, workspace=0x7000, workspace_bytes=255), -6),
    (dict(T=65, workspace=0x7002, workspace_bytes=256), -3),
])
def test_route_refusals(kw, code):
    assert _route(**kw) == code


def test_route_workspace_sizes():
    assert mx.mxgemm_route_workspace_bytes(64, 1024) == 0
    assert mx.mxgemm_route_workspace_bytes(0, 8) == 0 and mx.mxgemm_route_workspace_bytes(100, 1025) == 0
    for T in (65, 128, 1000, 16384, 16385, 100000, 1 << 30):
        for E in (1, 100, 1024):
            n = mx.mxgemm_route_workspace_bytes(T, E)
            assert 0 < n <= min(4 * E * -(-T // 64), 4 * E * 256)


def _grouped(**kw):
    a = dict(D=0x1000, A=0x2000, B=0x3000, scaleA=0x4000, scaleB=0x5000, offsets=0x6000, rows=64, N=256, K=512, groups=8,
             stream=0)
    a.update(kw)
    return mx.mxgemm_grouped_run(**a, check=False)


@pytest.mark.parametrize("kw,code", [
    (dict(D=None), -1), (dict(A=None), -1), (dict(B=None), -1), (dict(scaleA=None), -1), (dict(scaleB=None), -1),
    (dict(offsets=None), -1), (dict(a_format=2), -1), (dict(a_format=3), -1), (dict(a_format=-1), -1),
    (dict(rows=0), -2), (dict(rows=(1 << 30) + 1, a_rows=0x7000, a_count=1), -2), (dict(a_count=63), -2), (dict(a_rows=0x7000, a_count=0), -2), (dict(N=0), -2), (dict(K=48), -2),
    (dict(K=16), -2), (dict(K=(1 << 24) + 32), -2), (dict(groups=0), -2), (dict(groups=65536), -2), (dict(ldd=255), -2),
    (dict(lda=480), -2), (dict(ldsa=15), -2), (dict(ldb=480), -2), (dict(ldsb=15), -2), (dict(strideb=-32), -2),
    (dict(strideb_scale=-1), -2), (dict(ldb=1 << 24), -2), (dict(ldsb=1 << 23), -2), (dict(lda=1 << 24), -2),
    (dict(a_rows=0x7000, a_count=1 << 23), -2), (dict(a_rows=0x7000, a_count=1 << 10, ldsa=1 << 21), -2),
    (dict(A=0x2008), -3), (dict(B=0x3008), -3), (dict(D=0x1001), -3), (dict(offsets=0x6002), -3), (dict(a_rows=0x7002), -3),
    (dict(lda=513), -3), (dict(lda=528), -3), (dict(ldb=528), -3), (dict(strideb=256 * 512 + 16), -3),
    (dict(a_format=1, lda=520), -3),
])
def test_grouped_refusals(kw, code):
    assert _grouped(**kw) == code


@pytest.mark.parametrize("lda", [1 << 61, (1 << 62) - 32, 1 << 62, (1 << 62) + 32, (1 << 63) - 128])
@pytest.mark.parametrize("a_format", [0, 1])
@pytest.mark.parametrize("a_rows", [None, 0x7000])
def test_grouped_strides_past_64_bits_are_refused(lda, a_format, a_rows):
    """Strides whose bits are more than 64 bits count: their rows are past every span, not at a pitch of the low bits."""
    assert _grouped(lda=lda, a_format=a_format, a_rows=a_rows) == -2
    assert _grouped(ldb=lda, strideb=0, a_format=a_format, a_rows=a_rows) == -2


def _glu(**kw):
    a = dict(A=0x1000, scaleA=0x2000, X=0x3000, M=4, K=64, stream=0)
    a.update(kw)
    return mx.mxgemm_glu_quantize(**a, check=False)


@pytest.mark.parametrize("kw,code", [
    (dict(A=None), -1), (dict(scaleA=None), -1), (dict(X=None), -1), (dict(a_format=2), -1), (dict(a_format=4), -1),
    (dict(M=0), -2), (dict(K=0), -2), (dict(K=48), -2), (dict(K=(1 << 24) + 32), -2), (dict(ldx=120), -2), (dict(lda=32), -2),
    (dict(ldsa=1), -2), (dict(M=1 << 30, K=1 << 20), -2), (dict(M=1 << 30, K=32), -2), (dict(M=1 << 24, K=2048), -2),
    (dict(X=0x3008), -3), (dict(ldx=132), -3), (dict(A=0x1008), -3), (dict(lda=80), -3), (dict(a_format=1, lda=72), -3),
    (dict(live=0x4002), -3),
])
def test_glu_refusals(kw, code):
    assert _glu(**kw) == code


def _norm(**kw):
    a = dict(T=4, K=64, Y=0x1000, X=0x2000, H=0x3000, Z=0x4000, A=0x5000, scaleA=0x6000, w_post=0x7000, w_pre=0x8000,
             stream=0)
    a.update(kw)
    return mx.mxgemm_norm_quantize(**a, check=False)


@pytest.mark.parametrize("kw,code", [
    (dict(Y=None), -1), (dict(H=None, Z=None, A=None, scaleA=None), -1), (dict(A=None), -1), (dict(scaleA=None), -1),
    (dict(top_k=-1), -1), (dict(top_k=2), -1), (dict(top_k=2, pos=0x9000), -1), (dict(pos=0x9000, weights=0xA000), -1),
    (dict(eps=0.0), -1), (dict(eps=float("nan")), -1), (dict(a_format=2), -1),
    (dict(T=0), -2), (dict(K=0), -2), (dict(K=48), -2), (dict(K=16416), -2),
    (dict(T=1 << 26), -2), (dict(T=1 << 24, K=544), -2), (dict(T=1 << 23, K=4128), -2), (dict(T=1 << 22, K=8224), -2),
    (dict(ldy=32), -2), (dict(ldx=32), -2),
    (dict(gate=0x9000, ldg=32), -2), (dict(ldh=32), -2), (dict(ldz=32), -2), (dict(lda=32), -2), (dict(ldsa=1), -2),
    (dict(top_k=2, pos=0x9000, weights=0xA000, y_rows=0), -2), (dict(top_k=1025, pos=0x9000, weights=0xA000, y_rows=9), -2),
    (dict(Y=0x1008), -3), (dict(X=0x2008), -3), (dict(gate=0x9008), -3), (dict(H=0x3002), -3), (dict(Z=0x4008), -3),
    (dict(A=0x5008), -3), (dict(w_post=0x7008), -3), (dict(w_pre=0x8008), -3), (dict(ldy=68), -3), (dict(ldx=68), -3),
    (dict(gate=0x9000, ldg=68), -3), (dict(ldh=68), -3), (dict(ldz=68), -3), (dict(lda=80), -3),
    (dict(top_k=2, pos=0x9002, weights=0xA000, y_rows=9), -3), (dict(top_k=2, pos=0x9000, weights=0xA001, y_rows=9), -3),
])
def test_norm_refusals(kw, code):
    assert _norm(**kw) == code


# ---- the 64-bit implementations themselves ------------------------------------

def test_bf16_rounding_matches_torch():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(1)
    f = np.concatenate([rng.integers(0, 1 << 32, 200000, dtype=np.uint32).view(np.float32),
                        np.array([1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 3.3961775e38, 3.39e38, 2.0 ** -133, 1.5 * 2.0 ** -133], np.float32)])
    f = f[~np.isnan(f)]
    want = torch.from_numpy(f).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    assert np.array_equal(ref.f64_to_bf16(f.astype(np.float64)), want)


def test_fp8_quantizer_matches_torch_casts():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(2)
    bits = ref.f64_to_bf16(rng.standard_normal((64, 256)) * np.exp2(rng.uniform(-140, 120, (64, 1))))
    code, scale = ref.quantize_fp8(bits)
    v = ref.bf16_to_f64(bits).reshape(64, -1, 32)
    x = scale.astype(int) - 127
    most = np.abs(v).max(-1)
    assert ((most == 0) | (x == -127) | ((np.ldexp(most, -x) >= 256) & (np.ldexp(most, -x) < 512))).all()
    s = torch.from_numpy(np.clip(np.ldexp(v, -x[..., None]), -448, 448).reshape(64, 256).astype(np.float32))
    assert np.array_equal(code, s.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_fp8_codes_decode_to_their_values():
    bits = ref.f64_to_bf16(np.linspace(-300, 300, 64).reshape(1, 64))
    code, scale = ref.quantize_fp8(bits)
    got = np.array([oracle.decode(1, int(c)) for c in code[0]]) * np.exp2(scale[0].astype(float) - 127).repeat(32)
    assert np.abs(got - ref.bf16_to_f64(bits)[0]).max() <= 2.0 ** -4 * 300


def special_logits(rng, T, E):
    """Ties, zeros of both signs, masks, NaN, infinities and the type's lowest value; tokens of which nothing is left."""
    x = rng.integers(-2, 3, (T, E)).astype(np.float32) / 2
    x = np.where(rng.random((T, E)) < 0.5, x, 4 * rng.standard_normal((T, E)).astype(np.float32))
    x[rng.random((T, E)) < 0.1] = -0.0
    x[rng.random((T, E)) < 0.4] = -np.inf
    x[rng.random((T, E)) < 0.05] = np.nan
    x[rng.random((T, E)) < 0.3 / E] = np.inf
    x[rng.random((T, E)) < 0.02] = np.finfo(np.float32).min
    x[rng.random(T) < 0.1] = -np.inf
    x[0], x[1] = np.nan, np.finfo(np.float32).min
    x[2], x[2, E // 2] = -np.inf, 1.0
    x[3], x[3, 0], x[3, E - 1] = -100.0, 0.0, -90.0  # shares near fp32's least value
    return x


@pytest.mark.parametrize("T,E,k", [(50, 12, 4), (400, 40, 5), (90, 300, 12), (70, 1024, 16)])
def test_route_weight_bound_is_tight_beside_masks(T, E, k):
    x = special_logits(np.random.default_rng(T), T, E).astype(np.float64)
    for renorm in (True, False):
        with np.errstate(invalid="ignore"):
            ids, w, _, _, _ = ref.route(x, k, renorm)
        rel, small = ref.route_weight_bound(x, ids)
        assert rel.max() < 1e-3
        some = w > 2 * small
        assert some.any() and (np.abs(1.001 * w - w) > rel * w + small)[some].all()  # a mistake of a thousandth is seen


def test_glu_is_the_exact_rounding_but_for_ties_at_its_ends():
    """ref.glu (64 bits, rounded once) against 60 digits: the same bf16 value, unless gate * up or half of it is exactly in
    the middle between two bf16 values at a gate above 36 or below 2^-50 in magnitude; there the tie may go to even."""
    def rounded(v):  # to bf16, exactly; and whether v is a tie
        step = Fraction(2) ** max(math.frexp(float(v))[1] - 8, -133)
        return round(v / step) * step, (2 * v / step) % 2 == 1
    rng = np.random.default_rng(5)
    g = np.concatenate([rng.uniform(30, 45, 1500), 2.0 ** rng.uniform(5.2, 7, 300), rng.uniform(-60, 30, 700),
                        rng.choice([-1, 1], 1500) * 2.0 ** rng.uniform(-60, -40, 1500)])
    bits = np.stack([ref.f64_to_bf16(g), ref.f64_to_bf16(rng.standard_normal(len(g)))])
    got = ref.bf16_to_f64(ref.glu(bits.T.copy(), 1)[:, 0])
    g, u = ref.bf16_to_f64(bits)
    ties = off = 0
    with decimal.localcontext() as c:
        c.prec = 60
        for i in range(len(g)):
            v = decimal.Decimal(g[i]) / (1 + (-decimal.Decimal(g[i])).exp()) * decimal.Decimal(u[i])
            exact, _ = rounded(Fraction(v))
            even, tie = rounded(Fraction(g[i]) * Fraction(u[i]) / (1 if g[i] > 1 else 2))
            if tie and (g[i] > 36 or abs(g[i]) < 2.0 ** -50):
                ties += 1
                off += Fraction(got[i]) != exact
                assert Fraction(got[i]) in (even, exact), (g[i], u[i], got[i])
            else:
                assert Fraction(got[i]) == exact, (g[i], u[i], got[i])
    assert ties > 20 and off > 5  # the exception is there


def test_fingerprint_covers_what_the_kernels_are_built_from():
    import re
    from block_scaled_precision_mxfp4_amd import kernel_hash as kh
    csrc = os.path.join(ROOT, "block_scaled_precision_mxfp4_amd", "csrc")
    need, todo = set(), ["mx_route.hip", "mx_grouped.hip", "mx_tile_grouped.hip", "mx_glu.hip", "mx_norm.hip"]
    while todo:
        f = todo.pop()
        if f not in need:
            need.add(f)
            todo += re.findall(r'#include "(mx_[a-z0-9_]+\.hpp)"', open(os.path.join(csrc, f)).read())
    assert need <= set(kh.FAMILY_FILES["experts"]) and len(kh.kernel_family_hash("experts")) == 16
