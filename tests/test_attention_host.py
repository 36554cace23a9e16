"""Host-side checks of the paged-cache entry points (no GPU): every refusal
comes before any HIP call, struct layouts match the header, the frequencies,
and the 64-bit implementations that the GPU tests compare with."""
import ctypes
import math
import os
import shutil
import subprocess
import tempfile

import numpy as np
import pytest

import attention_ref as ref
import block_scaled_precision_mxfp4_amd as mx
from block_scaled_precision_mxfp4_amd import build as mxbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, SHAPE, ALIGN, WORKSPACE = -1, -2, -3, -6
REACHED = (0, -4, -5)  # past the checks: no device here


@pytest.fixture(scope="module", autouse=True)
def built():
    if mxbuild.is_stale():
        mxbuild.build()


STRUCTS = {"mxgemm_kv_cache": mx.KvCache, "mxgemm_append": mx.Append, "mxgemm_attention": mx.Attention}


def test_struct_layouts_match_the_header():
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    lines, want = [], []
    for cname, cls in STRUCTS.items():
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
    for pack, cls in ((mx._pack_cache, mx.KvCache), (mx._pack_append, mx.Append), (mx._pack_attention, mx.Attention)):
        v = [float(np.float32(rng.random())) if t is ctypes.c_float else int(rng.integers(1, 1 << 30)) for _, t in cls._fields_]
        assert pack(*v) == bytes(cls(*v))


def cache(**change):
    c = dict(k=0x1000, v=0x2000, page_stride=2048, head_stride=1024, token_stride=64, pages=0x3000, ld_pages=10, offsets=0x4000,
             lens=0x5000, k_scale=0, v_scale=0, num_pages=100, page_size=16, seqs=4, max_pages=10, kv_heads=2, head_dim=64, format=0)
    c.update(change)
    return mx.KvCache(**c)


def append(cache_=None, T=8, **change):
    p = dict(Q=0x10000, Q_out=0x20000, K=0x30000, V=0x40000, ldq=256, ldqo=256, ldk=128, ldv=128, freq=0x50000, factor=1.0, heads=4,
             rot_dim=64)
    p.update(change)
    c = cache() if cache_ is None else cache_
    return mx.lib().mxgemm_kv_append(bytes(c), bytes(mx.Append(**p)), T, None)


def attention(cache_=None, T=8, workspace=0x60000, nbytes=None, **change):
    p = dict(Q=0x10000, O=0x20000, ldq=256, ldo=256, scale=0.125, heads=4, causal=1)
    p.update(change)
    c = cache() if cache_ is None else cache_
    n = mx.mxgemm_paged_attention_workspace_bytes(T, 4, 4, 2, 64) if nbytes is None else nbytes
    return mx.lib().mxgemm_paged_attention(bytes(c), bytes(mx.Attention(**p)), T, workspace, n, None)


CACHES = [
    (INVALID, dict(offsets=0)), (INVALID, dict(lens=0)), (INVALID, dict(k=0)), (INVALID, dict(v=0)), (INVALID, dict(pages=0)),
    (INVALID, dict(format=2)), (INVALID, dict(format=-1)), (INVALID, dict(k_scale=0x100)), (INVALID, dict(v_scale=0x100)),
    (SHAPE, dict(seqs=0)), (SHAPE, dict(seqs=65537)), (SHAPE, dict(kv_heads=0)), (SHAPE, dict(head_dim=16)),
    (SHAPE, dict(head_dim=80)), (SHAPE, dict(head_dim=288, token_stride=288)), (SHAPE, dict(page_size=8)), (SHAPE, dict(page_size=24)),
    (SHAPE, dict(page_size=0)), (SHAPE, dict(page_size=-16)), (SHAPE, dict(page_size=131072)), (SHAPE, dict(num_pages=0)),
    (SHAPE, dict(max_pages=0)), (SHAPE, dict(max_pages=1 << 27, ld_pages=1 << 27)), (SHAPE, dict(ld_pages=9)),
    (SHAPE, dict(token_stride=56)), (SHAPE, dict(token_stride=1 << 26)), (SHAPE, dict(head_stride=0)), (SHAPE, dict(page_stride=-2048)),
    (SHAPE, dict(page_stride=1 << 62)), (SHAPE, dict(head_stride=1 << 62)),
    (ALIGN, dict(k=0x1008)), (ALIGN, dict(v=0x2004)), (ALIGN, dict(token_stride=68)), (ALIGN, dict(head_stride=1028)),
    (ALIGN, dict(page_stride=2052)), (ALIGN, dict(pages=0x3002)), (ALIGN, dict(offsets=0x4001)), (ALIGN, dict(lens=0x5002)),
    (ALIGN, dict(format=1, token_stride=72)), (ALIGN, dict(format=1, k_scale=0x102)), (ALIGN, dict(format=1, v_scale=0x101)),
]


@pytest.mark.parametrize("status,change", CACHES)
def test_caches_that_are_refused(status, change):
    assert append(cache(**change)) == status
    assert attention(cache(**change)) == status


def test_calls_that_pass_the_checks():
    assert append() in REACHED and attention() in REACHED
    f8 = cache(format=1, k_scale=0x100, v_scale=0x200)
    assert append(f8) in REACHED and attention(f8) in REACHED
    assert append(Q=0, Q_out=0, heads=0) in REACHED and append(rot_dim=0, freq=0) in REACHED
    assert append(cache(k=0, v=0, pages=0), K=0, V=0) in REACHED
    assert attention(O=0x10000) in REACHED and attention(O=0, A=0x70000, scaleA=0x80000, lda=256, ldsa=8) in REACHED
    assert mx.lib().mxgemm_kv_append(ctypes.byref(cache()), ctypes.byref(mx.Append(Q=0x100, Q_out=0x200, heads=4, ldq=256, ldqo=256)), 1, None) in REACHED


@pytest.mark.parametrize("status,change", [
    (INVALID, dict(Q=0)), (INVALID, dict(Q_out=0)), (INVALID, dict(K=0)), (INVALID, dict(V=0)), (INVALID, dict(Q=0, Q_out=0, K=0, V=0)),
    (INVALID, dict(interleaved=2)), (INVALID, dict(freq=0)), (SHAPE, dict(T=0)), (SHAPE, dict(T=-1)), (SHAPE, dict(T=(1 << 24) + 1)),
    (SHAPE, dict(heads=0)), (SHAPE, dict(heads=-3)), (SHAPE, dict(heads=509, ldq=1 << 20, ldqo=1 << 20)), (SHAPE, dict(rot_dim=-16)),
    (SHAPE, dict(rot_dim=80)), (SHAPE, dict(rot_dim=24)), (SHAPE, dict(ldq=248)), (SHAPE, dict(ldqo=255)), (SHAPE, dict(ldk=120)),
    (SHAPE, dict(ldv=0)), (ALIGN, dict(Q=0x10008)), (ALIGN, dict(Q_out=0x20002)), (ALIGN, dict(K=0x30004)), (ALIGN, dict(V=0x40001)),
    (ALIGN, dict(ldq=260)), (ALIGN, dict(ldqo=257)), (ALIGN, dict(ldk=132)), (ALIGN, dict(ldv=129)), (ALIGN, dict(positions=0x702)),
    (ALIGN, dict(freq=0x50004)),
])
def test_appends_that_are_refused(status, change):
    assert append(**change) == status
    assert mx.lib().mxgemm_kv_append(bytes(cache()), None, 8, None) == INVALID
    assert mx.lib().mxgemm_kv_append(None, bytes(mx.Append(Q=16, Q_out=16)), 8, None) == INVALID


@pytest.mark.parametrize("status,change", [
    (INVALID, dict(Q=0)), (INVALID, dict(O=0)), (INVALID, dict(A=0x70000, lda=256, ldsa=8)), (INVALID, dict(scaleA=0x80000)),
    (INVALID, dict(causal=2)), (INVALID, dict(scale=math.nan)), (INVALID, dict(scale=math.inf)), (INVALID, dict(a_format=2)),
    (SHAPE, dict(T=0)), (SHAPE, dict(T=(1 << 24) + 1)), (SHAPE, dict(heads=0)), (SHAPE, dict(heads=3)), (SHAPE, dict(heads=1)),
    (SHAPE, dict(heads=510, ldq=1 << 20, ldo=1 << 20)), (SHAPE, dict(window=-1)), (SHAPE, dict(max_new=-1)), (SHAPE, dict(ldq=248)),
    (SHAPE, dict(ldo=128)), (SHAPE, dict(A=0x70000, scaleA=0x80000, lda=224, ldsa=8)), (SHAPE, dict(A=0x70000, scaleA=0x80000, lda=256, ldsa=7)),
    (ALIGN, dict(Q=0x10008)), (ALIGN, dict(ldq=260)), (ALIGN, dict(O=0x20008)), (ALIGN, dict(ldo=260)), (ALIGN, dict(lse=0x702)),
    (ALIGN, dict(sinks=0x701)), (ALIGN, dict(A=0x70008, scaleA=0x80000, lda=256, ldsa=8)), (ALIGN, dict(A=0x70000, scaleA=0x80000, lda=272, ldsa=9)),
    (ALIGN, dict(A=0x70000, scaleA=0x80000, lda=264, ldsa=8, a_format=1)), (WORKSPACE, dict(workspace=None)), (WORKSPACE, dict(nbytes=4096)),
    (ALIGN, dict(workspace=0x60008)),
])
def test_attentions_that_are_refused(status, change):
    assert attention(**change) == status
    assert mx.lib().mxgemm_paged_attention(bytes(cache()), None, 8, 0x1000, 1 << 30, None) == INVALID


def test_work_that_would_not_be_countable_is_refused():
    big = cache(max_pages=(1 << 27) - 1, ld_pages=(1 << 27) - 1)
    assert attention(big, T=1 << 20, nbytes=1 << 40) == SHAPE
    assert attention(big, T=1) in REACHED


def test_outputs_in_place_with_other_strides_are_refused():
    assert append(Q_out=0x10000, ldqo=264) == SHAPE
    assert attention(O=0x10000, ldo=264) == SHAPE
    assert append(Q_out=0x10000) in REACHED and attention(O=0x10000) in REACHED


def test_more_rows_than_a_grid_has_are_refused():
    assert mx.mxgemm_paged_attention_workspace_bytes(1 << 24, 1, 64, 64, 32) > 0
    assert mx.mxgemm_paged_attention_workspace_bytes(1 << 24, 1, 65, 65, 32) == 0


@pytest.mark.parametrize("shape", [(0, 1, 4, 2, 64), (1, 0, 4, 2, 64), (1, 1, 4, 3, 64), (1, 1, 4, 2, 65), (1, 1, 2, 4, 64), (1 << 25, 1, 4, 2, 64)])
def test_workspace_of_an_invalid_shape(shape):
    assert mx.mxgemm_paged_attention_workspace_bytes(*shape) == 0


def test_workspace_is_enough_for_every_smaller_call():
    for D in (32, 64, 96, 128, 256):
        most = mx.mxgemm_paged_attention_workspace_bytes(1 << 20, 4096, 32, 4, D)
        assert 4096 < mx.mxgemm_paged_attention_workspace_bytes(1, 1, 32, 4, D) <= most < 192 << 20


def test_frequencies():
    plain = mx.mxgemm_rope_frequencies(128, 10000.0)
    assert np.allclose(plain, 10000.0 ** (-np.arange(64) / 64), rtol=1e-15)
    assert np.allclose(mx.mxgemm_rope_frequencies(128, 10000.0, 4.0), np.array(plain) / 4, rtol=1e-15)
    got = np.array(mx.mxgemm_rope_frequencies(128, 10000.0, 8.0, 8192, 1, 4))
    turns = 8192 * np.array(plain) / (2 * np.pi)
    assert np.array_equal(got[turns >= 4], np.array(plain)[turns >= 4])
    assert np.allclose(got[turns <= 1], np.array(plain)[turns <= 1] / 8, rtol=1e-15)
    mid = (turns > 1) & (turns < 4)
    keep = (turns[mid] - 1) / 3
    assert mid.any() and np.allclose(got[mid], np.array(plain)[mid] * (keep + (1 - keep) / 8), rtol=1e-14)


@pytest.mark.parametrize("status,a", [
    (INVALID, (64, 0.0, 1, 0, 0, 0)), (INVALID, (64, math.nan, 1, 0, 0, 0)), (INVALID, (64, math.inf, 1, 0, 0, 0)),
    (INVALID, (64, 1e4, 0, 0, 0, 0)), (INVALID, (64, 1e4, -1, 0, 0, 0)), (INVALID, (64, 1e4, 2, 0, 1, 4)),
    (INVALID, (64, 1e4, 2, 100, 4, 4)), (INVALID, (64, 1e4, 2, 100, -1, 4)), (INVALID, (64, 1e4, 2, 100, 1, math.inf)),
    (INVALID, (64, 1e4, 2, 100, math.nan, 4)), (SHAPE, (0, 1e4, 1, 0, 0, 0)), (SHAPE, (63, 1e4, 1, 0, 0, 0)), (SHAPE, (258, 1e4, 1, 0, 0, 0)),
])
def test_frequencies_that_are_refused(status, a):
    assert mx.lib().mxgemm_rope_frequencies((ctypes.c_double * 128)(), a[0], *map(float, a[1:])) == status
    assert mx.lib().mxgemm_rope_frequencies(None, 64, 1e4, 1.0, 0.0, 0.0, 0.0) == INVALID


# ---- the 64-bit implementations ------------------------------------------------

def test_e4m3_reference():
    v = ref.e4m3_values()
    fine = v[:127]
    assert fine[0] == 0 and fine[1] == 2.0 ** -9 and fine[8] == 2.0 ** -6 and fine[126] == 448 and np.isnan(v[127])
    assert np.array_equal(ref.to_e4m3(fine), np.arange(127)) and np.array_equal(ref.to_e4m3(-fine[1:]), np.arange(129, 255))
    mid = (fine[:-1] + fine[1:]) / 2  # ties go to the even code
    assert (ref.to_e4m3(mid) % 2 == 0).all()
    assert np.array_equal(ref.to_e4m3(np.nextafter(mid, 1e9)), np.arange(1, 127))


def small(new, lens, D=32, P=16, heads=1):
    rng = np.random.default_rng(3)
    S, per = len(new), max(-(-max(n, 1) // P) for n in lens)
    pages = rng.permutation(S * per).reshape(S, per)
    return dict(offsets=np.concatenate(([0], np.cumsum(new))), lens=np.array(lens), pages=pages, page_size=P, num_pages=S * per,
                k=rng.standard_normal((S * per, heads, P, D)), v=rng.standard_normal((S * per, heads, P, D)))


def test_attention_reference_against_sums():
    b = small([2, 3], [20, 3])
    rng = np.random.default_rng(4)
    q = rng.standard_normal((5, 2, 32))
    O, lse, _, _ = ref.attention(q, b, 0.2, True, 0, sinks=np.array([0.3, -1.0]))
    for s, t, h in ((0, 1, 0), (1, 2, 1), (1, 4, 0)):
        row = t - b["offsets"][s]
        p = b["lens"][s] - (b["offsets"][s + 1] - b["offsets"][s]) + row
        num, den = np.zeros(32), math.exp([0.3, -1.0][h])
        for j in range(p + 1):
            k, v = (b[x][b["pages"][s, j // 16], 0, j % 16] for x in ("k", "v"))
            e = math.exp(0.2 * float(k @ q[t, h]))
            num, den = num + e * v, den + e
        assert np.allclose(O[t, h], num / den, rtol=1e-12) and np.isclose(lse[t, h], math.log(den), rtol=1e-12)
    # a window of one sees itself alone
    O, _, _, _ = ref.attention(q, b, 0.2, True, 1)
    assert np.allclose(O[0, 0], b["v"][b["pages"][0, 1], 0, 2])


def test_bounds_hold_for_a_float32_and_bf16_evaluation():
    """What the kernels round, done in numpy: products and sums in float32, p in bf16, O in bf16."""
    b = small([4], [200])
    b["k"], b["v"] = (ref.bf16_to_f64(ref.f64_to_bf16(b[x])) for x in ("k", "v"))
    q = ref.bf16_to_f64(ref.f64_to_bf16(2 * np.random.default_rng(5).standard_normal((4, 1, 32))))
    O, lse, off, off_lse = ref.attention(q, b, 32 ** -0.5, True, 0)
    k, v = (ref.gather(b, 0, 200, b[x])[0].astype(np.float32) for x in ("k", "v"))
    for t in range(4):
        n = 197 + t
        x = (k[:n] @ q[t, 0].astype(np.float32)) * np.float32(32 ** -0.5)
        e = np.exp(x - x.max())
        p = ref.bf16_to_f64(ref.f64_to_bf16(e.astype(np.float64))).astype(np.float32)
        o = ref.bf16_to_f64(ref.f64_to_bf16((p @ v[:n] / e.sum(dtype=np.float32)).astype(np.float64)))
        assert (np.abs(o - O[t, 0]) <= off[t, 0]).all()
        assert abs(x.max() + np.log(e.sum(dtype=np.float32)) - lse[t, 0]) <= off_lse[t, 0]


def test_append_reference():
    b = small([3], [30])
    rng = np.random.default_rng(6)
    x = rng.standard_normal((3, 1, 32))
    freq = mx.mxgemm_rope_frequencies(32)
    for inter in (False, True):
        q, _, places = ref.append(b, x, x, x, freq, 32, inter, 1.0)
        assert np.allclose(np.linalg.norm(q, axis=-1), np.linalg.norm(x, axis=-1))
        # scores go by the positions' difference
        back, _, _ = ref.append(b, x, x, x, freq, 32, inter, 1.0, positions=[1000, 1001, 1002])
        assert np.isclose((q[0, 0] * q[2, 0]).sum(), (back[0, 0] * back[2, 0]).sum())
        assert set(places) == {(b["pages"][0, p // 16], p % 16) for p in (27, 28, 29)}
        # the inverse turn gives x again
        again, _ = ref.turn(q[1], -28, freq, 32, inter, 1.0)
        assert np.allclose(again, x[1])
