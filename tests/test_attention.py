"""GPU tests of the append to a paged cache and of the attention over it,
against 64-bit plain implementations (attention_ref.py, where the tolerances
are derived)."""
import sys

import numpy as np
import pytest

import attention_ref as ref
import block_scaled_precision_mxfp4_amd as mx
import experts_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mxgpu import dev_bf16, host_bits  # noqa: E402

E4M3 = ref.e4m3_values()


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bf16(rng, *shape, sigma=1.0):
    return ref.f64_to_bf16(rng.standard_normal(shape) * sigma)


class Batch:
    """A cache and a batch on the device, and the same as the reference has them."""

    def __init__(self, rng, new, lens, kv_heads, D, page=16, fp8=False, layout="head", spare=2, shuffle=True):
        S = len(new)
        per = [max(-(-n // page), 0) for n in lens]
        self.max_pages = max(max(per), 1) + 1
        self.num_pages = sum(per) + spare
        order = rng.permutation(self.num_pages) if shuffle else np.arange(self.num_pages)
        pages = np.full((S, self.max_pages), -3, np.int32)
        at = 0
        for s in range(S):
            pages[s, :per[s]] = order[at:at + per[s]]
            at += per[s]
        self.new, self.kv_heads, self.D, self.page, self.fp8, self.S = new, kv_heads, D, page, fp8, S
        self.T = sum(new)
        shape = (self.num_pages, kv_heads, page, D)
        if fp8:
            self.k_scale, self.v_scale = (rng.uniform(0.5, 2.0, kv_heads).astype(np.float32) / 64 for _ in range(2))
            self.kc, self.vc = (ref.to_e4m3(rng.standard_normal(shape) * 64) for _ in range(2))
        else:
            self.k_scale = self.v_scale = None
            self.kc, self.vc = bf16(rng, *shape), bf16(rng, *shape)
        self.offsets = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
        self.lens, self.pages, self.layout = np.array(lens, np.int32), pages, layout

    def values(self, codes, scale):
        if self.fp8:
            return E4M3[codes] * scale.astype(np.float64)[:, None, None]
        return ref.bf16_to_f64(codes)

    def host(self):
        return dict(offsets=self.offsets, lens=self.lens, pages=self.pages, page_size=self.page, num_pages=self.num_pages,
                    k=self.values(self.kc, self.k_scale), v=self.values(self.vc, self.v_scale))

    def cache(self):
        """layout: head: [page][head][row]; token: [page][row][head]; wide: rows and pages further apart."""
        def lay(codes):
            x = codes.transpose(0, 2, 1, 3) if self.layout == "token" else codes
            if self.layout == "wide":
                junk = np.full((*x.shape[:-1], self.D + 32), 0x7F if self.fp8 else 0x7FC0, x.dtype)  # NaN behind a row
                junk[..., :self.D] = x
                x = junk
            x = np.ascontiguousarray(x)
            return dev(x if self.fp8 else x.view(np.int16))
        self.k, self.v = lay(self.kc), lay(self.vc)
        D, P, H = self.D, self.page, self.kv_heads
        strides = {"head": {}, "token": dict(token_stride=H * D, head_stride=D, page_stride=P * H * D),
                   "wide": dict(token_stride=D + 32)}[self.layout]
        self.dev = [dev(x) for x in (self.pages, self.offsets, self.lens)]
        self.scales = [None if x is None else dev(x) for x in (self.k_scale, self.v_scale)]
        self.strides = strides
        return self.bind()

    def bind(self):
        return mx.make_kv_cache(self.k, self.v, *self.dev, seqs=self.S, num_pages=self.num_pages, page_size=self.page,
                                max_pages=self.max_pages, kv_heads=self.kv_heads, head_dim=self.D, fp8=self.fp8,
                                k_scale=self.scales[0], v_scale=self.scales[1], **self.strides)

    def pools(self):
        """What the device's cache holds, in the reference's order."""
        def back(x):
            x = x.cpu().numpy()
            x = x if self.fp8 else x.view(np.uint16)
            x = x[..., :self.D]
            return x.transpose(0, 2, 1, 3) if self.layout == "token" else x
        return back(self.k), back(self.v)


def workspace(T, S, H, Hk, D):
    n = mx.mxgemm_paged_attention_workspace_bytes(T, S, H, Hk, D)
    w = torch.zeros(n, dtype=torch.uint8, device="cuda")
    w[4096:] = 0xFF  # (NaN)
    return w


def attend(b, q, H, scale=None, causal=True, window=0, sinks=None, pad=0, rows=None, w=None, max_new=0, **more):
    T = b.T if rows is None else rows
    D = b.D
    scale = D ** -0.5 if scale is None else scale
    qq = np.full((T, H * D + pad), 0x7FC0, np.uint16)
    qq[:, :H * D] = q.reshape(T, -1)
    O = dev_bf16(np.full((T, H * D + pad), 0x1234, np.uint16))
    lse = torch.full((T, H), 77.0, device="cuda")
    w = workspace(T, b.S, H, b.kv_heads, D) if w is None else w
    mx.mxgemm_paged_attention(b.cache(), T, dev_bf16(qq), O, heads=H, scale=scale, lse=lse, ldq=H * D + pad, ldo=H * D + pad,
                              causal=causal, window=window, sinks=None if sinks is None else dev(sinks.astype(np.float32)),
                              workspace=w, workspace_bytes=w.numel(), max_new=max_new, **more)
    torch.cuda.synchronize()
    assert not w[:4096].any()
    bits = host_bits(O)
    assert (bits[:, H * D:] == 0x1234).all()
    return bits[:, :H * D].reshape(T, H, D), lse.cpu().numpy()


def check(b, q, H, got, scale=None, causal=True, window=0, sinks=None):
    O, lse, off, off_lse = ref.attention(ref.bf16_to_f64(q).reshape(-1, H, b.D), b.host(), b.D ** -0.5 if scale is None else scale,
                                         causal, window, sinks)
    bits, l = got
    none = np.isnan(lse) & (off_lse == 0)  # rows that no sequence has
    assert (bits[none] == 0x1234).all() and (l[none] == 77).all()
    o = ref.bf16_to_f64(bits)
    some = ~none
    with np.errstate(invalid="ignore"):
        bad = np.abs(o - O) > off
        bad |= np.isnan(o) != np.isnan(O)
        bad[np.isinf(O)] = o[np.isinf(O)] != O[np.isinf(O)]
    assert not bad[some].any(), "%d of %d, worst %.3g of its bound" % (bad[some].sum(), bad[some].size, np.nanmax((np.abs(o - O) / off)[some]))
    empty = np.isneginf(lse)
    assert np.isneginf(l[empty]).all()
    rest = some & np.isfinite(lse)
    assert (np.abs(l - lse)[rest] <= off_lse[rest]).all()


CASES = [  # new, lens, heads, kv_heads, D, page, fp8
    ([1], [1], 1, 1, 64, 16, False),
    ([1], [33], 4, 2, 128, 16, False),
    ([1], [700], 8, 2, 128, 16, False),
    ([1, 1, 1], [5, 129, 300], 5, 1, 128, 32, True),
    ([1] * 9, [1, 2, 31, 32, 33, 127, 128, 129, 1000], 16, 2, 64, 16, False),
    ([1, 1], [250, 91], 4, 4, 256, 64, False),
    ([1, 1], [250, 91], 16, 1, 256, 16, True),
    ([3, 0, 1, 17], [40, 77, 1, 17], 6, 2, 96, 16, False),
    ([3, 0, 1, 17], [40, 77, 1, 17], 6, 2, 160, 32, True),
    ([70, 5], [70, 205], 8, 1, 64, 128, True),
    ([40, 1, 90], [333, 20, 90], 3, 1, 128, 16, False),
    ([130], [130], 2, 2, 32, 16, False),
    ([65], [300], 12, 4, 64, 16, True),
]


@pytest.mark.parametrize("layout", ["head", "token", "wide"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(case, layout):
    new, lens, H, Hk, D, page, fp8 = CASES[case]
    rng = np.random.default_rng(100 + case)
    b = Batch(rng, new, lens, Hk, D, page, fp8, layout)
    q = bf16(rng, b.T, H * D, sigma=2.0)
    say("case attention", case, layout)
    got = attend(b, q, H, pad=8 * (layout == "wide"))
    check(b, q, H, got)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 5, 40, 200])
@pytest.mark.parametrize("sinks", [False, True])
def test_masks_and_sinks(causal, window, sinks):
    rng = np.random.default_rng(7)
    b = Batch(rng, [1, 50, 7, 0], [400, 50, 180, 9], 2, 64, 16, False)
    q = bf16(rng, b.T, 6 * 64, sigma=2.0)
    k = np.array([0.5, -3.0, 8.0, 0.0, -np.inf, 2.0]) if sinks else None
    say("case masks", causal, window, sinks)
    check(b, q, 6, attend(b, q, 6, causal=causal, window=window, sinks=k), causal=causal, window=window, sinks=k)


@pytest.mark.parametrize("scale", [0.0, -0.1, 1e-30, 3.0])
def test_scales(scale):
    rng = np.random.default_rng(8)
    b = Batch(rng, [2, 40], [90, 60], 1, 64, 16, True)
    q = bf16(rng, b.T, 4 * 64)
    check(b, q, 4, attend(b, q, 4, scale=scale), scale=scale)


def test_rows_without_keys_or_sequence():
    """Sequences shorter than their new tokens, of no tokens, pages that do not exist, rows behind the last sequence."""
    rng = np.random.default_rng(9)
    b = Batch(rng, [4, 3, 2, 40], [2, 0, 50, 41], 2, 64, 16, False)
    b.pages[2, 1], b.pages[3, 0] = -1, b.num_pages  # read as zeros
    rows = b.T + 5
    q = bf16(rng, rows, 4 * 64)
    got = attend(b, q, 4, rows=rows)
    check(b, q, 4, got)
    assert (got[0][b.T:] == 0x1234).all()
    assert (got[0][:2] == 0).all() and np.isneginf(got[1][:2]).all()
    check(b, q, 4, attend(b, q, 4, rows=rows, causal=False), causal=False)


@pytest.mark.parametrize("fp8", [False, True])
def test_special_values_in_places_that_a_row_does_not_see(fp8):
    rng = np.random.default_rng(10)
    b = Batch(rng, [12, 70, 1], [45, 70, 200], 1, 64, 16, fp8)
    nan, inf = (0x7F, 0xFF) if fp8 else (0x7FC0, 0x7F80)
    b.kc[:, :, :, :], b.vc[:, :, :, :] = b.kc, b.vc
    used = {(int(b.pages[s, i // 16]), i % 16) for s in range(3) for i in range(b.lens[s])}
    for p in range(b.num_pages):  # what no sequence has
        for r in range(16):
            if (p, r) not in used:
                b.kc[p, :, r], b.vc[p, :, r] = nan, nan
    # keys that only later tokens see, and one behind a window
    for s, i in ((0, 40), (1, 33), (1, 64), (2, 20)):
        b.vc[b.pages[s, i // 16], 0, i % 16, ::3] = nan
        b.kc[b.pages[s, i // 16], 0, i % 16, 5] = nan
    b.vc[b.pages[1, 2], 0, 9, 7] = inf
    q = bf16(rng, b.T, 4 * 64)
    say("case specials", fp8)
    check(b, q, 4, attend(b, q, 4))
    check(b, q, 4, attend(b, q, 4, window=30), window=30)


def test_infinite_scores():
    rng = np.random.default_rng(11)
    b = Batch(rng, [3], [60], 1, 64, 16, False)
    b.kc[b.pages[0, 1], 0, 4] = 0xFF80  # -inf against a positive query
    q = np.abs(ref.bf16_to_f64(bf16(rng, b.T, 2 * 64)))
    q = ref.f64_to_bf16(q)
    check(b, q, 2, attend(b, q, 2))
    b.kc[:] = 0xFF80  # every score -inf: as if the row saw no key
    O, lse = attend(b, q, 2)
    assert (O == 0).all() and np.isneginf(lse).all()


def test_long_context_of_one_token():
    """Every workgroup has a part of one sequence; and a workspace used again for other sizes."""
    rng = np.random.default_rng(12)
    w = max((workspace(64, 64, 16, 1, D) for D in (64, 128, 256)), key=len)
    for new, lens, H, Hk, D in (([1], [9000], 4, 1, 128), ([1, 1], [3000, 40], 8, 2, 64), ([2], [5000], 2, 1, 256), ([1], [9000], 4, 1, 128)):
        b = Batch(rng, new, lens, Hk, D, 64, False)
        q = bf16(rng, b.T, H * D, sigma=2.0)
        say("case long", lens)
        first = attend(b, q, H, w=w)
        check(b, q, H, first)
        again = attend(b, q, H, w=w)
        assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


@pytest.mark.parametrize("seqs", [63, 64, 65, 130, 700])
def test_many_sequences(seqs):
    rng = np.random.default_rng(13)
    new = [int(x) for x in rng.choice([0, 1, 1, 1, 2], seqs)]
    lens = [n + int(rng.integers(0, 60)) for n in new]
    b = Batch(rng, new, lens, 1, 32, 16, False)
    q = bf16(rng, b.T, 2 * 32)
    say("case seqs", seqs)
    check(b, q, 2, attend(b, q, 2))


def test_offsets_that_do_not_ascend_form_no_address_outside():
    """Values mean nothing then; later calls with the workspace are right."""
    rng = np.random.default_rng(14)
    b = Batch(rng, [1, 1, 1, 1], [50, 60, 70, 80], 1, 64, 16, False)
    q = bf16(rng, b.T, 2 * 64)
    w = workspace(4, 4, 2, 1, 64)
    good = b.offsets.copy(), b.lens.copy(), b.pages.copy()
    for bad in ([0, 4, 0, 4, 0], [3, 1, 9, -5, 2], [2 ** 31 - 1, -2 ** 31, 0, 4, 4], [0, 1, 2, 3, 100]):
        b.offsets = np.array(bad, np.int32)
        b.lens = np.array([2 ** 31 - 1, -7, 70, 10 ** 6], np.int32)
        b.pages = np.where(rng.random(b.pages.shape) < 0.5, 2 ** 31 - 1, b.pages).astype(np.int32)
        say("case offsets", bad)
        attend(b, q, 2, w=w)
    b.offsets, b.lens, b.pages = good
    check(b, q, 2, attend(b, q, 2, w=w))


def test_output_in_place_of_q():
    rng = np.random.default_rng(15)
    b = Batch(rng, [1, 40], [2000, 900], 2, 64, 16, False)
    q = bf16(rng, b.T, 4 * 64)
    want = attend(b, q, 4)
    w = workspace(b.T, 2, 4, 2, 64)
    x = dev_bf16(q.reshape(b.T, -1))
    mx.mxgemm_paged_attention(b.cache(), b.T, x, x, heads=4, scale=64 ** -0.5, ldq=256, ldo=256, workspace=w, workspace_bytes=w.numel())
    torch.cuda.synchronize()
    assert np.array_equal(host_bits(x).reshape(want[0].shape), want[0])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 256])
def test_quantized_rows(D, fp8):
    """A and scaleA are the bf16 rows quantized, split over workgroups or not, with and without O."""
    rng = np.random.default_rng(16)
    b = Batch(rng, [1, 3, 40], [1500, 20, 100], 1, D, 16, False)
    H = 4
    q = bf16(rng, b.T, H * D)
    b.vc[b.pages[1, 0], 0, 2, 3] = 0x7F80
    bytes_ = H * D if fp8 else H * D // 2
    pitch = -(-bytes_ // 16) * 16 + 16
    w = workspace(b.T, 3, H, 1, D)
    A = torch.full((b.T, pitch), 0xAB, dtype=torch.uint8, device="cuda")
    S = torch.full((b.T, H * D // 32 + 3), 0xCD, dtype=torch.uint8, device="cuda")
    more = dict(A=A, scaleA=S, lda=pitch if fp8 else 2 * pitch, ldsa=S.shape[1], a_format=mx.FMT_FP8_E4M3 if fp8 else mx.FMT_FP4)
    O, _ = attend(b, q, H, **more)
    want = experts_ref.quantize(O.reshape(b.T, -1), fp8)
    got = A.cpu().numpy(), S.cpu().numpy()
    assert np.array_equal(got[0][:, :bytes_], want[0]) and (got[0][:, bytes_:] == 0xAB).all()
    assert np.array_equal(got[1][:, :H * D // 32], want[1]) and (got[1][:, H * D // 32:] == 0xCD).all()
    A.zero_()
    mx.mxgemm_paged_attention(b.bind(), b.T, dev_bf16(q.reshape(b.T, -1)), heads=H, scale=D ** -0.5, ldq=H * D, workspace=w, workspace_bytes=w.numel(), **more)
    assert np.array_equal(A.cpu().numpy()[:, :bytes_], want[0])


# ---- append -------------------------------------------------------------------

def run_append(b, q, k, v, H, freq, rot, interleaved, factor=1.0, positions=None, in_place=False, pad=0, rows=None):
    T = b.T if rows is None else rows
    D = b.D

    def lay(x, heads):
        y = np.full((T, heads * D + pad), 0x7FC0, np.uint16)
        y[:, :heads * D] = x.reshape(T, -1)
        return dev_bf16(y)
    cache = b.cache()
    qd = None if q is None else lay(q, H)
    out = None if q is None else qd if in_place else dev_bf16(np.full((T, H * D + pad), 0x1234, np.uint16))
    kd, vd = (None, None) if k is None else (lay(k, b.kv_heads), lay(v, b.kv_heads))
    f = dev(np.asarray(freq, np.float64)) if rot else None
    pos = None if positions is None else dev(np.asarray(positions, np.int32))
    mx.mxgemm_kv_append(cache, T, Q=qd, Q_out=out, K=kd, V=vd, heads=H if q is not None else 0, ldq=H * D + pad, ldqo=H * D + pad,
                        ldk=b.kv_heads * D + pad, ldv=b.kv_heads * D + pad, freq=f, rot_dim=rot, interleaved=interleaved,
                        factor=factor, positions=pos)
    torch.cuda.synchronize()
    return None if q is None else host_bits(out)[:, :H * D].reshape(T, H, D)


def check_append(b, q, k, v, H, got, freq, rot, interleaved, factor=1.0, positions=None, in_place=False, rows=None):
    T = b.T if rows is None else rows
    D = b.D
    f64 = lambda x, heads: None if x is None else ref.bf16_to_f64(x).reshape(T, heads, D)  # noqa: E731
    out, qmag, places = ref.append(b.host(), f64(q, H), f64(k, b.kv_heads), f64(v, b.kv_heads), freq, rot, interleaved, factor, positions)
    if q is not None:
        none = np.isnan(out).all(axis=(1, 2))
        left = q.reshape(T, H, D) if in_place else np.full((T, H, D), 0x1234, np.uint16)
        assert np.array_equal(got[none], left[none])
        o = ref.bf16_to_f64(got)
        with np.errstate(invalid="ignore"):
            assert (np.abs(o - out) <= ref.BF16 * np.abs(out) + 1.01 * ref.TURN * qmag + 2.0 ** -133)[~none].all()
        same = slice(rot, D)
        assert np.array_equal(got[~none][..., same], q.reshape(T, H, D)[~none][..., same])
    kg, vg = b.pools()
    kept = np.ones(kg.shape[:3], bool)
    for (page, row), (kk, mag, vv) in places.items():
        kept[page, :, row] = False
        if b.fp8:
            sk, sv = (x.astype(np.float64)[:, None] for x in (b.k_scale, b.v_scale))
            assert np.array_equal(vg[page, :, row], ref.to_e4m3((vv.astype(np.float32) / b.v_scale[:, None]).astype(np.float32)))
            want = np.clip(kk / sk, -448, 448)
            # half a step of E4M3 (2^-10 below its normal range), the turn's error and the quotient's rounding
            tol = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) + 1.1 * (ref.TURN * mag / sk + 2 * ref.F32 * np.abs(want))
            assert (np.abs(E4M3[kg[page, :, row]] - want) <= tol).all()
        else:
            assert np.array_equal(vg[page, :, row], ref.f64_to_bf16(vv))
            assert (np.abs(ref.bf16_to_f64(kg[page, :, row]) - kk) <= ref.BF16 * np.abs(kk) + 1.01 * ref.TURN * mag + 2.0 ** -133).all()
    assert np.array_equal(kg[kept], b.kc[kept]) and np.array_equal(vg[kept], b.vc[kept])


APPENDS = [  # new, lens, heads, kv_heads, D, page, fp8, rot, interleaved
    ([1], [1], 1, 1, 32, 16, False, 32, False),
    ([1], [500], 32, 8, 128, 16, False, 128, False),
    ([1], [500], 32, 8, 128, 16, True, 128, True),
    ([3, 0, 1, 17], [40, 77, 1, 17], 6, 2, 96, 16, True, 48, False),
    ([3, 0, 1, 17], [40, 77, 1, 17], 6, 2, 96, 32, False, 16, True),
    ([33, 64], [33, 100000], 5, 5, 64, 64, False, 64, False),
    ([33, 64], [33, 100000], 4, 1, 256, 64, True, 0, False),
    ([2] * 80, [int(x) for x in range(2, 82)], 2, 1, 64, 16, False, 64, True),
]


@pytest.mark.parametrize("layout", ["head", "token", "wide"])
@pytest.mark.parametrize("case", range(len(APPENDS)))
def test_append(case, layout):
    new, lens, H, Hk, D, page, fp8, rot, inter = APPENDS[case]
    rng = np.random.default_rng(200 + case)
    # (only the new tokens' pages exist)
    b = Batch(rng, new, [min(n, 200) for n in lens], Hk, D, page, fp8, layout)
    positions = None
    if max(lens) > 200:
        positions = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)])
    q, k, v = (bf16(rng, b.T, h * D) for h in (H, Hk, Hk))
    freq = mx.mxgemm_rope_frequencies(rot) if rot else []
    say("case append", case, layout)
    for in_place in (False, True):
        got = run_append(b, q, k, v, H, freq, rot, inter, positions=positions, in_place=in_place, pad=8 * (layout == "wide"))
        check_append(b, q, k, v, H, got, freq, rot, inter, positions=positions, in_place=in_place)


def test_append_far_positions_and_factor():
    rng = np.random.default_rng(21)
    b = Batch(rng, [6], [6], 1, 64, 16, False)
    q, k, v = (bf16(rng, 6, h * 64) for h in (2, 1, 1))
    freq = mx.mxgemm_rope_frequencies(64, base=500000.0, factor=32.0, original=8192, low=1, high=4)
    pos = [0, 1, -5, 131071, 2 ** 24 + 1, 2 ** 31 - 1]
    got = run_append(b, q, k, v, 2, freq, 64, False, factor=1.2, positions=pos)
    check_append(b, q, k, v, 2, got, freq, 64, False, factor=1.2, positions=pos)


def test_append_tokens_without_a_place():
    rng = np.random.default_rng(22)
    b = Batch(rng, [4, 3, 2, 20], [2, 0, 50, 41], 2, 64, 16, False)
    b.pages[2, 3], b.pages[3, 2] = -1, b.num_pages
    rows = b.T + 3
    q, k, v = (bf16(rng, rows, h * 64) for h in (4, 2, 2))
    freq = mx.mxgemm_rope_frequencies(64)
    got = run_append(b, q, k, v, 4, freq, 64, False, rows=rows)
    check_append(b, q, k, v, 4, got, freq, 64, False, rows=rows)
    for bad in ([0, 4, 0, 4, 0], [3, 1, 9, -5, 2], [2 ** 31 - 1, -2 ** 31, 0, 4, 4], [5, 6, 7, 8, 2 ** 31 - 1]):
        b.offsets = np.array(bad, np.int32)
        b.lens = np.array([2 ** 31 - 1, -7, 70, 10 ** 6], np.int32)
        say("case append offsets", bad)
        run_append(b, q, k, v, 4, freq, 64, False, rows=rows)


def test_append_parts_alone():
    rng = np.random.default_rng(23)
    b = Batch(rng, [5, 9], [30, 9], 2, 64, 16, True)
    q, k, v = (bf16(rng, b.T, h * 64) for h in (6, 2, 2))
    freq = mx.mxgemm_rope_frequencies(32)
    got = run_append(b, q, None, None, 6, freq, 32, True)
    check_append(b, q, None, None, 6, got, freq, 32, True)
    run_append(b, None, k, v, 6, freq, 32, True)
    check_append(b, None, k, v, 6, None, freq, 32, True)


@pytest.mark.parametrize("fp8", [False, True])
def test_append_special_values(fp8):
    rng = np.random.default_rng(24)
    b = Batch(rng, [3], [3], 1, 32, 16, fp8)
    k, v = (bf16(rng, 3, 32) for _ in range(2))
    v[0, :6] = [0x7F80, 0xFF80, 0x7FC0, 0x7F7F, 0x8000, 0x0001]
    k[1, 20:23] = [0x7F80, 0x7FC0, 0xFF80]  # behind the turned part
    run_append(b, None, k, v, 1, mx.mxgemm_rope_frequencies(16), 16, False)
    kg, vg = b.pools()
    page = b.pages[0, 0]
    if fp8:
        want = E4M3[ref.to_e4m3(np.clip(ref.bf16_to_f64(v).astype(np.float32) / b.v_scale[0], -448, 448).astype(np.float32))]
        assert np.array_equal(E4M3[vg[page, 0, :3]], want, equal_nan=True)
        assert np.array_equal(E4M3[kg[page, 0, 1, 20:23]], [448, np.nan, -448], equal_nan=True)
    else:
        assert np.array_equal(vg[page, 0, :3], v) and np.array_equal(kg[page, 0, 1, 16:], k[1, 16:])
