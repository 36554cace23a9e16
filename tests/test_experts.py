"""GPU tests of the mixture-of-experts operators against 64-bit plain
implementations (experts_ref.py, where the tolerances are derived): each
operator over its types, sizes and special values, and the whole block as a
user runs it, eagerly, on another stream and from replayed graphs."""
import sys

import numpy as np
import pytest

import block_scaled_precision_mxfp4_amd as mx
import experts_ref as ref
from block_scaled_precision_mxfp4_amd import inputs

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mxgpu import dev_bf16, dev_u8, host_bits  # noqa: E402


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def i32(*shape, fill=-7):
    return torch.full(shape, fill, dtype=torch.int32, device="cuda")


def bf16_bits(rng, *shape, sigma=1.0):
    return ref.f64_to_bf16(rng.standard_normal(shape) * sigma)


# ---- router choice ------------------------------------------------------------

def run_route(x, k, renorm, bf16, ldl=None, stream=None):
    T, E = x.shape
    ldl = E if ldl is None else ldl
    pad = np.full((T, ldl), 1e30, np.float32)  # what is behind a row must not be read
    pad[:, :E] = x
    logits = dev_bf16(ref.f64_to_bf16(pad)) if bf16 else dev(pad)
    n = mx.mxgemm_route_workspace_bytes(T, E)
    ws = torch.full((max(n, 4),), 0xEE, dtype=torch.uint8, device="cuda")
    out = dict(ids=i32(T, k), weights=torch.full((T, k), np.nan, device="cuda"), pos=i32(T, k), offsets=i32(E + 1), rows=i32(T * k))
    mx.mxgemm_route(*out.values(), logits, T, E, k, ldl=ldl, bf16=bf16, renorm=renorm, workspace=ws, workspace_bytes=n)
    torch.cuda.synchronize()
    return {a: t.cpu().numpy() for a, t in out.items()}


def check_route(x, k, renorm, got):
    ids, weights, pos, offsets, rows = ref.route(x, k, renorm)
    for name, want in (("ids", ids), ("pos", pos), ("offsets", offsets), ("rows", rows)):
        assert np.array_equal(got[name], want), name
    rel, small = ref.route_weight_tol(x, x.shape[1])
    assert (np.abs(got["weights"] - weights) <= rel * weights + small).all()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 32, 4), (3, 5, 5), (63, 16, 2), (64, 33, 16), (65, 64, 6), (200, 100, 7), (1000, 24, 3),
                                   (130, 128, 8), (129, 256, 3), (70, 257, 16), (67, 1000, 9), (300, 1024, 1), (2050, 2, 1)])
def test_route(T, E, k, bf16):
    rng = np.random.default_rng(T * 1031 + E * 7 + k)
    x = (2 * rng.standard_normal((T, E))).astype(np.float32)
    if bf16:
        x = ref.bf16_to_f64(ref.f64_to_bf16(x)).astype(np.float32)
    say("case route", T, E, k, bf16)
    for renorm in (True, False):
        check_route(x.astype(np.float64), k, renorm, run_route(x, k, renorm, bf16, ldl=E + 3))


@pytest.mark.parametrize("T", [65, 80, 4096, 4097])
@pytest.mark.parametrize("E,k", [(7, 3), (40, 8), (100, 5), (200, 1), (384, 8), (700, 16)])
def test_route_units_and_expert_counts(T, E, k):
    x = np.random.default_rng(T * 7 + E).standard_normal((T, E)).astype(np.float32)
    say("case route", T, E, k)
    check_route(x.astype(np.float64), k, True, run_route(x, k, True, False))


def test_route_more_than_one_unit_a_workgroup():
    T, E, k = 64 * 256 + 100, 8, 2
    x = np.random.default_rng(5).standard_normal((T, E)).astype(np.float32)
    say("case route", T, E, k)
    check_route(x.astype(np.float64), k, True, run_route(x, k, True, False))


@pytest.mark.parametrize("T,E,k", [(50, 12, 4), (400, 40, 5), (90, 300, 12)])
def test_route_masks_ties_and_specials(T, E, k):
    rng = np.random.default_rng(T)
    x = rng.integers(-2, 3, (T, E)).astype(np.float32) / 2  # many equal logits
    x[rng.random((T, E)) < 0.1] = -0.0
    x[rng.random((T, E)) < 0.4] = -np.inf
    x[rng.random((T, E)) < 0.05] = np.nan
    x[rng.random((T, E)) < 0.02] = np.inf
    x[rng.random((T, E)) < 0.02] = np.finfo(np.float32).min  # a mask's lowest value: chosen after all others
    x[rng.random(T) < 0.2] = -np.inf
    x[0], x[1] = np.nan, np.finfo(np.float32).min
    x[2], x[2, E // 2] = -np.inf, 1.0  # one expert left
    say("case route specials", T, E, k)
    for renorm in (True, False):
        got = run_route(x, k, renorm, False)
        with np.errstate(invalid="ignore"):
            check_route(x.astype(np.float64), k, renorm, got)
        assert (got["ids"][0] == -1).all() and (got["weights"][0] == 0).all()


# ---- product grouped by expert ------------------------------------------------

def split_rows(rng, rows, E, kind):
    """offsets [E + 1] that end at or before rows."""
    if kind == "even":
        cut = np.linspace(0, rows, E + 1).astype(int)
    elif kind == "one":  # all rows with one expert in the middle
        cut = np.where(np.arange(E + 1) <= E // 2, 0, rows)
    elif kind == "none":
        cut = np.zeros(E + 1, int)
    else:  # ragged, some experts empty, rows left over at the end
        w = rng.random(E) ** 4 * (rng.random(E) < 0.7) + 1e-9
        cut = np.concatenate([[0], np.floor(np.cumsum(w) / w.sum() * (rows - rows // 8))]).astype(int)
    return cut.astype(np.int32)


TILES = 5  # the grouped product's tiles (indices of MXGEMM_GROUPED_TILE; -1: streaming)


def run_grouped(rng, rows, E, N, K, fp8, kind="ragged", gather=0, alpha=1.0, pads=(0, 0, 0, 0, 0), e=(118, 132),
                bad_rows=False, nan_first=False, cols=None, odd_scales=False, what="", special_scales=False):
    """pads: of ldd, lda, ldsa, ldb, ldsb (elements or bytes)."""
    a_count = gather if gather else rows
    bits = 8 if fp8 else 4
    seed = int(rng.integers(1 << 30))
    lda, ldb = K + pads[1], K + pads[3]
    KB = K // 32
    A = np.full((a_count, lda * bits // 8), 0x77 if not fp8 else 0x7E, np.uint8)
    A[:, :K * bits // 8] = inputs.wide_codes(seed, a_count, K, 1) if fp8 else inputs.fp4_codes_packed(seed, a_count, K)
    SA = np.full((a_count, KB + pads[2]), 0xFF, np.uint8)  # NaN behind every scale row
    SA[:, :KB] = inputs.e8m0_scales(seed + 1, a_count, K, *e)
    B = np.full((E, N, ldb // 2), 0x77, np.uint8)
    B[:, :, :K // 2] = inputs.fp4_codes_packed(seed + 2, E * N, K).reshape(E, N, K // 2)
    SB = np.full((E, N, KB + pads[4]), 0xFF, np.uint8)
    SB[:, :, :KB] = inputs.e8m0_scales(seed + 3, E * N, K, *e).reshape(E, N, KB)
    if special_scales:
        SA[rng.integers(0, a_count, 2), rng.integers(0, KB)] = 0xFF
        SB[rng.integers(0, E), rng.integers(0, N, 2), rng.integers(0, KB)] = 0xFF
    if nan_first:
        SA[0] = 0xFF
    off = split_rows(rng, rows, E, kind)
    a_rows = rng.integers(0, a_count, rows).astype(np.int32) if gather else None
    if bad_rows:
        a_rows[rng.integers(0, rows, max(1, rows // 10))] = -1
        a_rows[rng.integers(0, rows, max(1, rows // 10))] = a_count + 3
    ldd = N + pads[0]
    D = torch.full((rows, ldd), 123.0, dtype=torch.bfloat16, device="cuda")
    A_, SA_, B_, SB_ = dev_u8(A), dev_u8(SA), dev_u8(B), dev_u8(SB)
    if odd_scales:  # scale matrices at odd addresses
        shift = lambda t: torch.cat((t.new_zeros(1), t.reshape(-1)))[1:]  # noqa: E731
        SA_, SB_ = shift(SA_), shift(SB_)
    say("case grouped", what, rows, E, N, K, "fp8" if fp8 else "fp4", kind, gather, off[-1])
    mx.mxgemm_grouped_run(D, A_, B_, SA_, SB_, dev(off), rows, N, K, E, a_rows=dev(a_rows) if gather else None,
                          a_count=a_count, alpha=alpha, a_format=1 if fp8 else 0, ldd=ldd, lda=lda, ldsa=SA.shape[1], ldb=ldb,
                          ldsb=SB.shape[2])
    torch.cuda.synchronize()
    d = host_bits(D)
    cols = np.arange(N) if cols is None else cols
    r, m, written = ref.grouped(A[:, :K * bits // 8], SA[:, :KB], B[:, :, :K // 2], SB[:, :, :KB], K, off, a_rows, rows, fp8,
                                alpha, cols)
    ref.check_grouped(d[written][:, cols], r[written], m[written], K, fp8, "grouped " + what)
    left = ref.f64_to_bf16(123.0)
    assert (d[~written] == left).all() and (d[:, N:] == left).all(), "rows or columns without an expert were written"


SHAPES = [  # rows, E, N, K
    (1, 1, 1, 32), (3, 2, 16, 64), (5, 8, 40, 96), (16, 4, 64, 512), (33, 3, 100, 416), (70, 5, 130, 1024), (128, 32, 48, 544),
    (64, 70, 33, 128), (300, 6, 272, 320), (520, 2, 300, 288), (700, 3, 520, 768), (40, 150, 24, 64),
]


@pytest.mark.parametrize("fp8", [False, True], ids=["fp4", "fp8"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%dx%dx%dx%d" % s)
def test_grouped(shape, fp8):
    rows, E, N, K = shape
    rng = np.random.default_rng(rows * 17 + K + fp8)
    run_grouped(rng, rows, E, N, K, fp8)
    run_grouped(rng, rows, E, N, K, fp8, gather=max(1, rows // 3), alpha=-0.75)


@pytest.mark.parametrize("fp8", [False, True], ids=["fp4", "fp8"])
@pytest.mark.parametrize("kind", ["even", "one", "none"])
def test_grouped_splits(kind, fp8):
    rng = np.random.default_rng(77 + fp8)
    run_grouped(rng, 200, 9, 136, 512, fp8, kind, gather=50)
    run_grouped(rng, 1100, 4, 264, 512, fp8, kind)
    run_grouped(rng, 6, 40, 80, 2048, fp8, kind, gather=2)


@pytest.mark.parametrize("fp8", [False, True], ids=["fp4", "fp8"])
@pytest.mark.parametrize("rows", [20, 90, 600])
def test_grouped_strides_and_bad_rows(rows, fp8):
    rng = np.random.default_rng(rows + fp8)
    for K, pads in ((512, (5, 64, 3, 32, 7)), (480, (8, 32, 0, 96, 16)), (1024, (0, 32, 16, 64, 16))):
        run_grouped(rng, rows, 3, 150, K, fp8, gather=rows // 2, pads=pads, bad_rows=True)
        run_grouped(rng, rows, 3, 150, K, fp8, pads=pads)
    run_grouped(rng, rows, 3, 264, 512, fp8, gather=7, odd_scales=True)


@pytest.mark.parametrize("fp8", [False, True], ids=["fp4", "fp8"])
@pytest.mark.parametrize("K", [512, 544])
@pytest.mark.parametrize("tile", range(-1, TILES))
def test_grouped_rows_that_are_not_there_are_zeros_beside_a_nan_row(tile, K, fp8, monkeypatch):
    monkeypatch.setenv("MXGEMM_GROUPED_TILE", str(tile))
    run_grouped(np.random.default_rng(K + tile), 150, 3, 144, K, fp8, gather=40, bad_rows=True, nan_first=True, what="nan first")


@pytest.mark.parametrize("fp8", [False, True], ids=["fp4", "fp8"])
@pytest.mark.parametrize("kind", ["ragged", "one"])
def test_grouped_many_rows_of_a_short_k(kind, fp8):
    run_grouped(np.random.default_rng(5), 700, 4, 80, 96, fp8, kind=kind, gather=300, what="short K")


@pytest.mark.parametrize("fp8", [False, True], ids=["fp4", "fp8"])
@pytest.mark.parametrize("K", [32, 96, 128, 224, 256])
@pytest.mark.parametrize("tile", range(-1, TILES))
def test_grouped_short_k_of_every_kernel(tile, K, fp8, monkeypatch):
    monkeypatch.setenv("MXGEMM_GROUPED_TILE", str(tile))
    run_grouped(np.random.default_rng(K), 300, 3, 136, K, fp8, gather=40, bad_rows=True, nan_first=True, what="short K")
    run_grouped(np.random.default_rng(K), 33, 2, 70, K, fp8, pads=(1, 32, 3, 32, 5), what="short K")


@pytest.mark.parametrize("fp8", [False, True], ids=["fp4", "fp8"])
@pytest.mark.parametrize("rows", [9, 400])
def test_grouped_special_scales(rows, fp8):
    rng = np.random.default_rng(rows)
    run_grouped(rng, rows, 2, 96, 512, fp8, "even", special_scales=True)


@pytest.mark.parametrize("rows,E,N,K,fp8", [(4, 32, 4096, 2048, False), (128, 32, 4096, 2048, True), (2036, 64, 1440, 2880, True),
                                            (8192, 8, 2048, 2048, False), (4096, 4, 1000, 4096, True)])
def test_grouped_large(rows, E, N, K, fp8):
    rng = np.random.default_rng(rows)
    run_grouped(rng, rows, E, N, K, fp8, gather=max(1, rows // 4), cols=np.unique(rng.integers(0, N, 24)), e=(122, 130))


@pytest.mark.parametrize("fp8", [False, True], ids=["fp4", "fp8"])
@pytest.mark.parametrize("tile", range(-1, TILES))
def test_grouped_every_kernel(tile, fp8, monkeypatch):
    """Each kernel on sizes the plan would give to others: K of 8 blocks, odd block counts, whole pairs of stages; experts
    without rows, with one and with many; few and many experts."""
    monkeypatch.setenv("MXGEMM_GROUPED_TILE", str(tile))
    rng = np.random.default_rng(50 + tile)
    for rows, E, N, K, gather in ((7, 3, 40, 256, 0), (300, 5, 264, 288, 90), (333, 4, 130, 512, 0), (290, 70, 72, 480, 33),
                                  (257, 2, 512, 1056, 300), (400, 130, 48, 1024, 17)):
        run_grouped(rng, rows, E, N, K, fp8, gather=gather, what="tile %d" % tile)
    run_grouped(rng, 100, 3, 96, 544, fp8, gather=9, pads=(3, 32, 5, 96, 1), bad_rows=True, odd_scales=True)


@pytest.mark.parametrize("K", [512, 800, 1056, 2048])
def test_grouped_persistent_equals_plain(K, monkeypatch):
    """The persistent 8-bit tile (more tiles than compute units) against the plain grid, bit for bit, and the oracle: even and
    odd stage counts, partial tiles, experts without rows, more experts than its table holds."""
    monkeypatch.setenv("MXGEMM_GROUPED_TILE", "1")
    for rows, E, N, gather in ((8300, 7, 1096, 700), (5000, 40, 2048, 0), (6000, 1100, 264, 100)):
        rng = np.random.default_rng(K + rows)
        off = dev(split_rows(rng, rows, E, "ragged"))
        a = gather or rows
        A = dev_u8(inputs.wide_codes(1, a, K, 1))
        SA, SB = dev_u8(inputs.e8m0_scales(2, a, K, 122, 130)), dev_u8(inputs.e8m0_scales(3, E * N, K, 122, 130))
        B = dev_u8(inputs.fp4_codes_packed(4, E * N, K))
        a_rows = dev(rng.integers(0, a, rows).astype(np.int32)) if gather else None
        got = []
        for persist in "01":
            monkeypatch.setenv("MXGEMM_TILE_PERSIST", persist)
            D = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
            say("case grouped persistent", K, rows, E, N, persist)
            mx.mxgemm_grouped_run(D, A, B, SA, SB, off, rows, N, K, E, a_rows=a_rows, a_count=a, a_format=1)
            got.append(host_bits(D))
        assert np.array_equal(got[0], got[1])
        cols = np.unique(rng.integers(0, N, 9))
        shape = lambda t: t.cpu().numpy().reshape(E, N, -1)  # noqa: E731
        r, m, w = ref.grouped(A.cpu().numpy(), SA.cpu().numpy(), shape(B), shape(SB), K, off.cpu().numpy(),
                              a_rows.cpu().numpy() if gather else None, rows, True, cols=cols)
        ref.check_grouped(got[0][w][:, cols], r[w], m[w], K, True, "persistent")
        assert (got[0][~w] == ref.f64_to_bf16(7.0)).all()


@pytest.mark.parametrize("fp8", [False, True], ids=["fp4", "fp8"])
@pytest.mark.parametrize("K", [288, 320, 416, 480])
def test_grouped_codes_behind_k_add_nothing(K, fp8):
    """Rows padded with the largest codes and scales of 2^127 behind K: over zeros the product is exactly zero."""
    rows, N, pad = 80, 200, 128
    A = torch.full((rows, (K + pad) * (8 if fp8 else 4) // 8), 0x7E if fp8 else 0x77, dtype=torch.uint8, device="cuda")
    A[:, :K * (8 if fp8 else 4) // 8] = 0
    B = torch.full((1, N, (K + pad) // 2), 0x77, dtype=torch.uint8, device="cuda")
    B[:, :, :K // 2] = 0
    S = torch.full((rows, 24), 0xFE, dtype=torch.uint8, device="cuda")
    SB = torch.full((1, N, 24), 0xFE, dtype=torch.uint8, device="cuda")
    D = torch.full((rows, N), 3.0, dtype=torch.bfloat16, device="cuda")
    say("case grouped codes behind K", K, fp8)
    mx.mxgemm_grouped_run(D, A, B, S, SB, dev(np.array([0, rows], np.int32)), rows, N, K, 1, a_format=int(fp8), lda=K + pad,
                          ldb=K + pad, ldsa=24, ldsb=24)
    assert int(torch.count_nonzero(D)) == 0


@pytest.mark.parametrize("tile", [-1, 0, 3])
def test_grouped_offsets_beyond_32_bits(tile, monkeypatch):
    """A and D with rows 2^17 bytes and more apart, experts' B 5 GB apart: rows near the end and the second expert."""
    monkeypatch.setenv("MXGEMM_GROUPED_TILE", str(tile))
    rows, N, K, E, lda, ldd = 40000, 24, 256, 2, 1 << 18, 1 << 16
    rng = np.random.default_rng(4)
    a, sa = inputs.fp4_codes_packed(1, rows, K), inputs.e8m0_scales(2, rows, K, 120, 130)
    b, sb = inputs.fp4_codes_packed(3, E * N, K).reshape(E, N, -1), inputs.e8m0_scales(4, E * N, K, 120, 130).reshape(E, N, -1)
    A = torch.zeros(rows, lda // 2, dtype=torch.uint8, device="cuda")
    A[:, :K // 2] = dev_u8(a)
    apart = 5 << 30
    B = torch.zeros(apart + N * K // 2, dtype=torch.uint8, device="cuda")
    for e in range(E):
        B[e * apart:e * apart + N * K // 2] = dev_u8(b[e]).reshape(-1)
    D = torch.zeros(rows, ldd, dtype=torch.bfloat16, device="cuda")
    off = np.array([0, 20, rows] if tile < 0 else [0, rows - 70, rows], np.int32)
    if tile < 0:
        off[2] = 90
    say("case grouped 64-bit offsets", tile)
    mx.mxgemm_grouped_run(D, A, B, dev_u8(sa), dev_u8(sb), dev(off), rows, N, K, E, lda=lda, ldd=ldd, strideb=2 * apart)
    look = np.unique(np.concatenate([np.arange(90), rng.integers(0, off[2], 60), np.arange(off[2] - 60, off[2])]))
    look = look[look < off[2]]
    d = host_bits(D[torch.from_numpy(look).cuda(), :N])
    r, m, _ = ref.grouped(a, sa, b, sb, K, off, None, rows, False)
    ref.check_grouped(d, r[look], m[look], K, False)


@pytest.mark.parametrize("tile", range(-1, TILES))
def test_grouped_offsets_that_do_not_ascend_stay_inside(tile, monkeypatch):
    """What D holds is then not said; what is around D, and rows outside every range, stay as they were."""
    monkeypatch.setenv("MXGEMM_GROUPED_TILE", str(tile))
    rows, N, K = 90, 72, 512
    for off in ([0, 80, 10, 60], [85, 3, 3, 2], [0, 2 ** 31 - 1, -2 ** 31, 50], [40, 40, 40, 40]):
        whole = torch.full((rows + 64, N + 16), 11.0, dtype=torch.bfloat16, device="cuda")
        D = whole[32:32 + rows, 8:]
        say("case grouped offsets", tile, off)
        mx.mxgemm_grouped_run(D, dev_u8(inputs.fp4_codes_packed(1, rows, K)), dev_u8(inputs.fp4_codes_packed(2, 3 * N, K)),
                              dev_u8(inputs.e8m0_scales(3, rows, K, 120, 130)), dev_u8(inputs.e8m0_scales(4, 3 * N, K, 120, 130)),
                              dev(np.array(off, np.int32)), rows, N, K, 3, ldd=N + 16)
        torch.cuda.synchronize()
        assert (whole[:32] == 11).all() and (whole[32 + rows:] == 11).all()
        assert (whole[:, :8] == 11).all() and (whole[:, 8 + N:] == 11).all()


def test_grouped_one_weight_for_all_and_clamped_offsets():
    """strideb = 0 shares one B; offsets outside [0, rows] are clamped."""
    rng = np.random.default_rng(3)
    rows, N, K, E = 50, 64, 256, 3
    A, SA = inputs.fp4_codes_packed(1, rows, K), inputs.e8m0_scales(2, rows, K, 120, 130)
    B, SB = inputs.fp4_codes_packed(3, N, K), inputs.e8m0_scales(4, N, K, 120, 130)
    off = np.array([-5, 20, 20, 1000], np.int32)
    D = torch.full((rows, N), 5.0, dtype=torch.bfloat16, device="cuda")
    say("case grouped one weight")
    mx.mxgemm_grouped_run(D, dev_u8(A), dev_u8(B), dev_u8(SA), dev_u8(SB), dev(off), rows, N, K, E, strideb=0, strideb_scale=0)
    torch.cuda.synchronize()
    r, m, _ = ref.grouped(A, SA, np.stack([B] * E), np.stack([SB] * E), K, [0, 20, 20, rows], None, rows, False)
    ref.check_grouped(host_bits(D), r, m, K, False)


def test_fp8_products_are_kept_to_13_bits_below_the_largest():
    """What the tolerance for 8-bit A rests on: in a group of 8 products, a term 2^-13 of the largest survives its
    cancellation and one of 2^-14 does not; outside the group it does."""
    K = 128
    A = torch.zeros(16, K, device="cuda")
    A[:, 0], A[:, 1] = 256.0, -256.0
    for j in range(4, 16):
        A[j, 7 if j % 2 else 6] = 2.0 ** (8 - j)
    A[0, 8], A[1, 40] = 2.0 ** -6, 2.0 ** -6  # another group
    one = lambda *s: torch.full(s, 127, dtype=torch.uint8, device="cuda")  # noqa: E731
    B = torch.full((1, 16, K // 2), 0x22, dtype=torch.uint8, device="cuda")
    D = torch.zeros(16, 16, dtype=torch.bfloat16, device="cuda")
    say("case fp8 alignment")
    mx.mxgemm_grouped_run(D, A.to(torch.float8_e4m3fn).view(torch.uint8), B, one(16, 4), one(1, 16, 4),
                          dev(np.array([0, 16], np.int32)), 16, 16, K, 1, a_format=1)
    d = D[:, 0].float().cpu().numpy()
    assert d[0] == d[1] == 2.0 ** -6
    assert [d[j] for j in range(4, 16)] == [2.0 ** (8 - j) if j <= 13 else 0.0 for j in range(4, 16)]


# ---- gated activation and quantizer ---------------------------------------------

def run_glu(bits, K, fp8, live=None, pads=(0, 0, 0), fill=0xA5):
    M = bits.shape[0]
    ldx, lda, ldsa = 2 * K + pads[0], K + pads[1], K // 32 + pads[2]
    X = np.full((M, ldx), 0x7FC0, np.uint16)
    X[:, :2 * K] = bits
    A = torch.full((M, lda * (8 if fp8 else 4) // 8), fill, dtype=torch.uint8, device="cuda")
    S = torch.full((M, ldsa), fill, dtype=torch.uint8, device="cuda")
    mx.mxgemm_glu_quantize(A, S, dev_bf16(X), M, K, live=None if live is None else dev(np.array([live], np.int32)), ldx=ldx,
                           lda=lda, ldsa=ldsa, a_format=1 if fp8 else 0)
    torch.cuda.synchronize()
    A, S = A.cpu().numpy(), S.cpu().numpy()
    n = M if live is None else min(max(live, 0), M)
    w = K if fp8 else K // 2
    assert (A[n:] == fill).all() and (S[n:] == fill).all() and (A[:, w:] == fill).all() and (S[:, K // 32:] == fill).all()
    if n:
        a, s = ref.quantize(ref.glu(bits[:n], K), fp8)
        assert np.array_equal(S[:n, :K // 32], s), "%d scales differ" % (S[:n, :K // 32] != s).sum()
        assert np.array_equal(A[:n, :w], a), "%d code bytes differ" % (A[:n, :w] != a).sum()


@pytest.mark.parametrize("fp8", [False, True], ids=["fp4", "fp8"])
@pytest.mark.parametrize("M,K", [(1, 32), (3, 96), (4, 2048), (37, 416), (130, 1024), (1, 16384)])
def test_glu(M, K, fp8):
    rng = np.random.default_rng(M + K)
    say("case glu", M, K, fp8)
    run_glu(bf16_bits(rng, M, 2 * K), K, fp8)
    run_glu(bf16_bits(rng, M, 2 * K, sigma=6.0), K, fp8, live=M // 2, pads=(8, 32, 3))


@pytest.mark.parametrize("fp8", [False, True], ids=["fp4", "fp8"])
def test_glu_all_gates_and_specials(fp8):
    """Every bf16 gate (infinities and NaN among them) against up values over the whole range, and rows of zeros."""
    rng = np.random.default_rng(8)
    gates = np.arange(65536, dtype=np.uint16)
    for up in (bf16_bits(rng, 65536), rng.integers(0, 65536, 65536).astype(np.uint16), np.full(65536, 0x3F80, np.uint16),
               np.zeros(65536, np.uint16)):
        # a special value spoils its block: gates in order keep them together
        bits = np.concatenate([gates.reshape(64, 1024), up.reshape(64, 1024)], 1)
        say("case glu all gates", fp8)
        run_glu(bits, 1024, fp8)


def test_glu_and_norm_rows_far_apart():
    """Row strides of 2 GB and more."""
    rng = np.random.default_rng(21)
    K, T, ld = 96, 4, 3 << 29
    X = torch.zeros(T * ld, dtype=torch.bfloat16, device="cuda")
    rows = X.as_strided((T, 2 * K), (ld, 1))
    bits = bf16_bits(rng, T, 2 * K)
    rows.copy_(dev_bf16(bits))
    A, S = torch.zeros(T, K, dtype=torch.uint8, device="cuda"), torch.zeros(T, K // 32, dtype=torch.uint8, device="cuda")
    say("case glu far rows")
    mx.mxgemm_glu_quantize(A, S, X, T, K, ldx=ld, a_format=1)
    a, s = ref.quantize(ref.glu(bits, K), True)
    assert np.array_equal(A.cpu().numpy(), a) and np.array_equal(S.cpu().numpy(), s)
    H = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    w = bf16_bits(rng, K)
    say("case norm far rows")
    mx.mxgemm_norm_quantize(T, K, X, X=X[K:], H=H, w_post=dev_bf16(w), ldy=ld, ldx=ld, res_scale=0.5)
    h, _ = ref.norm(bits[:, :K], K, X=bits[:, K:], w_post=w, res_scale=0.5)
    assert np.array_equal(host_bits(H), h)


@pytest.mark.parametrize("live", [-3, 0, 5, 99])
def test_glu_live_rows_are_clamped(live):
    rng = np.random.default_rng(9)
    say("case glu live", live)
    run_glu(bf16_bits(rng, 11, 128), 64, True, live=live)


# ---- norms ------------------------------------------------------------------------

def run_norm(rng, T, K, fp8, top_k=0, post=True, gate=None, x=True, pre=True, h=True, z=True, q=True, pad=0, scale=0.75,
             sigma=1.0, missing=0.2, alias=False, y=None, nan_first=False):
    y_rows = T * max(top_k, 1) + (3 if top_k else 0)
    Y = bf16_bits(rng, y_rows, K, sigma=sigma) if y is None else y
    kw, dk = {}, {}

    def strided(bits):
        p = np.full((bits.shape[0], K + pad), 0x7FC0, np.uint16)
        p[:, :K] = bits
        return dev_bf16(p)
    if top_k and nan_first:
        Y[0] = 0x7FC0  # (no token's row)
    if top_k:
        pos = rng.permutation(y_rows)[:T * top_k].reshape(T, top_k).astype(np.int32)
        pos[rng.random((T, top_k)) < missing] = -1
        pos[rng.random((T, top_k)) < missing / 4] = y_rows + 2
        if T > 1:
            pos[1] = -1  # a token that no expert took
        weights = rng.random((T, top_k)).astype(np.float32)
        if nan_first:
            pos[pos == 0] = -1
            weights[(pos < 0) | (pos >= y_rows)] = np.nan
        kw.update(pos=pos, weights=weights)
        dk.update(pos=dev(pos), weights=dev(weights), top_k=top_k, y_rows=y_rows)
    if post:
        kw["w_post"] = bf16_bits(rng, K)
        dk["w_post"] = dev_bf16(kw["w_post"])
    if gate:
        kw["gate"] = bf16_bits(rng, T if gate == "rows" else 1, K)
        dk["gate"] = strided(kw["gate"])
    if x:
        kw["X"] = bf16_bits(rng, T, K, sigma=2.0)
        dk["X"] = strided(kw["X"])
    if pre:
        kw["w_pre"] = bf16_bits(rng, K)
        dk["w_pre"] = dev_bf16(kw["w_pre"])
    full = lambda: torch.full((T, K + pad), 9.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    Yd = strided(Y)
    H = (dk["X"] if alias and x else full()) if h else None
    Z = (Yd if alias and not top_k else full()) if z else None
    lda, ldsa = K + 32 * (pad > 0), K // 32 + (pad > 0)
    A = torch.full((T, lda * (8 if fp8 else 4) // 8), 0xA5, dtype=torch.uint8, device="cuda") if q else None
    S = torch.full((T, ldsa), 0xA5, dtype=torch.uint8, device="cuda") if q else None
    say("case norm", T, K, fp8, top_k, post, gate, x, pre, h, z, q, pad)
    mx.mxgemm_norm_quantize(T, K, Yd, H=H, Z=Z, A=A, scaleA=S, res_scale=scale, a_format=1 if fp8 else 0, ldy=K + pad,
                            ldg=0 if gate == "one" else K + pad, ldx=K + pad, ldh=K + pad, ldz=K + pad, lda=lda, ldsa=ldsa, **dk)
    torch.cuda.synchronize()
    hr, zr = ref.norm(Y, K, res_scale=scale, T=T, **kw)
    same = lambda a, b: np.array_equal(np.where(np.isnan(ref.bf16_to_f64(a)), 0x7FC0, a),  # noqa: E731
                                       np.where(np.isnan(ref.bf16_to_f64(b)), 0x7FC0, b))
    if h:
        got = host_bits(H)
        assert same(got[:, :K], hr), "%d of h differ" % (got[:, :K] != hr).sum()
        assert alias or (got[:, K:] == ref.f64_to_bf16(9.0)).all()
    if z:
        got = host_bits(Z)
        assert same(got[:, :K], zr), "%d of z differ" % (got[:, :K] != zr).sum()
    if q:
        w = K if fp8 else K // 2
        a, s = ref.quantize(zr, fp8)
        A, S = A.cpu().numpy(), S.cpu().numpy()
        assert np.array_equal(S[:, :K // 32], s) and np.array_equal(A[:, :w], a)
        assert (A[:, w:] == 0xA5).all() and (S[:, K // 32:] == 0xA5).all()


@pytest.mark.parametrize("fp8", [False, True], ids=["fp4", "fp8"])
@pytest.mark.parametrize("T,K", [(1, 32), (5, 96), (3, 512), (7, 544), (2, 2048), (4, 2080), (3, 4096), (2, 4128), (3, 8192),
                                 (2, 8224), (2, 16384)])
def test_norm(T, K, fp8):
    rng = np.random.default_rng(T * 31 + K)
    run_norm(rng, T, K, fp8, top_k=4)
    run_norm(rng, T, K, fp8, top_k=0, gate="rows", pad=8)


@pytest.mark.parametrize("K", [512, 2048, 2080, 4096, 4160, 8192, 8224])
def test_norm_of_more_tokens_than_compute_units(K):
    rng = np.random.default_rng(K)
    run_norm(rng, 300, K, True, top_k=2)
    run_norm(rng, 300, K, False, gate="rows")


@pytest.mark.parametrize("opts", [dict(post=False), dict(pre=False), dict(x=False, gate="one"), dict(h=False, z=False),
                                  dict(z=False, q=False), dict(post=False, pre=False, x=False), dict(top_k=1, gate="one", pad=16),
                                  dict(top_k=8, post=False, missing=0.6), dict(alias=True), dict(alias=True, top_k=2),
                                  dict(scale=-1.5, sigma=2.0 ** -60), dict(scale=0.0)], ids=lambda o: "-".join(map(str, o)))
def test_norm_options(opts):
    rng = np.random.default_rng(11)
    for T, K in ((9, 320), (3, 4096)):
        run_norm(rng, T, K, True, **opts)
        run_norm(rng, T, K, False, **opts)


def test_norm_absent_rows_add_nothing_whatever_stands_there():
    rng = np.random.default_rng(13)
    for T, K, k in ((5, 320, 3), (3, 4096, 4), (300, 2080, 5)):
        run_norm(rng, T, K, True, top_k=k, nan_first=True)


def test_norm_zeros_and_specials():
    rng = np.random.default_rng(12)
    y = bf16_bits(rng, 6, 256)
    y[0], y[1, 7], y[2, 9] = 0, 0x7F80, 0x7FC0  # zeros; an infinity; a NaN: their tokens alone are affected
    run_norm(rng, 6, 256, True, y=y)
    run_norm(rng, 6, 256, False, y=y, x=False)
    run_norm(rng, 6, 256, False, y=y, post=False)


# ---- the block as it is used ----------------------------------------------------

class Block:
    """Router choice, gate/up product, activation, down product, norms, as a user's program holds them."""

    def __init__(self, T, E, k, hidden, inner, seed, fp8):
        g = np.random.default_rng(seed)
        self.T, self.E, self.k, self.hidden, self.inner, self.fmt = T, E, k, hidden, inner, 1 if fp8 else 0
        self.fp8 = fp8
        w = 1 if fp8 else 2
        u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
        bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        codes = lambda r, K: inputs.fp4_codes_packed(int(g.integers(1 << 30)), r, K)  # noqa: E731
        scales = lambda r, K: inputs.e8m0_scales(int(g.integers(1 << 30)), r, K, 117, 121)  # noqa: E731
        self.B1n, self.SB1n = codes(E * 2 * inner, hidden), scales(E * 2 * inner, hidden)
        self.B2n, self.SB2n = codes(E * hidden, inner), scales(E * hidden, inner)
        self.B1, self.SB1, self.B2, self.SB2 = dev_u8(self.B1n), dev_u8(self.SB1n), dev_u8(self.B2n), dev_u8(self.SB2n)
        self.w_post, self.w_pre = dev_bf16(bf16_bits(g, hidden)), dev_bf16(bf16_bits(g, hidden))
        self.logits, self.X = torch.zeros(T, E, device="cuda"), bf(T, hidden)
        self.XA, self.XS = u8(T, hidden // w), u8(T, hidden // 32)
        R = T * k
        self.ids, self.pos, self.offsets, self.rows = i32(T, k), i32(T, k), i32(E + 1), i32(R)
        self.weights = torch.zeros(T, k, device="cuda")
        n = mx.mxgemm_route_workspace_bytes(T, E)
        self.ws = u8(max(n, 4))
        self.D1, self.D2 = bf(R, 2 * inner), bf(R, hidden)
        self.IA, self.IS = u8(R, inner // w), u8(R, inner // 32)
        self.H, self.Z = bf(T, hidden), bf(T, hidden)
        self.A, self.S = u8(T, hidden // w), u8(T, hidden // 32)

    def feed(self, seed):
        g = np.random.default_rng(seed)
        x = g.standard_normal((self.T, self.E)).astype(np.float32)
        x[g.random(self.T) < 0.1] = -np.inf
        self.logits.copy_(dev(x))
        bits = bf16_bits(g, self.T, self.hidden)
        self.X.copy_(dev_bf16(bits))
        a, s = ref.quantize(bits, self.fp8)
        self.XA.copy_(dev_u8(a))
        self.XS.copy_(dev_u8(s))
        torch.cuda.synchronize()

    def run(self, stream=None):
        T, E, k, R = self.T, self.E, self.k, self.T * self.k
        mx.mxgemm_route(self.ids, self.weights, self.pos, self.offsets, self.rows, self.logits, T, E, k, workspace=self.ws,
                        workspace_bytes=self.ws.numel(), stream=stream)
        mx.mxgemm_grouped_run(self.D1, self.XA, self.B1, self.XS, self.SB1, self.offsets, R, 2 * self.inner, self.hidden, E,
                              a_rows=self.rows, a_count=T, a_format=self.fmt, stream=stream)
        mx.mxgemm_glu_quantize(self.IA, self.IS, self.D1, R, self.inner, live=self.offsets[E:], a_format=self.fmt, stream=stream)
        mx.mxgemm_grouped_run(self.D2, self.IA, self.B2, self.IS, self.SB2, self.offsets, R, self.hidden, self.inner, E,
                              a_format=self.fmt, stream=stream)
        mx.mxgemm_norm_quantize(T, self.hidden, self.D2, X=self.X, H=self.H, Z=self.Z, A=self.A, scaleA=self.S, pos=self.pos,
                                weights=self.weights, top_k=k, y_rows=R, w_post=self.w_post, w_pre=self.w_pre,
                                a_format=self.fmt, stream=stream)

    def outputs(self):
        torch.cuda.synchronize()
        n = int(self.offsets[-1])
        return [t.clone() for t in (self.ids, self.weights, self.pos, self.offsets, self.rows, self.D1[:n], self.IA[:n],
                                    self.IS[:n], self.D2[:n], self.H, self.Z, self.A, self.S)]

    def check(self):
        """Every step against the 64-bit implementation on the step's own inputs."""
        torch.cuda.synchronize()
        n = lambda t: t.cpu().numpy()  # noqa: E731
        x = n(self.logits).astype(np.float64)
        got = {a: n(getattr(self, a)) for a in ("ids", "weights", "pos", "offsets", "rows")}
        check_route(x, self.k, True, got)
        off, R = got["offsets"], self.T * self.k
        live = off[-1]
        E, inner, hidden = self.E, self.inner, self.hidden
        shape = lambda a, N: a.reshape(E, N, -1)  # noqa: E731
        r, m, w = ref.grouped(n(self.XA), n(self.XS), shape(self.B1n, 2 * inner), shape(self.SB1n, 2 * inner), hidden, off,
                              got["rows"], R, self.fp8)
        ref.check_grouped(host_bits(self.D1)[w], r[w], m[w], hidden, self.fp8, "gate and up")
        a, s = ref.quantize(ref.glu(host_bits(self.D1)[:live], inner), self.fp8)
        assert np.array_equal(n(self.IA)[:live], a) and np.array_equal(n(self.IS)[:live], s)
        r, m, w = ref.grouped(n(self.IA), n(self.IS), shape(self.B2n, hidden), shape(self.SB2n, hidden), inner, off, None, R,
                              self.fp8)
        ref.check_grouped(host_bits(self.D2)[w], r[w], m[w], inner, self.fp8, "down")
        h, z = ref.norm(host_bits(self.D2), hidden, X=host_bits(self.X), pos=got["pos"], weights=got["weights"],
                        w_post=host_bits(self.w_post), w_pre=host_bits(self.w_pre), T=self.T)
        assert np.array_equal(host_bits(self.H), h) and np.array_equal(host_bits(self.Z), z)
        a, s = ref.quantize(z, self.fp8)
        assert np.array_equal(n(self.A), a) and np.array_equal(n(self.S), s)


def equal(a, b):
    return all(x.shape == y.shape and torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("fp8", [False, True], ids=["fp4", "fp8"])
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (5, 16, 4), (150, 6, 3), (400, 4, 2)])
def test_block(T, E, k, fp8):
    b = Block(T, E, k, 256, 160, T, fp8)
    b.feed(1)
    say("case block", T, E, k, fp8)
    b.run()
    b.check()
    first = b.outputs()
    b.run()
    assert equal(first, b.outputs()), "a second run gives other bits"


def test_block_on_another_stream():
    b = Block(40, 8, 2, 256, 128, 3, True)
    b.feed(2)
    b.run()
    eager = b.outputs()
    s = torch.cuda.Stream()
    say("case block on another stream")
    b.feed(2)
    s.wait_stream(torch.cuda.current_stream())
    b.run(stream=s)
    s.synchronize()
    assert equal(eager, b.outputs())


def test_two_blocks_at_once():
    """Two blocks on two streams without an order between them, each as alone."""
    blocks = [Block(60, 8, 2, 256, 128, 3, False), Block(33, 16, 4, 256, 96, 6, True)]
    want = []
    for i, b in enumerate(blocks):
        b.feed(i)
        b.run()
        want.append(b.outputs())
    streams = [torch.cuda.Stream() for _ in blocks]
    say("case two blocks at once")
    for _ in range(5):
        for b, s in zip(blocks, streams):
            b.run(stream=s)
    torch.cuda.synchronize()
    for b, w in zip(blocks, want):
        assert equal(w, b.outputs())


def test_two_captured_blocks_replay():
    """Two blocks captured on their own, replayed in turn with new inputs, other work and synchronizations between: each
    replay equals the eager result."""
    blocks = [Block(70, 8, 2, 256, 128, 4, False), Block(9, 16, 4, 128, 96, 5, True)]
    graphs = []
    for b in blocks:
        b.feed(0)
        b.run()
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            b.run(stream=s)
        graphs.append(g)
    say("case captured blocks")
    for i in range(4):
        want = []
        for b in blocks:
            b.feed(10 + i)
            b.run()
            want.append(b.outputs())
        for b in blocks:
            for t in (b.D1, b.D2, b.H, b.Z, b.A, b.S, b.ids, b.weights, b.pos, b.rows, b.offsets):
                t.zero_()
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for b, w in zip(blocks, want):
            assert equal(w, b.outputs()), "replay %d" % i
