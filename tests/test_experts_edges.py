"""GPU tests of the mixture-of-experts operators at their edges: routings that
give one expert everything, weights of masked tokens against a bound that does
not grow with the mask, and the persistent product on bad rows and offsets."""
import numpy as np
import pytest

import block_scaled_precision_mxfp4_amd as mx
import experts_ref as ref
from block_scaled_precision_mxfp4_amd import inputs

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mxgpu import dev_u8  # noqa: E402
from test_experts import dev, run_grouped, run_route, say  # noqa: E402
from test_experts_host import special_logits  # noqa: E402


# ---- router choice ------------------------------------------------------------

def check_weights(x, k, renorm):
    got = run_route(x, k, renorm, False)
    x = x.astype(np.float64)
    with np.errstate(invalid="ignore"):
        ids, weights, pos, offsets, rows = ref.route(x, k, renorm)
    for name, want in (("ids", ids), ("pos", pos), ("offsets", offsets), ("rows", rows)):
        assert np.array_equal(got[name], want), name
    rel, small = ref.route_weight_bound(x, ids)
    off = np.abs(got["weights"] - weights) > rel * weights + small
    assert not off.any(), "%d weights outside, e.g. %r, not %r" % (off.sum(), got["weights"][off][0], weights[off][0])


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(50, 12, 4), (64, 200, 16), (400, 40, 5), (90, 300, 12), (70, 1024, 16), (5000, 24, 3)])
def test_route_weights_beside_masks(T, E, k, renorm):
    say("case route weights", T, E, k, renorm)
    check_weights(special_logits(np.random.default_rng(T), T, E), k, renorm)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(33, 64, 6), (700, 128, 8), (66, 512, 4)])
def test_route_weights_of_wide_logits(T, E, k, renorm):
    """Shares from 1 down to fp32's least value, with masked logits among them."""
    rng = np.random.default_rng(E)
    x = (25 * rng.standard_normal((T, E))).astype(np.float32)
    x[rng.random((T, E)) < 0.3] = -np.inf
    x[rng.random((T, E)) < 0.1] = np.finfo(np.float32).min
    say("case route wide", T, E, k, renorm)
    check_weights(x, k, renorm)


# ---- product grouped by expert: streaming ---------------------------------------

@pytest.mark.parametrize("fp8", [False, True], ids=["fp4", "fp8"])
@pytest.mark.parametrize("kind", ["one", "even", "ragged"])
@pytest.mark.parametrize("rows,E,N,K", [(1024, 64, 256, 512), (1000, 70, 40, 544), (33, 3, 100, 1056), (520, 130, 24, 96)])
def test_grouped_streamed_groups_of_rows(rows, E, N, K, kind, fp8, monkeypatch):
    monkeypatch.setenv("MXGEMM_GROUPED_TILE", "-1")
    run_grouped(np.random.default_rng(rows + K), rows, E, N, K, fp8, kind, gather=rows // 3, what="streamed")
    run_grouped(np.random.default_rng(rows + K), rows, E, N, K, fp8, kind, what="streamed")


@pytest.mark.parametrize("fp8", [False, True], ids=["fp4", "fp8"])
def test_grouped_one_expert_with_all_rows_is_not_serial(fp8, monkeypatch):
    """Rows that the plan streams because their experts' tiles would be few (64 experts, N = 256), all of one expert's: done
    one group of 16 after another they took 24 times the time of the smallest tile, side by side they take about as long."""
    rows, E, N, K = 1024, 64, 256, 2048
    w = 1 if fp8 else 2
    A, SA = torch.randint(0, 120, (rows, K // w), dtype=torch.uint8, device="cuda"), torch.full((rows, K // 32), 120, dtype=torch.uint8, device="cuda")
    B, SB = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda"), torch.full((E, N, K // 32), 120, dtype=torch.uint8, device="cuda")
    off = dev(np.where(np.arange(E + 1) <= E // 2, 0, rows).astype(np.int32))
    D = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")

    def us(tile):
        if tile is None:
            monkeypatch.delenv("MXGEMM_GROUPED_TILE", raising=False)
        else:
            monkeypatch.setenv("MXGEMM_GROUPED_TILE", str(tile))
        call = lambda: mx.mxgemm_grouped_run(D, A, B, SA, SB, off, rows, N, K, E, a_format=1 if fp8 else 0)  # noqa: E731
        call()
        torch.cuda.synchronize()
        best = []
        for _ in range(9):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(8):
                call()
            b.record()
            torch.cuda.synchronize()
            best.append(a.elapsed_time(b) * 125)
        return min(best)
    say("case grouped one expert", fp8)
    plan, tile = us(None), us(4)
    say("us: plan %.1f, smallest tile %.1f" % (plan, tile))
    assert plan < 5 * tile


# ---- product grouped by expert: the persistent 8-bit tile -------------------------

@pytest.mark.parametrize("K,pads", [(512, (8, 64, 16, 32, 16)), (512, (0, 32, 3, 0, 7)), (800, (16, 16, 5, 32, 1)), (2048, (8, 0, 0, 64, 0))],
                         ids=["whole-groups", "odd-scales", "odd-stages", "one-group-more"])
@pytest.mark.parametrize("rows,E,N,gather", [(8300, 7, 1096, 700), (6000, 1000, 264, 100)])
def test_grouped_persistent_rows_strides_and_alpha(rows, E, N, gather, K, pads, monkeypatch):
    """More tiles than compute units on the persistent form (8-bit A, D in 16-byte rows): row indexes that are not there beside a
    row 0 of NaN scales, padded strides, scale rows of any alignment, a factor."""
    monkeypatch.setenv("MXGEMM_GROUPED_TILE", "1")
    rng = np.random.default_rng(rows + K)
    cols = np.unique(np.concatenate([rng.integers(0, N, 7), [0, N - 1]]))
    run_grouped(rng, rows, E, N, K, True, gather=gather, alpha=-0.75, pads=pads, bad_rows=True, nan_first=True, cols=cols,
                odd_scales=pads[2] % 2 == 1, what="persistent")


@pytest.mark.parametrize("persist", ["0", "1"])
@pytest.mark.parametrize("tile", [-1, 1, 3, 4])
@pytest.mark.parametrize("rows,E,N,K", [(90, 6, 64, 512), (9000, 9, 1032, 544)])
def test_grouped_8_bit_offsets_that_do_not_ascend_stay_inside(rows, E, N, K, tile, persist, monkeypatch):
    """Whatever the offsets and the row list hold, nothing outside D's rows and columns is written, by any 8-bit kernel."""
    monkeypatch.setenv("MXGEMM_GROUPED_TILE", str(tile))
    monkeypatch.setenv("MXGEMM_TILE_PERSIST", persist)
    rng = np.random.default_rng(rows)
    wild = rng.integers(-2 ** 31, 2 ** 31, E + 1)
    back = np.linspace(rows, 0, E + 1).astype(int)
    over = np.where(np.arange(E + 1) % 2 == 0, 0, rows)
    for off in (wild, back, over, rng.integers(0, rows + 1, E + 1)):
        whole = torch.full((rows + 64, N + 16), 11.0, dtype=torch.bfloat16, device="cuda")
        D = whole[32:32 + rows, 8:]
        a_rows = np.where(rng.random(rows) < 0.2, rng.integers(-2 ** 31, 2 ** 31, rows), rng.integers(0, 50, rows)).astype(np.int32)
        say("case grouped offsets", tile, persist, rows, off)
        mx.mxgemm_grouped_run(D, dev_u8(inputs.wide_codes(1, 50, K, 1)), dev_u8(inputs.fp4_codes_packed(2, E * N, K)),
                              dev_u8(inputs.e8m0_scales(3, 50, K, 120, 130)), dev_u8(inputs.e8m0_scales(4, E * N, K, 120, 130)),
                              dev(off.astype(np.int32)), rows, N, K, E, a_rows=dev(a_rows), a_count=50, a_format=1, ldd=N + 16)
        torch.cuda.synchronize()
        assert (whole[:32] == 11).all() and (whole[32 + rows:] == 11).all()
        assert (whole[:, :8] == 11).all() and (whole[:, 8 + N:] == 11).all()


# ---- streams ----------------------------------------------------------------------

def test_calls_go_to_torchs_current_stream():
    """By default a call is on torch's current stream, also inside a stream context."""
    s = torch.cuda.Stream()
    assert mx._stream(None) == torch.cuda.current_stream().cuda_stream
    with torch.cuda.stream(s):
        assert mx._stream(None) == s.cuda_stream == mx._stream(s)
    assert mx._stream(None) == torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("persist", ["0", "1"])
@pytest.mark.parametrize("K", [96, 288, 544, 800])
@pytest.mark.parametrize("tile", [-1, 1, 3, 4])
def test_grouped_8_bit_nan_codes_behind_k_are_not_seen(tile, K, persist, monkeypatch):
    """Rows of A padded with NaN codes behind K, in sizes that end inside a step, a stage and a pair of stages; with more tiles
    than compute units too."""
    monkeypatch.setenv("MXGEMM_GROUPED_TILE", str(tile))
    monkeypatch.setenv("MXGEMM_TILE_PERSIST", persist)
    rng = np.random.default_rng(K)
    N, E, pad = 264, 3, 160
    for rows in (70, 17000):
        A = torch.full((rows, K + pad), 0x7F, dtype=torch.uint8, device="cuda")
        A[1::2, K:] = 0xFF
        A[:, :K] = 0x38  # 1
        B = torch.full((E, N, (K + pad) // 2), 0x77, dtype=torch.uint8, device="cuda")
        B[:, :, :K // 2] = 0x22  # 1, 1
        KB = K // 32
        S = torch.full((rows, KB + 5), 0xFF, dtype=torch.uint8, device="cuda")
        S[:, :KB] = 127
        SB = torch.full((E, N, KB + 5), 0xFF, dtype=torch.uint8, device="cuda")
        SB[:, :, :KB] = 127
        off = np.array([0, rows // 3, rows // 3, rows], np.int32)
        a_rows = dev(rng.integers(0, rows, rows).astype(np.int32))
        D = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
        say("case grouped NaN behind K", tile, K, persist, rows)
        mx.mxgemm_grouped_run(D, A, B, S, SB, dev(off), rows, N, K, E, a_rows=a_rows, a_count=rows, a_format=1, lda=K + pad,
                              ldb=K + pad, ldsa=KB + 5, ldsb=KB + 5)
        torch.cuda.synchronize()
        assert (D == K).all()
