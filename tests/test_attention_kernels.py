"""GPU tests of each kernel of the attention over a paged cache: all four are
made to run every batch, against the 64-bit plain implementation
(attention_ref.py)."""
import numpy as np
import pytest

import attention_ref as ref
import block_scaled_precision_mxfp4_amd as mx
from test_attention import CASES, Batch, attend, bf16, check, dev, run_append, say, workspace

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mxgpu import dev_bf16, host_bits  # noqa: E402

KERNELS = range(4)  # MXGEMM_ATTENTION_KERNEL: keys in turn over 32 or 64 rows, tiles of rows small and large

MORE = [  # new, lens, heads, kv_heads, D, page, fp8
    ([1, 1, 2], [1000, 333, 64], 4, 1, 64, 16, False),
    ([1, 1, 2], [1000, 333, 64], 4, 1, 128, 64, True),
    ([20, 3], [1500, 700], 8, 2, 128, 16, False),
    ([64], [2000], 4, 1, 128, 16, True),
    ([33, 64], [900, 64], 4, 1, 256, 16, False),
    ([260, 1, 130], [700, 900, 131], 2, 1, 64, 16, True),
    ([300, 20], [300, 900], 2, 1, 128, 32, False),
]


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("case", range(len(CASES) + len(MORE)))
def test_each_kernel(case, kernel, monkeypatch):
    new, lens, H, Hk, D, page, fp8 = (CASES + MORE)[case]
    monkeypatch.setenv("MXGEMM_ATTENTION_KERNEL", str(kernel))
    rng = np.random.default_rng(300 + case)
    b = Batch(rng, new, lens, Hk, D, page, fp8)
    q = bf16(rng, b.T, H * D, sigma=2.0)
    say("case kernel", case, kernel)
    w = workspace(b.T, b.S, H, Hk, D)
    got = attend(b, q, H, w=w)
    check(b, q, H, got)
    again = attend(b, q, H, w=w)
    assert np.array_equal(got[0], again[0]) and np.array_equal(got[1], again[1])


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 100, 500])
def test_windows(window, causal, kernel, monkeypatch):
    """Few keys of a long context: pieces of it that no row sees, and steps that end behind the last key."""
    monkeypatch.setenv("MXGEMM_ATTENTION_KERNEL", str(kernel))
    for fp8, D, new, lens in ((False, 64, [1, 3, 40], [1000, 333, 150]), (True, 128, [1, 90], [701, 600])):
        rng = np.random.default_rng(40)
        b = Batch(rng, new, lens, 1, D, 16, fp8)
        q = bf16(rng, b.T, 4 * D, sigma=2.0)
        say("case windows", window, causal, kernel, D)
        check(b, q, 4, attend(b, q, 4, causal=causal, window=window), causal=causal, window=window)


@pytest.mark.parametrize("max_new", [1, 7, 70, 10 ** 6])
def test_any_hint_of_the_most_new_tokens(max_new):
    rng = np.random.default_rng(41)
    b = Batch(rng, [1, 70, 2], [300, 200, 64], 2, 64, 16, False)
    q = bf16(rng, b.T, 8 * 64)
    check(b, q, 8, attend(b, q, 8, max_new=max_new))


@pytest.mark.parametrize("kernel", KERNELS)
def test_quantized_rows_of_each_kernel(kernel, monkeypatch):
    monkeypatch.setenv("MXGEMM_ATTENTION_KERNEL", str(kernel))
    import experts_ref
    for D, fp8 in ((64, False), (96, True), (128, False), (256, True)):
        rng = np.random.default_rng(42)
        b = Batch(rng, [1, 3, 70], [1500, 20, 700], 2, D, 16, False)
        H = 4
        q = bf16(rng, b.T, H * D)
        n = H * D if fp8 else H * D // 2
        A = torch.zeros((b.T, n), dtype=torch.uint8, device="cuda")
        S = torch.zeros((b.T, H * D // 32), dtype=torch.uint8, device="cuda")
        say("case quantized rows", D, kernel)
        O, _ = attend(b, q, H, A=A, scaleA=S, lda=H * D, ldsa=H * D // 32, a_format=mx.FMT_FP8_E4M3 if fp8 else mx.FMT_FP4)
        want = experts_ref.quantize(O.reshape(b.T, -1), fp8)
        assert np.array_equal(A.cpu().numpy(), want[0]) and np.array_equal(S.cpu().numpy(), want[1])


@pytest.mark.parametrize("kernel", KERNELS)
def test_cache_and_rows_of_more_than_32_bits(kernel, monkeypatch):
    """Pages, heads and rows of Q and O that stand more than 4 GiB apart: append, then attend."""
    monkeypatch.setenv("MXGEMM_ATTENTION_KERNEL", str(kernel))
    rng = np.random.default_rng(43)
    H, Hk, D = 4, 2, 64
    b = Batch(rng, [40, 1], [45, 70], Hk, D, 16, False)
    q, k, v = (bf16(rng, b.T, h * D) for h in (H, Hk, Hk))
    freq = mx.mxgemm_rope_frequencies(D)
    turned = run_append(b, q, k, v, H, freq, D, False)
    before = b.kc, b.vc
    b.kc, b.vc = b.pools()
    want = attend(b, turned, H)
    # the same with everything far apart
    page = 1 << 28  # elements
    head = b.num_pages * page
    far = torch.empty(4 * head, dtype=torch.int16, device="cuda")
    K, V = far[:far.numel() // 2], far[far.numel() // 2:]
    K, V = (x.as_strided((b.num_pages, Hk, 16, D), (page, head, D, 1)) for x in (K, V))
    K.copy_(dev(before[0].view(np.int16)))
    V.copy_(dev(before[1].view(np.int16)))
    ld = 1 << 26
    rows = torch.empty(b.T * ld, dtype=torch.bfloat16, device="cuda").as_strided((b.T, H * D), (ld, 1))
    rows.copy_(dev_bf16(q))
    cache = mx.make_kv_cache(K, V, *b.dev, seqs=b.S, num_pages=b.num_pages, page_size=16, max_pages=b.max_pages, kv_heads=Hk,
                             head_dim=D, page_stride=page, head_stride=head)
    say("case far", kernel)
    mx.mxgemm_kv_append(cache, b.T, Q=rows, Q_out=rows, heads=H, ldq=ld, ldqo=ld, K=dev_bf16(k), V=dev_bf16(v), ldk=Hk * D,
                        ldv=Hk * D, freq=dev(np.asarray(freq)), rot_dim=D)
    assert np.array_equal(host_bits(rows).reshape(turned.shape), turned)
    w = workspace(b.T, b.S, H, Hk, D)
    mx.mxgemm_paged_attention(cache, b.T, rows, rows, heads=H, scale=D ** -0.5, ldq=ld, ldo=ld, workspace=w, workspace_bytes=w.numel())
    assert np.array_equal(host_bits(rows).reshape(want[0].shape), want[0])


def test_pages_that_sequences_share():
    """Two sequences with the same first pages, and one page twice in a sequence."""
    rng = np.random.default_rng(44)
    b = Batch(rng, [2, 3], [100, 90], 2, 64, 16, True)
    b.pages[1, :4] = b.pages[0, :4]
    b.pages[1, 4] = b.pages[1, 5]
    q = bf16(rng, b.T, 4 * 64)
    check(b, q, 4, attend(b, q, 4))


def test_no_new_tokens_of_any_sequence():
    """Nothing is written, whatever T says."""
    rng = np.random.default_rng(45)
    b = Batch(rng, [0, 0], [100, 0], 2, 64, 16, False)
    q = bf16(rng, 5, 4 * 64)
    O, lse = attend(b, q, 4, rows=5)
    assert (O == 0x1234).all() and (lse == 77).all()


def test_a_column_block_of_a_wider_cache():
    """E4M3 without scales; keys and values interleaved in one buffer."""
    rng = np.random.default_rng(46)
    b = Batch(rng, [1, 20], [130, 20], 2, 128, 16, True)
    b.k_scale = b.v_scale = np.ones(2, np.float32)
    b.kc, b.vc = (ref.to_e4m3(rng.standard_normal(b.kc.shape)) for _ in range(2))
    both = dev(np.ascontiguousarray(np.stack([b.kc, b.vc], axis=3)))  # [page][head][row][2][D]
    q = bf16(rng, b.T, 4 * 128)
    b.cache()
    cache = mx.make_kv_cache(both, both.data_ptr() + 128, *b.dev, seqs=b.S, num_pages=b.num_pages, page_size=16,
                             max_pages=b.max_pages, kv_heads=2, head_dim=128, fp8=True, token_stride=256)
    w = workspace(b.T, b.S, 4, 2, 128)
    O = dev_bf16(np.zeros((b.T, 512), np.uint16))
    lse = torch.zeros((b.T, 4), device="cuda")
    mx.mxgemm_paged_attention(cache, b.T, dev_bf16(q), O, heads=4, scale=128 ** -0.5, lse=lse, ldq=512, ldo=512, workspace=w,
                              workspace_bytes=w.numel())
    check(b, q, 4, (host_bits(O).reshape(b.T, 4, 128), lse.cpu().numpy()))


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("seqs", [64, 65, 130])
def test_many_sequences_of_each_kernel(seqs, kernel, monkeypatch):
    monkeypatch.setenv("MXGEMM_ATTENTION_KERNEL", str(kernel))
    rng = np.random.default_rng(47)
    new = [int(x) for x in rng.choice([0, 1, 1, 2, 40], seqs)]
    lens = [max(n + int(rng.integers(-3, 200)), 0) for n in new]
    b = Batch(rng, new, lens, 1, 64, 16, False)
    q = bf16(rng, b.T, 4 * 64)
    say("case sequences", seqs, kernel)
    check(b, q, 4, attend(b, q, 4))


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 50)])
def test_more_units_than_workgroups(causal, window, kernel, monkeypatch):
    """Units that go out whole, by their keys: every one is done once."""
    monkeypatch.setenv("MXGEMM_ATTENTION_KERNEL", str(kernel))
    rng = np.random.default_rng(48)
    new = [1, 40, 7, 0, 33, 2, 1, 64, 5, 5, 90, 1, 3, 20, 8, 11, 0, 30, 2, 1, 9, 17, 4, 1, 6, 25, 1, 2, 3, 1, 50, 4]
    lens = [n + int(x) for n, x in zip(new, rng.integers(-4, 300, len(new)))]
    lens = [max(x, 0) for x in lens]
    b = Batch(rng, new, lens, 64, 32, 16, causal, "token")
    q = bf16(rng, b.T, 64 * 32)
    say("case units", causal, window, kernel)
    check(b, q, 64, attend(b, q, 64, causal=causal, window=window), causal=causal, window=window)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("page", [512, 4096, 65536])
def test_large_pages_and_a_wider_table(page, kernel, monkeypatch):
    monkeypatch.setenv("MXGEMM_ATTENTION_KERNEL", str(kernel))
    rng = np.random.default_rng(49)
    b = Batch(rng, [1, 3], [70000, 5000], 1, 64, page, False, spare=1)
    q = bf16(rng, b.T, 2 * 64)
    b.cache()
    table = np.full((2, b.max_pages + 5), 2 ** 30, np.int32)
    table[:, :b.max_pages] = b.pages
    table = dev(table)
    cache = mx.make_kv_cache(b.k, b.v, table, b.dev[1], b.dev[2], seqs=2, num_pages=b.num_pages, page_size=page,
                             max_pages=b.max_pages, ld_pages=b.max_pages + 5, kv_heads=1, head_dim=64)
    w = workspace(b.T, 2, 2, 1, 64)
    O = dev_bf16(np.zeros((b.T, 128), np.uint16))
    lse = torch.zeros((b.T, 2), device="cuda")
    say("case pages", page, kernel)
    mx.mxgemm_paged_attention(cache, b.T, dev_bf16(q), O, heads=2, scale=0.125, lse=lse, ldq=128, ldo=128, workspace=w,
                              workspace_bytes=w.numel())
    check(b, q, 2, (host_bits(O).reshape(b.T, 2, 64), lse.cpu().numpy()))


@pytest.mark.parametrize("kernel", KERNELS)
def test_rows_that_see_a_nan(kernel, monkeypatch):
    """A NaN among a row's keys or its query makes that row NaN, also where nothing else is seen; no other row."""
    monkeypatch.setenv("MXGEMM_ATTENTION_KERNEL", str(kernel))
    rng = np.random.default_rng(50)
    b = Batch(rng, [1, 50, 2], [1, 60, 900], 1, 64, 16, False)
    q = bf16(rng, b.T, 2 * 64)
    b.kc[b.pages[0, 0], 0, 0, 3] = 0x7FC0   # the only key of the first row
    b.kc[b.pages[1, 2], 0, 8, 1] = 0x7FC0   # key 40: rows of positions 40 to 59
    b.vc[b.pages[1, 3], 0, 2, 5] = 0x7F80   # value 50, column 5
    q[51, 2] = 0x7FC0                       # the first head of a row of 900 keys
    say("case nan", kernel)
    check(b, q, 2, attend(b, q, 2))
    sinks = np.array([0.0, -np.inf])
    check(b, q, 2, attend(b, q, 2, sinks=sinks), sinks=sinks)


@pytest.mark.parametrize("kernel", KERNELS)
def test_more_units_than_workgroups_of_many_sequences(kernel, monkeypatch):
    monkeypatch.setenv("MXGEMM_ATTENTION_KERNEL", str(kernel))
    rng = np.random.default_rng(51)
    new = [int(x) for x in rng.choice([0, 1, 1, 2, 20], 140)]
    lens = [max(n + int(rng.integers(-2, 60)), 0) for n in new]
    b = Batch(rng, new, lens, 8, 32, 16, False)
    q = bf16(rng, b.T, 8 * 32)
    say("case many units", kernel)
    check(b, q, 8, attend(b, q, 8))
    check(b, q, 8, attend(b, q, 8, window=9), window=9)


@pytest.mark.parametrize("kernel", KERNELS)
def test_bad_tables_of_each_kernel(kernel, monkeypatch):
    """Values mean nothing then; no address outside is formed and a later call is right."""
    monkeypatch.setenv("MXGEMM_ATTENTION_KERNEL", str(kernel))
    rng = np.random.default_rng(52)
    b = Batch(rng, [1, 150, 7, 1], [50, 160, 70, 80], 1, 64, 16, False)
    q = bf16(rng, b.T, 2 * 64)
    w = workspace(b.T, 4, 2, 1, 64)
    good = b.offsets.copy(), b.lens.copy(), b.pages.copy()
    for bad in ([0, 159, 0, 159, 0], [3, 1, 9, -5, 2], [2 ** 31 - 1, -2 ** 31, 0, 159, 159], [0, 1, 2, 3, 1000]):
        b.offsets = np.array(bad, np.int32)
        b.lens = np.array([2 ** 31 - 1, -7, 70, 10 ** 6], np.int32)
        b.pages = np.where(rng.random(b.pages.shape) < 0.5, 2 ** 31 - 1, b.pages).astype(np.int32)
        say("case tables", kernel, bad)
        attend(b, q, 2, w=w)
    b.offsets, b.lens, b.pages = good
    check(b, q, 2, attend(b, q, 2, w=w))
