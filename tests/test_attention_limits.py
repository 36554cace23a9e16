"""GPU tests of the attention over a paged cache at the limits of its
arguments, where 32-bit counts of keys, windows and workgroups end."""
import numpy as np
import pytest

import attention_ref as ref
import block_scaled_precision_mxfp4_amd as mx
from test_attention import Batch, attend, bf16, check, dev, say, workspace

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mxgpu import dev_bf16, host_bits  # noqa: E402

KERNELS = range(4)  # MXGEMM_ATTENTION_KERNEL: keys in turn over 32 or 64 rows, tiles of rows small and large


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 50])
def test_windows_longer_than_any_sequence_hide_nothing(window, causal, kernel, monkeypatch):
    """Sequences longer and shorter than their new tokens: positions from -70 on."""
    monkeypatch.setenv("MXGEMM_ATTENTION_KERNEL", str(kernel))
    for heads, D, fp8 in ((1, 64, False), (4, 128, True), (2, 256, False)):
        rng = np.random.default_rng(60)
        b = Batch(rng, [40, 100, 1, 90], [35, 100, 300, 20], 1, D, 16, fp8)
        q = bf16(rng, b.T, heads * D, sigma=2.0)
        say("case long windows", window, causal, kernel, D)
        check(b, q, heads, attend(b, q, heads, causal=causal, window=window), causal=causal, window=window)


@pytest.mark.parametrize("kernel", KERNELS)
def test_lengths_up_to_the_largest_capacity(kernel, monkeypatch):
    """Contexts of up to 2^31 - 16 keys, nearly all of them the same two pages again and again.

    Those have scores of 0, and values that are small whole numbers: their sums (of up to 2^24 in a wave) are exact.  The
    last 240 keys and more weigh as much as all others together.  What may be off: as in attention_ref.attention, with the
    additions of the parts (512 at most) in the place of those of the keys."""
    monkeypatch.setenv("MXGEMM_ATTENTION_KERNEL", str(kernel))
    rng = np.random.default_rng(61)
    H, D, P, n = 2, 64, 16, 3
    max_pages = 2 ** 27 - 1
    last = max_pages - 15  # from this page of the sequence on: page 2
    half = max_pages // 2
    kc, vc = bf16(rng, 3, 1, P, D), bf16(rng, 3, 1, P, D)
    kc[:2] = 0
    vc[0], vc[1] = 0x3F80, 0xC000  # 1, -2
    kc[2, :, :, 0] = 0x41C0        # 24
    q = bf16(rng, n, H, D, sigma=0.25)
    q[:, :, 0] = 0x3F80            # 1
    k, v, qf = (ref.bf16_to_f64(x) for x in (kc, vc, q))
    scale = 0.6875
    table = torch.zeros((1, max_pages), dtype=torch.int32, device="cuda")
    table[0, half:], table[0, last:] = 1, 2
    offsets, K, V, Q = dev(np.array([0, n], np.int32)), dev_bf16(kc), dev_bf16(vc), dev_bf16(q.reshape(n, -1))
    w = workspace(n, 1, H, 1, D)

    def seen(page, row, lo, hi):
        """Keys of [lo, hi) that are this row of this page."""
        first = (0, half, last)[page] * P
        end = (half, last, max_pages)[page] * P
        a, b = max(lo, first), min(hi, end)
        return max((b - row + P - 1) // P - (a - row + P - 1) // P, 0) if b > a else 0

    for length in (max_pages * P, max_pages * P - 1, max_pages * P - 100, 2 ** 31 - 128):
        for causal, window in ((True, 0), (False, 0), (True, 150), (True, 2 ** 31 - 200)):
            lens = dev(np.array([length], np.int32))
            cache = mx.make_kv_cache(K, V, table, offsets, lens, seqs=1, num_pages=3, page_size=P, max_pages=max_pages,
                                     kv_heads=1, head_dim=D)
            O = dev_bf16(np.zeros((n, H * D), np.uint16))
            lse = torch.zeros((n, H), device="cuda")
            say("case capacity", kernel, length, causal, window)
            mx.mxgemm_paged_attention(cache, n, Q, O, heads=H, scale=scale, lse=lse, ldq=H * D, ldo=H * D, causal=causal,
                                      window=window, workspace=w, workspace_bytes=w.numel())
            o, l = ref.bf16_to_f64(host_bits(O)).reshape(n, H, D), lse.cpu().numpy()
            for t in range(n):
                p = length - n + t
                lo, hi = max(p - window + 1, 0) if window else 0, p + 1 if causal else length
                count = np.array([[seen(page, row, lo, hi) for row in range(P)] for page in range(3)])
                assert count.sum() == hi - lo
                for h in range(H):
                    x = k[:, 0] @ qf[t, h] * scale
                    size = np.abs(k[:, 0]) @ np.abs(qf[t, h]) * scale
                    m = x[count > 0].max()
                    e = count * np.exp(x - m)
                    total = e.sum()
                    want = np.einsum("pr,prd->d", e, v[:, 0]) / total
                    mag = np.einsum("pr,prd->d", e, np.abs(v[:, 0])) / total
                    dx = (D + 5) * ref.F32 * size.max() + 4 * ref.F32 * np.abs(x).max()
                    sums = (512 + 64) * ref.F32
                    off = ref.BF16 * np.abs(want) * (1 + ref.BF16) + (ref.BF16 + 2 * dx + 2 ** -21 + 2 * sums) * mag
                    assert (np.abs(o[t, h] - want) <= off).all()
                    full = m + np.log(total)
                    assert abs(l[t, h] - full) <= 2 * dx + 2 ** -21 + sums + 8 * ref.F32 * abs(full)
    assert not w[:4096].any()


def test_more_tiles_than_a_launch_has_workgroups_for():
    """65536 sequences of 170 key heads that may each end in a tile of their own: 2^24 workgroups of 256 threads would
    be 2^32.  Few sequences have tokens; the rows behind them are left as they were (and most of them never touched)."""
    rng = np.random.default_rng(62)
    H, D, S, T = 170, 32, 65536, 4310000
    assert H * ((T + S * 127) // 128) * 256 >= 2 ** 32
    b = Batch(rng, [1, 70, 0, 3, 1], [30, 75, 5, 2, 1], H, D, 16, False)
    q = bf16(rng, b.T, H * D, sigma=2.0)
    b.cache()
    at = np.array([0, 64, 65, 40000, S - 1])  # where those sequences are
    new, lens = np.zeros(S, np.int64), np.zeros(S, np.int32)
    new[at], lens[at] = b.new, b.lens
    offsets = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    pages = np.zeros((S, b.max_pages), np.int32)
    pages[at] = b.pages
    cache_dev = dev(pages), dev(offsets), dev(lens)
    cache = mx.make_kv_cache(b.k, b.v, *cache_dev, seqs=S, num_pages=b.num_pages, page_size=16, max_pages=b.max_pages,
                             kv_heads=H, head_dim=D)
    rows = torch.empty((T, H * D), dtype=torch.bfloat16, device="cuda")  # 47 GB, in place
    rows[:b.T] = dev_bf16(q)
    rows[b.T:b.T + 50] = 3.0
    w = workspace(T, S, H, H, D)
    lse = torch.full((T, H), 77.0, device="cuda")
    say("case tiles")
    mx.mxgemm_paged_attention(cache, T, rows, rows, heads=H, scale=D ** -0.5, lse=lse, ldq=H * D, ldo=H * D, workspace=w,
                              workspace_bytes=w.numel())
    torch.cuda.synchronize()
    assert not w[:4096].any()
    assert (rows[b.T:b.T + 50] == 3.0).all() and (lse[b.T:] == 77).all()
    check(b, q, H, (host_bits(rows[:b.T]).reshape(b.T, H, D), lse[:b.T].cpu().numpy()))
    del rows, lse
    torch.cuda.empty_cache()


def nan_batch(rng):
    """As in test_attention_kernels.test_rows_that_see_a_nan: NaN keys, a NaN query, an infinite value."""
    b = Batch(rng, [1, 50, 2], [1, 60, 900], 1, 64, 16, False)
    q = bf16(rng, b.T, 2 * 64)
    b.kc[b.pages[0, 0], 0, 0, 3] = 0x7FC0
    b.kc[b.pages[1, 2], 0, 8, 1] = 0x7FC0
    b.vc[b.pages[1, 3], 0, 2, 5] = 0x7F80
    q[51, 2] = 0x7FC0
    return b, q


@pytest.mark.parametrize("kernel", KERNELS)
def test_logarithms_of_rows_that_see_a_nan(kernel, monkeypatch):
    """lse is NaN where a score is, and nowhere else."""
    monkeypatch.setenv("MXGEMM_ATTENTION_KERNEL", str(kernel))
    b, q = nan_batch(np.random.default_rng(63))
    for sinks in (None, np.array([0.0, -np.inf])):
        _, want, _, _ = ref.attention(ref.bf16_to_f64(q).reshape(-1, 2, 64), b.host(), 0.125, True, 0, sinks)
        say("case nan logarithms", kernel)
        _, lse = attend(b, q, 2, sinks=sinks)
        assert np.isnan(want).any() and not np.isnan(want).all()
        assert np.array_equal(np.isnan(lse), np.isnan(want))


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("sink", [np.nan, np.inf])
def test_a_sink_without_a_value_makes_every_row_of_its_head_nan(sink, kernel, monkeypatch):
    """Rows without a key too (the first 6 and the last sequence's); the other head is as if alone."""
    monkeypatch.setenv("MXGEMM_ATTENTION_KERNEL", str(kernel))
    rng = np.random.default_rng(64)
    b = Batch(rng, [40, 1, 3], [34, 500, 0], 1, 64, 16, False)
    q = bf16(rng, b.T, 2 * 64)
    say("case sinks without a value", sink, kernel)
    O, lse = attend(b, q, 2, sinks=np.array([sink, 0.5]))
    assert np.isnan(ref.bf16_to_f64(O[:, 0])).all() and np.isnan(lse[:, 0]).all()
    want = attend(b, q, 2, sinks=np.array([0.5, 0.5]))
    assert np.array_equal(O[:, 1], want[0][:, 1]) and np.array_equal(lse[:, 1], want[1][:, 1])
    check(b, q, 2, want, sinks=np.array([0.5, 0.5]))
