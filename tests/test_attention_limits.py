"""GPU tests of the attention over a paged cache at the limits of its
arguments, where 32-bit counts of keys, windows and workgroups end."""
import numpy as np
import pytest

from test_attention import Batch, attend, bf16, check, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

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
