"""Host-side checks of the attention's limits on counts (no GPU)."""
import pytest

import block_scaled_precision_mxfp4_amd as mx
from test_attention_host import REACHED, SHAPE, attention, built, cache  # noqa: F401


def units_and_groups(T, seqs, heads, kv_heads, capacity):
    """Tiles of 32 rows at most, and the steps that a unit may count."""
    return kv_heads * ((T * heads // kv_heads + min(T, seqs) * 31) // 32), -(-capacity // 128) + 2


@pytest.mark.parametrize("T,seqs,heads,capacity,status", [
    (65, 64, 102, 42107264, SHAPE),         # 2^31 - 128 steps: 512 workgroups' whole pieces would pass 2^31
    (65, 64, 102, 42107264 - 128, REACHED),
    (149761, 1, 7, 1 << 23, SHAPE),         # 2^31 - 2
    (149761, 1, 7, (1 << 23) - 128, REACHED),
])
def test_steps_that_whole_pieces_would_take_past_32_bits_are_refused(T, seqs, heads, capacity, status):
    units, steps = units_and_groups(T, seqs, heads, heads, capacity)
    assert (units * steps > 2 ** 31 - 1 - 512) == (status == SHAPE) and units * steps < 2 ** 31
    c = cache(seqs=seqs, kv_heads=heads, max_pages=capacity // 16, ld_pages=capacity // 16)
    n = mx.mxgemm_paged_attention_workspace_bytes(T, seqs, heads, heads, 64)
    got = attention(c, T=T, nbytes=n, heads=heads, ldq=heads * 64, ldo=heads * 64)
    assert got == status if status == SHAPE else got in status
