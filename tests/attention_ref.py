"""Plain 64-bit implementations of the attention operators over a paged cache,
in numpy, sharing no code with the library, and the tolerances their tests use.

A batch is a dict of numpy arrays and plain values: offsets, lens, pages,
page_size, num_pages, and the cache's k and v [num_pages, kv_heads, page_size,
D] as the values that their elements stand for."""
from __future__ import annotations

import numpy as np

from experts_ref import bf16_to_f64, f64_to_bf16  # noqa: F401

BF16 = 2.0 ** -8   # half a step, relative
F32 = 2.0 ** -24


def e4m3_values():
    """The value of each E4M3 code, by its fields."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, (c & 7).astype(np.float64)
    v = np.where(e == 0, f / 512, (8 + f) * np.ldexp(1.0, e - 10))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >> 7, -v, v)


def to_e4m3(x):
    """float32 or float64 values to codes: nearest even, saturating at 448, NaN 0x7F with the sign left open."""
    x = np.asarray(x, np.float64)
    m = np.minimum(np.where(np.isnan(x), 0, np.abs(x)), 448.0)
    e = np.maximum(np.frexp(m)[1] - 1, -6)
    q = np.rint(np.ldexp(m, 3 - e)).astype(int)
    code = np.where(q >= 8, (e + 7) * 8 + (q - 8), q)  # (16: the next exponent's 8, which the sum gives)
    return np.where(np.isnan(x), 127, code).astype(np.uint8) | np.where(np.signbit(x), 128, 0).astype(np.uint8)


def sequences(b, T):
    """(s, first row, new tokens, length) as the operators clamp them."""
    cap = b["pages"].shape[1] * b["page_size"]
    for s in range(len(b["lens"])):
        o0, o1 = (int(np.clip(b["offsets"][s + i], 0, T)) for i in (0, 1))
        yield s, o0, max(o1 - o0, 0), int(np.clip(b["lens"][s], 0, cap))


def gather(b, s, n, pool):
    """The first n tokens of sequence s: [kv_heads, n, D]; pages that do not exist are zeros."""
    P = b["page_size"]
    out = np.zeros((pool.shape[1], n, pool.shape[3]))
    for i in range(n):
        page = int(b["pages"][s, i // P])
        if 0 <= page < b["num_pages"]:
            out[:, i] = pool[page, :, i % P]
    return out


def attention(Q, b, scale, causal, window, sinks=None):
    """Q [T, H, D] -> O, lse, how far O and lse may be off.  Rows without a sequence: NaN, NaN, 0, 0.

    Off: a score is a sum of D exact products in fp32, (D + 1) 2^-24 of its terms' magnitudes, times a factor with three
    roundings, and its difference to the maximum is rounded once more (2^-24 of the larger; the maximum itself drops
    out): an error dx of the exponent, and 2^-22 for the exponential itself.  Each p is rounded to bf16, half a step, and
    enters a sum over the keys that rounds each partial sum; so does l.  Then O is rounded to bf16, half a step."""
    T, H, D = Q.shape
    Hk = b["k"].shape[1]
    G = H // Hk
    O, lse = np.full((T, H, D), np.nan), np.full((T, H), np.nan)
    off, off_lse = np.zeros((T, H, D)), np.zeros((T, H))
    for s, t0, n, L in sequences(b, T):
        if n == 0:
            continue
        k, v = gather(b, s, L, b["k"]), gather(b, s, L, b["v"])
        for i in range(n):
            p = L - n + i
            lo = max(p - window + 1, 0) if window else 0
            hi = 0 if p < 0 else min(p + 1, L) if causal else L
            for h in range(H):
                kk, vv = k[h // G, lo:hi], v[h // G, lo:hi]
                with np.errstate(invalid="ignore", over="ignore"):
                    x = kk @ Q[t0 + i, h] * scale
                    size = np.abs(kk) @ np.abs(Q[t0 + i, h]) * abs(scale)
                sink = -np.inf if sinks is None else float(sinks[h])
                m = max(x.max(initial=-np.inf), sink)
                if m == -np.inf:
                    O[t0 + i, h], lse[t0 + i, h] = 0, -np.inf
                    continue
                with np.errstate(invalid="ignore", over="ignore"):
                    e = np.exp(x - m)
                    total = e.sum() + np.exp(sink - m)
                    O[t0 + i, h] = e @ vv / total
                    mag = e @ np.abs(vv) / total
                    lse[t0 + i, h] = m + np.log(total)
                    fin = np.isfinite(x)
                    dx = ((D + 5) * F32 * size[fin].max(initial=0) + 4 * F32 * np.abs(x[fin]).max(initial=0)
                          + 4 * F32 * (abs(sink) if sink > -np.inf else 0))
                    keys = (len(x) + 64) * F32
                    off[t0 + i, h] = BF16 * np.abs(O[t0 + i, h]) * (1 + BF16) + (BF16 + 2 * dx + 2 ** -21 + 2 * keys) * mag + 2.0 ** -133
                    off_lse[t0 + i, h] = 2 * dx + 2 ** -21 + keys + 8 * F32 * abs(lse[t0 + i, h])
    return O, lse, off, off_lse


def turn(x, pos, freq, rot, interleaved, factor):
    """x [heads, D] of one token turned to position pos; and the magnitudes its errors go by."""
    y, mag = x.copy(), np.zeros_like(x)
    a = float(pos) * np.asarray(freq, np.float64)
    c, s = np.cos(a) * factor, np.sin(a) * factor
    h = rot // 2
    i, j = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved else (np.arange(h), h + np.arange(h))
    y[:, i], y[:, j] = x[:, i] * c - x[:, j] * s, x[:, j] * c + x[:, i] * s
    mag[:, i] = mag[:, j] = (np.abs(x[:, i]) + np.abs(x[:, j])) * abs(factor)
    return y, mag


# What the turn's arithmetic may be off, relative to turn()'s magnitudes: the reduced angle is rounded to fp32 (up to a
# half turn: pi 2^-24), cosine and sine are good to 2^-22, and the products and their sum round three times.
TURN = 2.0 ** -20


def append(b, Q, K, V, freq, rot, interleaved, factor, positions=None):
    """-> turned Q, rows of K and V by (page, row) for the tokens that have a place, magnitudes; NaN rows: no sequence."""
    T = next(x.shape[0] for x in (Q, K) if x is not None)
    P = b["page_size"]
    out = np.full_like(Q, np.nan) if Q is not None else None
    qmag = np.zeros_like(Q) if Q is not None else None
    places = {}
    for s, t0, n, L in sequences(b, T):
        for i in range(n):
            t, p = t0 + i, L - n + i
            at = p if positions is None else int(positions[t])
            if Q is not None:
                out[t], qmag[t] = turn(Q[t], at, freq, rot, interleaved, factor)
            if K is not None and p >= 0:
                page = int(b["pages"][s, p // P])
                if 0 <= page < b["num_pages"]:
                    places[page, p % P] = (*turn(K[t], at, freq, rot, interleaved, factor), V[t])
    return out, qmag, places
