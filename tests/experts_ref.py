"""Plain 64-bit implementations of the mixture-of-experts operators, in numpy,
sharing no code with the library, and the tolerances their tests use."""
from __future__ import annotations

import numpy as np

import oracle


def bf16_to_f64(bits):
    with np.errstate(invalid="ignore"):
        return (np.asarray(bits, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def f64_to_bf16(x):
    """One rounding from 64 bits to bf16 bits (nearest, ties to even; overflow to inf)."""
    x = np.asarray(x, dtype=np.float64)
    m, e = np.frexp(np.where(np.isfinite(x), x, 0.0))
    drop = np.maximum(e - 8, -133)  # the exponent of one bf16 step (2^-133 below the normal range)
    with np.errstate(over="ignore", invalid="ignore"):
        r = np.ldexp(np.rint(np.ldexp(x, -drop)), drop)
        f = np.where(np.isfinite(x), r, x).astype(np.float32)  # exact, or beyond the range
    bits = (f.view(np.uint32) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), bits)


def quantize_fp8(bits):
    """bf16 bits [M, K] -> (E4M3 codes [M, K], E8M0 scales [M, K/32])."""
    v = bf16_to_f64(bits).reshape(bits.shape[0], -1, 32)
    special = ~np.isfinite(v).all(-1)
    v = np.where(special[..., None], 0.0, v)
    most = np.abs(v).max(-1)
    x = np.where(most > 0, np.frexp(most)[1] - 1 - 8, -127)
    x = np.clip(x, -127, 127)
    s = np.ldexp(v, -x[..., None])
    m = np.minimum(np.abs(s), 448.0)
    e = np.maximum(np.frexp(m)[1] - 1, -6)  # exponent, from the smallest normal on down the subnormal step
    q = np.rint(np.ldexp(m, 3 - e))         # in steps of 2^(e-3): 8 .. 16, below 8 only for subnormals
    e = np.where(q == 16, e + 1, e)
    q = np.where(q == 16, 8, q).astype(int)
    code = np.where(q >= 8, (e + 7) * 8 + (q - 8), q).astype(np.uint8) | np.where(np.signbit(s), 128, 0).astype(np.uint8)
    code = np.where(special[..., None], 0, code)
    return code.reshape(bits.shape).astype(np.uint8), np.where(special, 255, x + 127).astype(np.uint8)


def quantize(bits, fp8):
    return quantize_fp8(bits) if fp8 else oracle.quantize_mxfp4(bits)


def route(x, k, renorm):
    """x: float64 logits [T, E] -> ids, weights, pos, offsets, rows."""
    T, E = x.shape
    ids, weights = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        can = [e for e in range(E) if x[t, e] > -np.inf]
        best = sorted(can, key=lambda e: (-x[t, e], e))[:k]
        if not best:
            continue
        m = x[t, best[0]]
        share = lambda e: 1.0 if x[t, e] == m else np.exp(x[t, e] - m)  # noqa: E731
        total = sum(share(e) for e in (best if renorm else can))
        ids[t, :len(best)] = best
        weights[t, :len(best)] = [share(e) / total for e in best]
    rows, offsets, pos = np.full(T * k, -1, np.int32), [0], np.full((T, k), -1, np.int32)
    flat = ids.reshape(-1)
    for e in range(E):
        at = np.flatnonzero(flat == e)
        pos.reshape(-1)[at] = offsets[-1] + np.arange(len(at))
        rows[offsets[-1]:offsets[-1] + len(at)] = at // k
        offsets.append(offsets[-1] + len(at))
    return ids, weights, pos, np.array(offsets, np.int32), rows


def route_weight_tol(x, E):
    """Relative: the difference to the maximum rounds once (2^-24 of itself, which the exponential turns into a
    relative error), the exponential is good to 2^-23, each of up to E additions and the division to 2^-24; both the
    numerator and the sum carry the first two.  Absolute: fp32's smallest normal value, below which a share may be
    flushed or lose bits."""
    fin = np.where(np.isfinite(x), x, 0.0)
    span = fin.max() - fin.min()
    return (2 * span + 4 + E + 1) * 2.0 ** -24, 2.0 ** -126


def route_weight_bound(x, ids):
    """Absolute bounds [T, k] of the weights of ids (route's): relative to a weight, its own logit's distance d to its
    token's maximum rounds once (2^-24 of itself, which the exponential turns into a relative error) and the exponential is
    good to 2^-23; in the sum every share carries the same, of which the first is at most 1/e (d e^-d), each of up to E
    additions and the division round to 2^-24.  A share of d > 104 is below half of fp32's least value: with it the bound
    is fp32's smallest normal value, below which a share may be flushed or lose bits.  A logit that is masked or has the
    type's lowest value does not widen the others' bounds."""
    E = x.shape[1]
    can = np.where(x > -np.inf, x, -np.inf)
    m = can.max(1, keepdims=True)
    with np.errstate(invalid="ignore", over="ignore"):
        d = np.where(can == m, 0.0, np.minimum(m - can, 104.0))
    d = np.take_along_axis(d, np.where(ids < 0, 0, ids), 1)
    return (d + 2 + E / np.e + 2 + E + 1) * 2.0 ** -24, 2.0 ** -126


def glu(bits, K):
    """bf16 bits [M, 2K] -> bf16 bits of silu(gate) * up [M, K]."""
    g, u = bf16_to_f64(bits[:, :K]), bf16_to_f64(bits[:, K:])
    with np.errstate(over="ignore", invalid="ignore"):
        return f64_to_bf16(g / (1.0 + np.exp(-g)) * u)


def norm(Y, K, *, X=None, pos=None, weights=None, w_post=None, gate=None, res_scale=1.0, w_pre=None, eps=1e-6, T=None):
    """bf16 bits in, (h, z) bf16 bits out."""
    y = bf16_to_f64(Y)
    T = y.shape[0] if T is None else T
    if pos is not None:
        ok = (pos >= 0) & (pos < y.shape[0])
        y = (np.where(ok, weights.astype(np.float64), 0.0)[..., None] * np.where(ok[..., None], y[np.where(ok, pos, 0)], 0.0)).sum(1)
    eps = float(np.float32(eps))
    rms = lambda v: 1.0 / np.sqrt((v * v).sum(-1, keepdims=True) / K + eps)  # noqa: E731
    with np.errstate(over="ignore", invalid="ignore"):
        n = y * rms(y) * bf16_to_f64(w_post) if w_post is not None else y
        n = n * bf16_to_f64(gate) if gate is not None else n
        h = f64_to_bf16(float(np.float32(res_scale)) * n + (bf16_to_f64(X) if X is not None else 0.0))
        hv = bf16_to_f64(h)
        z = f64_to_bf16(hv * rms(hv) * bf16_to_f64(w_pre)) if w_pre is not None else h
    return h, z


def grouped(A, SA, B, SB, K, offsets, a_rows, rows, fp8, alpha=1.0, cols=None):
    """(ref, mag, written) of D [rows, len(cols)]: values in 64 bits, sums of |products|, rows that some expert has."""
    N = B.shape[1]
    cols = np.arange(N) if cols is None else cols
    ref, mag = np.zeros((rows, len(cols))), np.zeros((rows, len(cols)))
    written = np.zeros(rows, bool)
    for e in range(len(offsets) - 1):
        lo, hi = offsets[e], offsets[e + 1]
        if hi <= lo:
            continue
        src = a_rows[lo:hi] if a_rows is not None else np.arange(lo, hi)
        ok = (src >= 0) & (src < A.shape[0])
        r, m, _ = oracle.mxgemm(A, SA, B[e], SB[e], K, alpha, 0.0, rows=np.where(ok, src, 0), cols=cols,
                                a_fmt=1 if fp8 else 0)
        ref[lo:hi], mag[lo:hi] = np.where(ok[:, None], r, 0.0), np.where(ok[:, None], m, 0.0)
        written[lo:hi] = True
    return ref, abs(alpha) * mag, written


def check_grouped(d_bits, ref, mag, K, fp8, what=""):
    """|d - ref| <= 2^-8 |ref| (the output's rounding; 2^-134 below the normal range) plus the accumulation.  K additions
    each lose at most 2^-23 of a partial sum, which |products| bounds (a truncating adder loses twice a rounding one).
    With 8-bit A the instruction first adds 8 products aligned to the one with the largest exponent E and keeps them down
    to 2^(E-13) (test_experts.py pins that); each of the 7 others loses less than 2^(E-13), and the largest is at least
    2^E, so a group loses at most 7 * 2^-13 of its largest product, all groups 7 * 2^-13 of the sum of |products|.  FP4's
    products are multiples of 1/4 up to 36: nothing is lost there.  The factor 1 + 2^-8 carries the sum's error through
    the output's rounding."""
    d = bf16_to_f64(d_bits)
    assert np.array_equal(np.isnan(d), np.isnan(ref)), what + ": NaN in other places"
    fin = np.isfinite(ref)
    lost = K * 2.0 ** -23 + (7 * 2.0 ** -13 if fp8 else 0.0)
    tol = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * lost * mag + 2.0 ** -134
    off = np.where(fin, np.abs(d - np.where(fin, ref, 0.0)) - np.where(fin, tol, np.inf), -1.0)
    bad = np.argwhere(off > 0)
    assert len(bad) == 0, "%s: %d of %d outside, e.g. %s: %r, not %r" % (
        what, len(bad), d.size, tuple(bad[0]), d[tuple(bad[0])], ref[tuple(bad[0])])
