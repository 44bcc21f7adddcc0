"""Attention over the paged 8-bit cache in float64, with a bound for every output.

A probability enters P V rounded to bf16 or f16 (at most half a step, 2^-8
relative) while the normaliser is not rounded, and the exponentials and float32
sums are good to 2^-12 together (ex2 of a difference of logits to 2^-14, sums of
a few thousand terms), so an output is off by at most (2^-8 + 2^-12) sum p |v|
and by its own rounding, 2^-8 of it.  The probabilities' roundings are
independent, so this also bounds what a kernel may lose of any one key."""

import math

import numpy as np

from tests.parity import np64


def cache_attention(q, cache, table, lengths, offsets, step=0):
    """(out, lse, bound) of float64; pages outside the pool are left out."""
    qn = np64(q)
    k, v = (np64(c) * np64(s)[:, :, None, None] for c, s in ((cache.k, cache.k_scale),
                                                            (cache.v, cache.v_scale)))
    pool, hk, page, _ = k.shape
    n_rows, heads = qn.shape[:2]
    out, bound = np.zeros(qn.shape), np.zeros(qn.shape)
    lse = np.full((heads, n_rows), -np.inf)
    for r, n in enumerate(lengths):
        rows = np.arange(offsets[r], offsets[r + 1])
        cell = np.arange(n)
        ids = np.asarray(table[r])[cell // page] if n else cell
        here = (ids >= 0) & (ids < pool)
        ids = np.where(here, ids, 0)
        pos = n - len(rows) + np.arange(len(rows))
        end = np.full(len(rows), n) if step == 0 else \
            np.where(pos >= 0, np.minimum(n, (pos // step + 1) * step), 0)
        seen = here[None] & (cell[None] < end[:, None])
        for h in range(heads):
            K, V = (x[ids, h // (heads // hk), cell % page] for x in (k, v))
            for i, row in enumerate(rows):
                ok = seen[i]
                if not ok.any():
                    continue
                s = K[ok] @ qn[row, h] / 8.0
                top = s.max()
                p = np.exp(s - top)
                z = p.sum()
                lse[h, row] = top + math.log(z)
                out[row, h] = p @ V[ok] / z
                bound[row, h] = (2.0 ** -8 + 2.0 ** -12) * (p @ np.abs(V[ok]) / z)
    return out, lse, bound + 2.0 ** -8 * np.abs(out)


def check_cache_attention(out, lse, ref):
    """Every output within its bound, and lse within 1e-4 + 1e-5 |lse|: logits are
    float32 sums of 64 exact products (|error| <= 64 * 2^-24 * sum |q k| / 8, below
    2^-14 for sums up to 64), and ex2 and lg2 are good to 2^-20."""
    want, wlse, bound = ref
    o, l = np64(out), np64(lse)
    assert np.isfinite(o).all()
    far = np.abs(o - want) / (bound + 1e-300)
    assert far.max(initial=0.0) <= 1.0, (float(far.max()), np.unravel_index(far.argmax(), far.shape))
    dead = np.isinf(wlse)
    assert np.array_equal(np.isinf(l), dead) and (l[dead] < 0).all()
    err = np.abs(l[~dead] - wlse[~dead])
    assert (err <= 1e-4 + 1e-5 * np.abs(wlse[~dead])).all(), err.max()
