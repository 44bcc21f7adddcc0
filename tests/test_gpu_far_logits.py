"""Logits far beyond the exponential's range, up to the 2^30 that the operators are
made for: one key takes each row.

A float32 logit is off by at most 64 * 2^-24 of the sum N of its terms' magnitudes
(N = sum |q k| / 8), and by 2^-22 of itself from its scaling, so rows whose largest
logit lies more than 2^-16 N above the second are decided, by hundreds of nats here:
their output is the winner's value, and lse is the winner's logit to 2^-17 N.  The
winner's probability against the running reference is not 1: it holds what rounding
took from the reference, and up to 2^8 by which the row's maximum may pass it.  It
enters P V rounded to bf16 (2^-8 at most) and the normaliser unrounded, so an output is
off by (2^-8 + 2^-12) |v|, and by its own rounding, 2^-8 of it."""

import numpy as np
import pytest
import torch

from tests.parity import np64

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _ok(ress):
    status, detail = ress.ress_check_device_errors()
    assert status == 0, (status, detail)


def check(out, lse, q, k, v):
    """q, out [m, heads, 64], lse [heads, m] against k, v [n, 64]."""
    o, l = np64(out), np64(lse)
    assert np.isfinite(o).all() and np.isfinite(l).all()
    q, k, v = np64(q), np64(k), np64(v)
    for h in range(q.shape[1]):
        s = q[:, h] @ k.T / 8.0
        size = (np.abs(q[:, h]) @ np.abs(k).T / 8.0).max(axis=1)
        order = np.sort(s, axis=1)
        sure = order[:, -1] - order[:, -2] > 2.0 ** -16 * size
        assert sure.mean() > 0.9
        want = v[s.argmax(axis=1)]
        assert (np.abs(o[:, h] - want) <= (2.0 ** -7 + 2.0 ** -12) * np.abs(want))[sure].all()
        assert (np.abs(l[h] - order[:, -1]) <= 2.0 ** -17 * size)[sure].all()


@pytest.mark.parametrize("rows,keys", [(1, 40), (5, 300), (70, 500), (300, 200)])
@pytest.mark.parametrize("size", [2.0 ** 9, 2.0 ** 13])
def test_cross_attention(rows, keys, size, ress_gpu):
    g = torch.Generator().manual_seed(rows)
    q = (torch.randn(rows, 2, 64, generator=g) * size).to(torch.bfloat16)
    k = (torch.randn(keys, 1, 64, generator=g) * size).to(torch.bfloat16)
    v = torch.randn(keys, 1, 64, generator=g).to(torch.bfloat16)
    out, lse = ress_gpu.ress_cross_attn(q.cuda(), k.cuda(), v.cuda())
    _ok(ress_gpu)
    check(out, lse, q, k[:, 0], v[:, 0])


@pytest.mark.parametrize("rows,keys", [(1, 40), (5, 300), (70, 500), (300, 200)])
@pytest.mark.parametrize("size", [2.0 ** 9, 2.0 ** 13])
def test_cache_attention(rows, keys, size, ress_gpu):
    g = torch.Generator().manual_seed(rows)
    q = (torch.randn(rows, 2, 64, generator=g) * size).to(torch.bfloat16)
    k = torch.randn(keys, 1, 64, generator=g) * size
    v = torch.randn(keys, 1, 64, generator=g)
    pages = -(-keys // 64)
    cache = ress_gpu.make_cache(pages, 1, 64)
    ress_gpu.ress_cache_append(k.cuda(), v.cuda(),
                               torch.arange(keys, dtype=torch.int32, device="cuda"), cache)
    table = _i32([list(range(pages))])
    out, lse = ress_gpu.ress_cache_attn(q.cuda(), cache, table, _i32([keys]), _i32([0, rows]))
    _ok(ress_gpu)
    held = [(np64(c) * np64(s)[:, :, None, None]).reshape(-1, 64)[:keys]
            for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
    check(out, lse, q, *(torch.from_numpy(x) for x in held))
