"""NaN codes in the cache: a token whose key or value holds one makes NaN every row
that sees it (all 64 values and lse), whichever kernel serves the call, and changes no
bit of any other row."""

import numpy as np
import pytest
import torch

from tests.test_gpu_cache import _i32, _ok, make_requests

pytestmark = pytest.mark.gpu


def sees(rows, n, step):
    """[rows, n]: which tokens the last `rows` of n tokens see."""
    pos = n - rows + np.arange(rows)
    end = np.full(rows, n) if step == 0 else \
        np.where(pos >= 0, np.minimum(n, (pos // step + 1) * step), 0)
    return np.arange(n)[None] < end[:, None]


@pytest.mark.parametrize("part", ["k", "v"])
@pytest.mark.parametrize("code", [0x7F, 0xFF])
@pytest.mark.parametrize("page,heads,kv_heads,queries,step", [
    (64, 2, 2, [1, 1], 0), (64, 4, 1, [5, 2], 1), (128, 4, 2, [16, 7], 3), (64, 1, 1, [33, 20], 1),
    (64, 4, 2, [150, 80], 0), (64, 2, 2, [150, 80], 1), (128, 6, 2, [200, 64], 100),
    (64, 4, 4, [300, 90], 7)])
def test_nan_codes_reach_the_rows_that_see_them(page, heads, kv_heads, queries, step, code, part,
                                                ress_gpu):
    lengths = [300, 90]
    q, cache, table, off = make_requests(ress_gpu, lengths, queries, page, heads, kv_heads,
                                         seed=heads + step)
    args = _i32(table), _i32(lengths), _i32(off)
    want, wlse = ress_gpu.ress_cache_attn(q.cuda(), cache, *args, step=step)
    for r, token, head in ((0, 297, 0), (0, 140, kv_heads - 1), (1, 3, 0), (1, 88, kv_heads - 1)):
        bad = ress_gpu.ress_cache(*(t.clone() for t in cache))
        cells = getattr(bad, part).view(torch.uint8)
        cells[table[r][token // page], head, token % page, 61] = code
        out, lse = ress_gpu.ress_cache_attn(q.cuda(), bad, *args, step=step)
        _ok(ress_gpu)
        rows = torch.zeros(q.shape[0], heads, dtype=torch.bool)
        g = heads // kv_heads
        rows[off[r]:off[r + 1], head * g:(head + 1) * g] = torch.from_numpy(
            sees(queries[r], lengths[r], step)[:, token])[:, None]
        rows = rows.cuda()
        assert out[rows].isnan().all() and lse.t()[rows].isnan().all(), (r, token)
        assert torch.equal(out[~rows], want[~rows]), (r, token)
        assert torch.equal(lse.t()[~rows], wlse.t()[~rows]), (r, token)
