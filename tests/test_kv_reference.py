"""The bounds of tests/kv_reference.py tell a lost chunk of keys, and a page with its
neighbour's scale, from rounding (mistakes planted in the reference, on the CPU)."""

import numpy as np
import pytest
import torch

from block_sparse_global_mean_b200.ress import ress_cache
from tests.kv_reference import cache_attention, check_cache_attention

FP8 = torch.float8_e4m3fn


def _cache(n, seed):
    g = torch.Generator().manual_seed(seed)
    pages = -(-n // 64)
    codes = [(torch.randn(pages, 1, 64, 64, generator=g) * 100).clamp(-448, 448).to(FP8)
             for _ in range(2)]
    return ress_cache(*codes, *(torch.full((pages, 1), 2.0 ** -7) for _ in range(2)))


@pytest.mark.parametrize("mistake,n", [("none", 300), ("none", 2000), ("chunk", 300),
                                       ("chunk", 2000), ("scale", 300), ("scale", 2000),
                                       ("keys", 300)])
def test_mistakes_exceed_the_bound(mistake, n):
    """Chunks and scales in long requests too, two values exchanged in a short one."""
    q = torch.randn(6, 1, 64, generator=torch.Generator().manual_seed(n))
    cache = _cache(n, n)
    table, off = [list(range(-(-n // 64)))], [0, 6]
    ref = cache_attention(q, cache, table, [n], off)
    v, scale = cache.v.float(), cache.v_scale.clone()
    if mistake == "chunk":
        v[2, :, 32:] = 0
    elif mistake == "scale":
        scale[3] *= 2
    elif mistake == "keys":
        v[1, :, 5], v[1, :, 6] = v[1, :, 6].clone(), v[1, :, 5].clone()
    wrong = cache_attention(q, cache._replace(v=v, v_scale=scale), table, [n], off)
    out, lse = torch.from_numpy(wrong[0]).to(torch.bfloat16), torch.from_numpy(wrong[1])
    if mistake == "none":
        check_cache_attention(out, lse, ref)
        return
    assert np.array_equal(wrong[1], ref[1])      # nothing of it shows in lse
    with pytest.raises(AssertionError):
        check_cache_attention(out, lse, ref)
