"""Attention over the cache against float64 with a bound for every output by itself
(tests/kv_reference.py), so that no key of a long request can be lost, misplaced or
wrongly scaled within a tolerance that the largest value of the pool sets."""

import numpy as np
import pytest
import torch

from tests.kv_reference import cache_attention, check_cache_attention
from tests.parity import np64
from tests.test_gpu_cache import CASES, FP8, _i32, _ok, make_requests

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("spread", [0, 6])
@pytest.mark.parametrize("lengths,queries,page,heads,kv_heads,step", CASES + [
    ([6000, 31, 2049], [1, 1, 1], 64, 4, 2, 0), ([4000, 100], [3, 30], 128, 8, 2, 1),
    ([5000], [70], 64, 2, 2, 0)])
def test_every_output_is_within_its_bound(lengths, queries, page, heads, kv_heads, step, spread,
                                          ress_gpu):
    """With `spread`, tokens of magnitudes 2^-6 to 2^6, and in dimensions 32 to 63 only
    a few chunks of 32 keys have values, so that these chunks are all of the output."""
    q, cache, table, off = make_requests(ress_gpu, lengths, queries, page, heads, kv_heads,
                                         seed=sum(lengths) + heads + spread, spread=spread)
    if spread:
        cache.k_scale.clamp_(max=2.0 ** -7)   # logits of order one
        v = cache.v.view(torch.uint8)
        dim = torch.arange(64, device="cuda")
        chunk = torch.arange(v.shape[0] * (page // 32), device="cuda").view(-1, page // 32, 1)
        keep = (dim < 32) | (chunk % 8 * 4 == (dim - 32) // 4 * 4)
        v.mul_(keep.repeat_interleave(32, dim=1)[:, None].to(torch.uint8))
    out, lse = ress_gpu.ress_cache_attn(q.cuda(), cache, _i32(table), _i32(lengths), _i32(off),
                                        step=step)
    _ok(ress_gpu)
    check_cache_attention(out, lse, cache_attention(q, cache, table, lengths, off, step))


@pytest.mark.parametrize("page", [64, 128])
@pytest.mark.parametrize("queries", [1, 200])
def test_each_page_counts_by_its_own_scale(queries, page, ress_gpu):
    """Pages whose value scales differ by 2^6 from one to the next, each with dimensions
    that no other page has values in: a page that is lost, or scaled like its neighbour,
    shows in its dimensions by all of them."""
    pages = 10
    n = pages * page - 7
    q, cache, table, off = make_requests(ress_gpu, [n], [queries], page, 2, 1, seed=3)
    v = cache.v.view(torch.uint8)
    for j, i in enumerate(table[0][:pages]):
        cache.v_scale[i] = 2.0 ** (6 * j - 40)
        cache.k_scale[i] = 2.0 ** (-6 - j % 4)
        mine = torch.arange(64, device="cuda") // 6 == j
        v[i].mul_(mine.to(torch.uint8))
    out, lse = ress_gpu.ress_cache_attn(q.cuda(), cache, _i32(table), _i32([n]), _i32(off))
    _ok(ress_gpu)
    ref = cache_attention(q, cache, table, [n], off)
    check_cache_attention(out, lse, ref)
    for j in range(pages):   # a page's values stand far above what the bound allows to lose
        mine = slice(6 * j, 6 * j + 6)
        assert (np.abs(ref[0][:, :, mine]) > 8 * ref[2][:, :, mine]).any()


def test_a_free_page_that_is_not_taken_is_not_flagged(ress_gpu):
    """The id 100 of no pool stands in the free list behind the one that is taken."""
    table = _i32([[5, -1], [9, -1]])
    _, slots, _, cursor = ress_gpu.ress_cache_plan(_i32([1, 64]), _i32([3, 1]), table, _i32([7, 100]),
                                                   _i32([0]), 64, 65, pages=10)
    assert ress_gpu.ress_check_device_errors() == (0, 0)
    assert slots.tolist() == [5 * 64 + 3] + list(range(9 * 64 + 1, 10 * 64)) + [7 * 64]
    assert int(cursor) == 1 and table.tolist() == [[5, -1], [9, 7]]
