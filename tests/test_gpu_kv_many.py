"""Batches of more sequences than a warp has lanes (the plan then reads their lengths
again where it needs them), up to the largest number, and head groups of every size,
against float64."""

import numpy as np
import pytest
import torch

from tests.kv_reference import cache_attention, check_cache_attention
from tests.parity import np64
from tests.test_gpu_cache import (_filled_cache, _i32, _ok, _slots_of, append_ref,
                                  make_requests)
from tests.test_gpu_cross import _off, close, close_lse, make, reference

pytestmark = pytest.mark.gpu


def _ragged(seed, count, most, empty=0.2):
    rng = np.random.default_rng(seed)
    n = rng.integers(1, most + 1, count)
    n[rng.random(count) < empty] = 0
    return n.tolist()


def _check_cross(nq, nk, heads, kv_heads, qlen, klen, ress):
    q, k, v, do = make(nq, nk, heads, kv_heads, seed=len(nq) + heads, qlen=qlen, klen=klen)
    dev = [t.cuda() for t in (q, k, v)]
    seqs = dict(q_offsets=_off(nq), kv_offsets=_off(nk),
                q_lens=None if qlen is None else _i32(qlen),
                kv_lens=None if klen is None else _i32(klen))
    out, lse = ress.ress_cross_attn(*dev, **seqs)
    grads = ress.ress_cross_attn_bwd(*dev, out, lse, do.cuda(), **seqs)
    _ok(ress)
    ref = reference(q, k, v, nq, nk, qlen, klen, do, out, lse)
    close(out, ref, "out")
    close_lse(lse, ref)
    for name, t in zip(("dq", "dk", "dv"), grads):
        close(t, ref, name)


@pytest.mark.parametrize("count,mq,mk,heads,kv_heads", [
    (33, 40, 300, 2, 2), (100, 200, 60, 4, 1), (700, 9, 20, 2, 1), (8192, 2, 5, 1, 1),
    (40, 1, 400, 2, 2)])
def test_cross_attention_of_many_sequences(count, mq, mk, heads, kv_heads, ress_gpu):
    nq, nk = _ragged(count, count, mq), _ragged(count + 1, count, mk)
    _check_cross(nq, nk, heads, kv_heads, None, None, ress_gpu)
    rng = np.random.default_rng(count)
    _check_cross(nq, nk, heads, kv_heads, [int(rng.integers(0, n + 1)) for n in nq],
                 [int(rng.integers(0, n + 1)) for n in nk], ress_gpu)


def test_cross_attention_of_many_equal_sequences(ress_gpu):
    _check_cross([20] * 64, [150] * 64, 4, 2, None, None, ress_gpu)


@pytest.mark.parametrize("heads,kv_heads", [(64, 1), (48, 1), (60, 4), (63, 9), (50, 2), (5, 1)])
def test_cross_attention_of_any_group(heads, kv_heads, ress_gpu):
    """Groups that do not divide a tile of 128 rows, and one that leaves two tokens to it."""
    _check_cross([37, 5], [200, 131], heads, kv_heads, [30, 5], [200, 100], ress_gpu)


@pytest.mark.parametrize("count,most,queries,heads,kv_heads,step", [
    (33, 500, 1, 2, 1, 0), (300, 90, 3, 2, 2, 1), (8192, 40, 1, 1, 1, 0), (8192, 3, 2, 2, 1, 1),
    (40, 300, 120, 2, 2, 0), (60, 200, 90, 2, 1, 7), (2000, 70, 1, 64, 8, 0)])
def test_cache_attention_of_many_requests(count, most, queries, heads, kv_heads, step, ress_gpu):
    lengths = _ragged(count, count, most)
    rows = [min(queries, max(n, 1)) for n in lengths]
    q, cache, table, off = make_requests(ress_gpu, lengths, rows, 64, heads, kv_heads, seed=count)
    if heads > 8:          # the reference is a loop over rows and heads
        keep = slice(0, 60)
        lengths, rows = lengths[keep], rows[keep]
    out, lse = ress_gpu.ress_cache_attn(q.cuda(), cache, _i32(table), _i32(lengths + [0] * (count - len(lengths))),
                                        _i32(off), step=step)
    _ok(ress_gpu)
    n = sum(rows)
    check_cache_attention(out[:n], lse[:, :n],
                          cache_attention(q[:n], cache, table, lengths, off, step))


@pytest.mark.parametrize("heads,kv_heads", [(64, 1), (48, 1), (60, 4), (63, 9), (50, 2), (5, 1)])
@pytest.mark.parametrize("queries,step", [([1, 2], 0), ([3, 1], 1), ([90, 20], 1)])
def test_cache_attention_of_any_group(queries, step, heads, kv_heads, ress_gpu):
    lengths = [150, 70]
    q, cache, table, off = make_requests(ress_gpu, lengths, queries, 128, heads, kv_heads,
                                         seed=heads)
    out, lse = ress_gpu.ress_cache_attn(q.cuda(), cache, _i32(table), _i32(lengths), _i32(off),
                                        step=step)
    _ok(ress_gpu)
    check_cache_attention(out, lse, cache_attention(q, cache, table, lengths, off, step))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page,heads,counts", [
    (64, 1, [1] * 5000), (128, 1, [1] * 4200), (64, 2, [3, 1, 70, 5, 130] * 30),
    (128, 1, [2, 300, 1, 7] * 20), (64, 1, [1] * 1500 + [200])])
def test_append_of_many_short_runs(page, heads, counts, dtype, ress_gpu):
    """Runs that start next to one another in the windows of every size that the kernel
    takes (a token, eight, a page), with gaps of skipped tokens between them."""
    rng = np.random.default_rng(len(counts) + page)
    starts = [int(x) for x in rng.integers(0, page, len(counts))]
    pages = sum(-(-(s + n) // page) for s, n in zip(starts, counts)) + 1
    ids = rng.permutation(pages).tolist()
    slots = _slots_of(starts, counts, page, ids)
    for i in rng.integers(0, len(slots), len(slots) // 50):
        slots[i] = -1                                   # the run ends here
    # what is behind a gap would be a second run of its page: it goes as well
    for i in range(1, len(slots)):
        if slots[i - 1] == -1 and slots[i] >= 0 and slots[i] % page and \
                any(s >= 0 and s // page == slots[i] // page for s in slots[max(0, i - page):i]):
            slots[i] = -1
    g = torch.Generator().manual_seed(page)
    cache = _filled_cache(ress_gpu, pages, heads, page, seed=7)
    x = [(torch.randn(len(slots), heads, 64, generator=g)
          * torch.exp2(torch.randint(-3, 6, (len(slots), heads, 1), generator=g).float())).to(dtype)
         for _ in range(2)]
    ref = [append_ref(np64(t), slots, np64(c), np64(s), page)
           for t, c, s in ((x[0], cache.k, cache.k_scale), (x[1], cache.v, cache.v_scale))]
    ress_gpu.ress_cache_append(x[0].cuda(), x[1].cuda(), _i32(slots), cache)
    _ok(ress_gpu)
    for (codes, scale), c, s in ((ref[0], cache.k, cache.k_scale), (ref[1], cache.v, cache.v_scale)):
        assert np.array_equal(np64(s), scale) and np.array_equal(np64(c), codes)
