"""The binding's C++ part and the Python code behind it: the same results from either,
and the same refusals, for the cache's calls (test_gpu_cross.py has the others)."""

import pytest
import torch

from tests.test_gpu_cache import _i32, _ok, make_requests

pytestmark = pytest.mark.gpu


def _equal(a, b):
    return all(torch.equal(x.view(torch.uint8) if x.element_size() == 1 else x,
                           y.view(torch.uint8) if y.element_size() == 1 else y)
               for x, y in zip(a, b))


def _without(ress, monkeypatch):
    monkeypatch.setattr(ress, "_call", None)


@pytest.mark.parametrize("queries", [1, 150])
def test_both_ways_give_the_same(queries, ress_gpu, monkeypatch):
    q, cache, table, off = make_requests(ress_gpu, [300, 200], [queries] * 2, 64, 4, 2, seed=61)
    q, table, lengths, off = q.cuda(), _i32(table), _i32([300, 200]), _i32(off)
    kv = torch.randn(70, 2, 2, 64, generator=torch.Generator().manual_seed(1)).cuda()
    slots = torch.arange(70, dtype=torch.int32, device="cuda")
    plan = _i32([40, 30]), lengths
    call, got = ress_gpu._call, []
    assert call is not None
    for fast in (True, False):
        if not fast:
            _without(ress_gpu, monkeypatch)
        mine = ress_gpu.ress_cache(*(t.clone() for t in cache))
        rows = table.clone()
        free = torch.arange(9, dtype=torch.int32, device="cuda")
        res = list(ress_gpu.ress_cache_plan(*plan, rows, free, _i32([2]), 64, 75, pages=12))
        for step in (0, 1):
            res += ress_gpu.ress_cache_attn(q, mine, table, lengths, off, step=step)
        ress_gpu.ress_cache_append(kv[:, 0], kv[:, 1], slots, mine)
        ress_gpu.ress_cache_append(kv[:, 0].bfloat16(), kv[:, 1].bfloat16(), slots + 70, mine)
        out, none = ress_gpu.ress_cache_attn(q, mine, table, lengths, off, want_lse=False)
        assert none is None
        got.append(res + [rows, out] + list(mine))
    _ok(ress_gpu)
    assert _equal(*got)
    # the C++ part made the first calls itself
    assert call.cache_attn(q, *cache, table, lengths, off, 0, True) is not None
    assert call.cache_plan(*plan, table.clone(), free, _i32([2]), 64, 75, None) is not None
    torch.cuda.synchronize()
    ress_gpu.ress_check_device_errors()


def test_both_ways_refuse_the_same(ress_gpu, monkeypatch):
    q, cache, table, off = make_requests(ress_gpu, [300, 200], [1, 1], 64, 4, 2, seed=62)
    q, table, lengths, off = q.cuda(), _i32(table), _i32([300, 200]), _i32(off)
    k = torch.randn(5, 2, 64, device="cuda")
    slots, one = _i32([0, 1, 2, 3, 4]), _i32([0])
    attn, append, plan = (ress_gpu.ress_cache_attn, ress_gpu.ress_cache_append,
                          ress_gpu.ress_cache_plan)
    free = torch.arange(9, dtype=torch.int32, device="cuda")
    calls = [
        lambda: attn(q.float(), cache, table, lengths, off),
        lambda: attn(q[:, :3].contiguous(), cache, table, lengths, off),      # 3 heads over 2
        lambda: attn(q, cache, table.long(), lengths, off),
        lambda: attn(q, cache, table, lengths[:1], off),
        lambda: attn(q, cache, table, lengths, off[:2]),
        lambda: attn(q, cache, table.t(), lengths, off),
        lambda: attn(q, cache, table, lengths, off, step=-1),
        lambda: attn(q, cache, table, lengths, off, step=2 ** 31),
        lambda: attn(q, cache._replace(k=cache.k.view(torch.uint8)), table, lengths, off),
        lambda: attn(q, cache._replace(v_scale=cache.v_scale.double()), table, lengths, off),
        lambda: attn(q, cache._replace(v=cache.v[:-1]), table, lengths, off),
        lambda: attn(q, cache, table.cpu(), lengths, off),
        lambda: attn(q[:, :, :32].contiguous(), cache, table, lengths, off),
        lambda: attn(q[:, :, ::2], cache, table, lengths, off),
        lambda: append(k, k, slots[:4], cache),
        lambda: append(k, k.bfloat16(), slots, cache),
        lambda: append(k.half(), k.half(), slots, cache),
        lambda: append(k[:, :1], k[:, :1], slots, cache),
        lambda: append(k.transpose(0, 1).contiguous().transpose(0, 1), k, slots, cache),
        lambda: append(k, k, slots.long(), cache),
        lambda: plan(lengths, lengths, table, free, one, 32, 5),
        lambda: plan(lengths, lengths, table, free, one, 64, -5),
        lambda: plan(lengths, lengths, table, free, free[:2], 64, 5),
        lambda: plan(lengths.float(), lengths, table, free, one, 64, 5),
        lambda: plan(lengths[:1], lengths, table, free, one, 64, 5),
        lambda: plan(lengths, lengths, table, free, one, 64, 5, pages=0),
        lambda: plan(lengths, lengths, table, free, one, 64, 2 ** 30 + 1),
    ]
    errors = []
    for fast in (True, False):
        if not fast:
            _without(ress_gpu, monkeypatch)
        for i, f in enumerate(calls):
            with pytest.raises((ValueError, TypeError, ress_gpu.RessError)) as e:
                f()
            errors.append((i, type(e.value), str(e.value)))
    assert errors[:len(calls)] == errors[len(calls):]
    _ok(ress_gpu)
