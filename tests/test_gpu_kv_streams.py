"""Calls whose inputs another stream writes: each operator's first kernel starts while the
kernel before it on its own stream ends, and must wait for the other stream all the same."""

import pytest
import torch

from tests.test_gpu_cache import _i32, _ok, make_requests

pytestmark = pytest.mark.gpu


def _ops(ress):
    """name -> (input that the other stream writes, its new contents, call)."""
    g = torch.Generator().manual_seed(9)
    q = torch.randn(300, 4, 64, generator=g).to(torch.bfloat16).cuda()
    k, v = (torch.randn(500, 2, 64, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    out, lse = ress.ress_cross_attn(q, k, v)
    qc, cache, table, off = make_requests(ress, [300, 200], [1, 1], 64, 4, 2, seed=71)
    qm, cache2, table2, off2 = make_requests(ress, [300, 200], [150, 60], 64, 4, 2, seed=72)
    qc, qm, table, table2 = qc.cuda(), qm.cuda(), _i32(table), _i32(table2)
    off, off2, lengths = _i32(off), _i32(off2), _i32([300, 200])
    added, free = _i32([3, 70]), torch.arange(10, dtype=torch.int32, device="cuda")
    slots = torch.arange(64, dtype=torch.int32, device="cuda")
    new = torch.randn(64, 2, 64, generator=g).cuda()

    def append():
        mine = ress.make_cache(1, 2, 64)
        ress.ress_cache_append(new, new, slots, mine)
        return [t.view(torch.uint8) if t.element_size() == 1 else t for t in mine]

    return {
        "cross": (k, torch.randn(k.shape, generator=g), lambda: ress.ress_cross_attn(q, k, v)),
        "bwd": (v, torch.randn(v.shape, generator=g),
                lambda: ress.ress_cross_attn_bwd(q, k, v, out, lse, q)),
        "plan": (added, torch.tensor([64, 1]), lambda: ress.ress_cache_plan(
            added, lengths, table.clone(), free, _i32([0]), 64, 80)),
        "append": (new, torch.randn(new.shape, generator=g), append),
        "decode": (lengths, torch.tensor([77, 130]), lambda: ress.ress_cache_attn(
            qc, cache, table, lengths, off)),
        "prefill": (qm, torch.randn(qm.shape, generator=g), lambda: ress.ress_cache_attn(
            qm, cache2, table2, _i32([300, 200]), off2, step=1)),
    }


@pytest.mark.parametrize("name", ["cross", "bwd", "plan", "append", "decode", "prefill"])
def test_inputs_written_by_another_stream(name, ress_gpu):
    x, new, call = _ops(ress_gpu)[name]
    old = x.clone()
    other, mine = torch.cuda.Stream(), torch.cuda.Stream()
    x.copy_(new)
    want = [t.clone() for t in call()]
    new = new.to(x.dtype).cuda()
    torch.cuda.synchronize()
    for _ in range(5):
        x.copy_(old)
        torch.cuda.synchronize()
        with torch.cuda.stream(mine):
            call()                                   # the kernel before, on this stream
        with torch.cuda.stream(other):
            torch.cuda._sleep(5_000_000)
            other.wait_stream(mine)                  # it has read the old contents
            x.copy_(new)
        mine.wait_stream(other)
        with torch.cuda.stream(mine):
            got = call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    _ok(ress_gpu)
