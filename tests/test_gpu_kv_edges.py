"""Edges of the paged 8-bit cache on the GPU: the largest numbers it can hold and
what lies beyond them."""

import math

import numpy as np
import pytest
import torch

from tests.kv_reference import cache_attention, check_cache_attention
from tests.parity import np64
from tests.test_gpu_cache import make_requests

pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn


def _i32(v, device="cuda"):
    return torch.tensor(v, dtype=torch.int32, device=device)


def _ok(ress):
    status, detail = ress.ress_check_device_errors()
    assert status == 0, (status, detail)


# ------------------------------------------------------------------------------------------
# the largest numbers
# ------------------------------------------------------------------------------------------
MOST = 448.0 * 2.0 ** 119


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("big,flagged", [(MOST, False), (3.3e38, True), (-3.3895e38, True)])
def test_append_of_the_largest_numbers(big, flagged, dtype, ress_gpu):
    """448 * 2^119 is what a cell holds at most: larger values are flagged, stand as
    that number and raise the scale to 2^119 and no further."""
    x = torch.full((3, 1, 64), 2.0 ** 118, dtype=dtype)
    x[1, 0, 5] = big
    cache = ress_gpu.make_cache(1, 1, 64)
    ress_gpu.ress_cache_append(x.cuda(), x.cuda(), _i32([0, 1, 2]), cache)
    status, detail = ress_gpu.ress_check_device_errors()
    assert (status, detail) == ((ress_gpu.RESS_ERR_INVALID_ARG, 105) if flagged else (0, 0))
    want = np64(x)[:, 0]
    want[1, 5] = math.copysign(MOST, big)
    for codes, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        assert np64(scale)[0, 0] == 2.0 ** 119
        assert np.array_equal(np64(codes)[0, 0, :3] * 2.0 ** 119, want)


@pytest.mark.parametrize("queries", [1, 70])
def test_attention_over_the_largest_numbers(queries, ress_gpu):
    """Values near the largest float come back finite from both kernels.  Codes and
    the probabilities 1/2 are exact here, so outputs differ by their rounding alone
    (half a step, 2^-8), and the keys' logits of 0 make lse = ln 2.  (The float32
    sums before the division stay below 3.4e38 as well.)"""
    x = torch.full((2, 2, 64), 2.9e38)
    x[1] = -1.0e38
    zero = torch.zeros(2, 2, 64)
    cache = ress_gpu.make_cache(1, 2, 64)
    ress_gpu.ress_cache_append(zero.cuda(), x.cuda(), _i32([0, 1]), cache)
    _ok(ress_gpu)
    q = torch.ones(queries, 2, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = ress_gpu.ress_cache_attn(q, cache, _i32([[0]]), _i32([2]), _i32([0, queries]))
    _ok(ress_gpu)
    held = (np64(cache.v) * np64(cache.v_scale)[:, :, None, None])[0, :, :2]
    assert np.isfinite(held).all()
    want = held.mean(axis=1)[None]
    assert np.isfinite(np64(out)).all()
    assert (np.abs(np64(out) - want) <= 2.0 ** -8 * np.abs(want)).all()
    assert np.abs(np64(lse) - math.log(2)).max() <= 1e-5


def test_plan_with_the_longest_slot_map(ress_gpu):
    """2^30 slots, all but the first few of no token."""
    tokens = 1 << 30
    off, slots, lengths, cursor = ress_gpu.ress_cache_plan(
        _i32([5]), _i32([3]), _i32([[7, -1]]), _i32([1]), _i32([0]), 64, tokens)
    _ok(ress_gpu)
    assert slots.shape == (tokens,) and off.tolist() == [0, 5]
    assert slots[:5].tolist() == list(range(7 * 64 + 3, 7 * 64 + 8))
    assert int(slots[5:].max()) == -1 and int(slots[5:].min()) == -1
    assert lengths.tolist() == [8] and int(cursor) == 0


@pytest.mark.parametrize("step", [0, 1])
@pytest.mark.parametrize("queries", [1, 128])
def test_the_longest_request(queries, step, ress_gpu):
    """2^31 - 64 cached tokens, which end inside a 128-key chunk: a table that names
    two pages over and over, and another page at its end.  The keys of the two are
    zero and those of the last one make logits of 32, so a row that sees none of it
    gives the mean of the values 1 and 3 (sums of whole numbers, exact in float32 for
    each CTA's share) and lse = ln of its keys, and a row that does gives the last
    page's value 7 (the others weigh 2^31 e^-32 < 3e-5 of it) and 32 + ln of the
    last page's keys it sees, both to the 3e-5 and bf16's rounding."""
    page, n = 64, 2 ** 31 - 64
    pages = n // page
    cache = ress_gpu.make_cache(3, 1, page)
    for c in (cache.k_scale, cache.v_scale):
        c.fill_(1.0)
    for i, (key, value) in enumerate(((0.0, 1.0), (0.0, 3.0), (4.0, 7.0))):
        cache.k[i], cache.v[i] = torch.tensor(key).to(FP8), torch.tensor(value).to(FP8)
    table = (torch.arange(pages, dtype=torch.int32, device="cuda") & 1)[None].contiguous()
    table[0, -1] = 2
    q = torch.ones(queries, 1, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = ress_gpu.ress_cache_attn(q, cache, table, _i32([n]), _i32([0, queries]), step=step)
    _ok(ress_gpu)
    at = np.arange(queries) - queries      # positions from the end
    seen = np.full(queries, 64) if step == 0 else np.maximum(at + 65, 0)
    for i in range(queries):
        want = 7.0 if seen[i] else 2.0
        wlse = 32 + math.log(seen[i]) if seen[i] else math.log(n + int(at[i]) + 1)
        assert (np.abs(np64(out)[i] - want) <= want * (2.0 ** -8 + 3e-5)).all(), i
        assert abs(float(lse[0, i]) - wlse) <= 3e-5 + 1e-5 * wlse, i


@pytest.mark.parametrize("queries", [1, 70])
@pytest.mark.parametrize("up", [102, 106, -100, -113])
def test_queries_of_any_magnitude(up, queries, ress_gpu):
    """Queries of magnitudes around 2^up and keys around 2^-up, so that the logits are
    of order one, with one query row of ones beside the large ones (logits of zero)."""
    g = torch.Generator().manual_seed(up + queries)
    n, heads = 150, 2
    x = torch.randn(n, 1, 64, generator=g) * 2.0 ** -up
    v = torch.randn(n, 1, 64, generator=g)
    cache = ress_gpu.make_cache(3, 1, 64)
    ress_gpu.ress_cache_append(x.cuda(), v.cuda(),
                               torch.arange(n, dtype=torch.int32, device="cuda"), cache)
    q = (torch.randn(queries, heads, 64, generator=g) * 2.0 ** up).to(torch.bfloat16)
    if up > 0:
        q[0, 1] = 1.0
    out, lse = ress_gpu.ress_cache_attn(q.cuda(), cache, _i32([[0, 1, 2]]), _i32([n]),
                                        _i32([0, queries]))
    _ok(ress_gpu)
    check_cache_attention(out, lse, cache_attention(q, cache, [[0, 1, 2]], [n], [0, queries]))


@pytest.mark.parametrize("queries", [1, 150])
@pytest.mark.parametrize("part", ["k_scale", "v_scale"])
@pytest.mark.parametrize("scale", [3.0, 2.0 ** -101, 2.0 ** 120, -1.0, math.inf, math.nan, 1e-40])
def test_pages_of_a_wrong_scale_are_flagged_and_left_out(scale, part, queries, ress_gpu):
    lengths = [300, 200]
    q, cache, table, off = make_requests(ress_gpu, lengths, [queries] * 2, 64, 4, 2, seed=23)
    args = _i32(table), _i32(lengths), _i32(off)
    for page in (table[0][2], table[1][3]):          # inside a request, and its last one
        getattr(cache, part)[page, 1] = scale
    out, lse = ress_gpu.ress_cache_attn(q.cuda(), cache, *args)
    assert ress_gpu.ress_check_device_errors() == (ress_gpu.RESS_ERR_INVALID_ARG, 96)
    for head in range(2):                            # the other key head keeps its pages
        t = [list(row) for row in table]
        if head == 1:
            t[0][2], t[1][3] = -1, -1
        one = type(cache)(*(x[:, head:head + 1].contiguous() for x in cache))
        h = slice(2 * head, 2 * head + 2)
        one.k_scale[~torch.isfinite(one.k_scale)], one.v_scale[~torch.isfinite(one.v_scale)] = 1., 1.
        ref = cache_attention(q[:, h], one, t, lengths, off)
        check_cache_attention(out[:, h], lse[h], ref)


@pytest.mark.parametrize("queries", [1, 150])
def test_scales_of_zero_and_at_the_ends_are_taken(queries, ress_gpu):
    """A page that was never written stands for zeros; 2^-100 and 2^119 are scales."""
    q, cache, table, off = make_requests(ress_gpu, [200], [queries], 64, 2, 1, seed=29)
    cache.k_scale[table[0][0]], cache.v_scale[table[0][0]] = 0.0, 0.0
    cache.k_scale[table[0][1]], cache.v_scale[table[0][1]] = 2.0 ** -100, 2.0 ** -100
    out, lse = ress_gpu.ress_cache_attn(q.cuda(), cache, _i32(table), _i32([200]), _i32(off))
    _ok(ress_gpu)
    check_cache_attention(out, lse, cache_attention(q, cache, table, [200], off))
    cache.v_scale[table[0][2]] = 2.0 ** 119
    cache.v.view(torch.uint8)[table[0][2]] &= 0x8F      # codes below 2^-5: sums stay in float32
    out, lse = ress_gpu.ress_cache_attn(q.cuda(), cache, _i32(table), _i32([200]), _i32(off))
    _ok(ress_gpu)
    check_cache_attention(out, lse, cache_attention(q, cache, table, [200], off))


def test_plans_of_many_requests_from_two_threads(ress_gpu):
    """Plans that need more shared memory than a kernel has by default, of different
    sizes, from two threads at once."""
    import threading
    sizes, failed = (8192, 4200), []
    ins = [(_i32([1] * r), _i32([0] * r), torch.full((r, 1), -1, dtype=torch.int32, device="cuda"),
            torch.arange(r, dtype=torch.int32, device="cuda"), _i32([0])) for r in sizes]
    streams = [torch.cuda.Stream() for _ in sizes]
    torch.cuda.synchronize()

    def work(i):
        try:
            for _ in range(400):
                off, slots, lengths, cursor = ress_gpu.ress_cache_plan(
                    *ins[i], 64, sizes[i], stream=streams[i])
            streams[i].synchronize()
            assert torch.equal(slots, torch.arange(sizes[i], dtype=torch.int32, device="cuda") * 64)
        except Exception as e:   # (a thread's exception would pass unseen)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    _ok(ress_gpu)
    assert not failed, failed
