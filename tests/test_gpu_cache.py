"""The paged 8-bit cache on the GPU: block tables and slot maps, the writer,
and attention over the pages, against plain implementations (whole numbers in
Python, values in float64).

Tolerances, derived before the first run.  Codes and scales are exact: a scale
is a power of two, so x / s is exact and its rounding to e4m3 is the only one.
Attention: a probability enters P V rounded to bf16 (half a step, 2^-9 below a
power of two, at most 2^-8 relative) while the normaliser is not rounded, so
|out - ref| <= 2^-8 * sum_t p_t |v_t| <= 2^-8 * max|v| from P, plus the output's
own rounding 2^-8 |out|, plus float32 noise: 2^-7 * max|v| in all.  lse is a
float32 sum: the logits are float32 sums of 64 exact products (|error| <= 64 *
2^-24 * sum |q k| / 8, below 2^-14 for |logit sums| <= 64) and ex2 and lg2 are
good to 2^-20, so 1e-4 + 1e-5 |lse| covers it."""

import math

import numpy as np
import pytest
import torch

from tests.parity import np64, poison

pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn


def _i32(v, device="cuda"):
    return torch.tensor(v, dtype=torch.int32, device=device)


def _offsets(v):
    return _i32(np.concatenate([[0], np.cumsum(v)]).astype(np.int64).tolist())


def _ok(ress):
    status, detail = ress.ress_check_device_errors()
    assert status == 0, (status, detail)


# ------------------------------------------------------------------------------------------
# plan
# ------------------------------------------------------------------------------------------
def plan_ref(added, lengths, table, free, cursor, page, tokens, width):
    """The rules of ress_cache_plan in Python; returns also the details flagged."""
    table = [list(r) for r in table]
    offsets, slots, new_len, flags = [0], [-1] * tokens, [], set()
    first = tok = taken = 0
    for r, (a, n) in enumerate(zip(added, lengths)):
        row_ok = a >= 0 and n >= 0 and n + a <= width * page
        a0 = max(a, 0)
        need = -(-(n + a) // page) - -(-n // page) if row_ok else 0
        tok_ok = tok + a0 <= tokens
        list_ok = need == 0 or cursor + first + need <= len(free)
        if row_ok and tok_ok and list_ok:
            base = -(-n // page)
            for i in range(need):
                table[r][base + i] = free[cursor + first + i]
            for i in range(a):
                pos = n + i
                slots[tok + i] = table[r][pos // page] * page + pos % page
            new_len.append(n + a)
            if need:
                taken = first + need
        else:
            flags.add(100 if not row_ok else 102 if not tok_ok else 101)
            new_len.append(n)
        first += need
        tok += a0
        offsets.append(tok)
    return table, offsets, slots, new_len, cursor + taken, flags


def run_plan(ress, added, lengths, table, free, cursor, page, tokens, **kw):
    t = _i32(table)
    got = ress.ress_cache_plan(_i32(added), _i32(lengths), t, _i32(free), _i32([cursor]), page,
                               tokens, offsets=poison((len(added) + 1,), torch.int32),
                               slots=torch.full((tokens,), -7, dtype=torch.int32, device="cuda"),
                               new_lengths=poison((len(added),), torch.int32),
                               new_cursor=poison((1,), torch.int32), **kw)
    return [t.tolist()] + [x.tolist() for x in got]


def _plan_case(rng, requests, page, width, most, add):
    lengths = [int(rng.integers(0, most + 1)) for _ in range(requests)]
    added = [int(rng.integers(0, add + 1)) for _ in range(requests)]
    ids = rng.permutation(requests * width + 50).tolist()
    table = [[-1] * width for _ in range(requests)]
    for r, n in enumerate(lengths):
        for j in range(min(width, -(-n // page))):
            table[r][j] = ids.pop()
    return added, lengths, table, ids


@pytest.mark.parametrize("requests,page,most,add,slack", [
    (1, 64, 0, 1, 0), (1, 64, 64, 64, 3), (7, 64, 200, 130, 0), (33, 128, 300, 1, 5),
    (600, 64, 500, 70, 11), (1100, 128, 100, 300, 0)])
def test_plan_matches_the_rules(requests, page, most, add, slack, ress_gpu):
    rng = np.random.default_rng(requests * page + add)
    width = -(-(most + add) // page) + 1
    added, lengths, table, free = _plan_case(rng, requests, page, width, most, add)
    tokens = sum(added) + slack
    ref = plan_ref(added, lengths, table, free, 3, page, tokens, width)
    got = run_plan(ress_gpu, added, lengths, table, free, 3, page, tokens)
    _ok(ress_gpu)
    assert not ref[5]
    assert got[0] == ref[0] and got[1] == ref[1] and got[2] == ref[2] and got[3] == ref[3]
    assert got[4] == [ref[4]]


def test_plan_of_the_largest_number_of_requests(ress_gpu):
    rng = np.random.default_rng(5)
    added, lengths, table, free = _plan_case(rng, 8192, 64, 3, 100, 60)
    tokens = sum(added)
    ref = plan_ref(added, lengths, table, free, 0, 64, tokens, 3)
    got = run_plan(ress_gpu, added, lengths, table, free, 0, 64, tokens)
    _ok(ress_gpu)
    assert got[:4] == list(ref[:4]) and got[4] == [ref[4]]


@pytest.mark.parametrize("what", ["row", "negative", "list", "slots", "cursor", "huge"])
def test_plan_leaves_a_request_that_does_not_fit(what, ress_gpu):
    page, width = 64, 3
    rng = np.random.default_rng(11)
    added, lengths, table, free = _plan_case(rng, 9, page, width, 60, 100)
    added[4] = 70
    tokens, cursor, detail = sum(added), 2, 0
    if what == "row":
        added[4], detail = 200, 100
        tokens = sum(added)
    elif what == "negative":
        lengths[4], detail = -1, 100
    elif what == "huge":
        added[4], added[5], detail = 2 ** 31 - 1, 2 ** 31 - 1, 100
    elif what == "list":
        need = [-(-(n + a) // page) - -(-n // page) for a, n in zip(added, lengths)]
        free, detail = free[:cursor + sum(need[:4])], 101
    elif what == "cursor":
        cursor, detail = len(free) + 1, 101
    else:
        tokens, detail = sum(added[:4]) + 69, 102
    ref = plan_ref(added, lengths, table, free, cursor, page, tokens, width)
    got = run_plan(ress_gpu, added, lengths, table, free, cursor, page, tokens)
    status, seen = ress_gpu.ress_check_device_errors()
    assert status == ress_gpu.RESS_ERR_BAD_INDEX and detail in ref[5] and seen in ref[5]
    assert got[0] == ref[0] and got[2] == ref[2] and got[3] == ref[3] and got[4] == [ref[4]]
    assert got[1] == [min(x, 2 ** 31 - 1) for x in ref[1]]


def test_plan_flags_a_page_outside_the_pool(ress_gpu):
    table = [[5, -1], [9, -1]]
    got = run_plan(ress_gpu, [1, 64], [3, 1], table, [7, 100], 0, 64, 65, pages=10)
    status, detail = ress_gpu.ress_check_device_errors()
    assert status == ress_gpu.RESS_ERR_BAD_INDEX and detail == 103 or status == 0
    assert got[2][0] == 5 * 64 + 3 and got[2][1] == 9 * 64 + 1 and got[2][63] == 9 * 64 + 63
    assert got[2][64] == 7 * 64
    got = run_plan(ress_gpu, [1, 64], [3, 1], [[5, -1], [9, -1]], [100], 0, 64, 65, pages=10)
    status, detail = ress_gpu.ress_check_device_errors()
    assert status == ress_gpu.RESS_ERR_BAD_INDEX and detail == 103
    assert got[2][64] == -1 and got[2][:64] == [5 * 64 + 3] + list(range(9 * 64 + 1, 10 * 64))


# ------------------------------------------------------------------------------------------
# append
# ------------------------------------------------------------------------------------------
def to_e4m3(y):
    e = np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -60)))
    grid = 2.0 ** (np.maximum(e, -6) - 3)
    return np.clip(np.round(y / grid) * grid, -448, 448)


def scale_ref(amax):
    s = 2.0 ** -100
    while amax > 448 * s:
        s *= 2
    return s


def append_ref(x, slots, codes, scale, page):
    """The rules of ress_cache_append in float64 on numpy copies."""
    codes, scale = codes.copy(), scale.copy()
    i = 0
    while i < len(slots):
        if slots[i] < 0:
            i += 1
            continue
        j = i + 1
        while j < len(slots) and slots[j] == slots[j - 1] + 1 and slots[j] % page:
            j += 1
        p, c = slots[i] // page, slots[i] % page
        for h in range(x.shape[1]):
            s = scale_ref(np.abs(x[i:j, h]).max())
            if c:
                s = max(s, scale[p, h])
                codes[p, h, :c] = to_e4m3(codes[p, h, :c] * (scale[p, h] / s))
            codes[p, h, c:c + j - i] = to_e4m3(x[i:j, h] / s)
            scale[p, h] = s
        i = j
    return codes, scale


def _filled_cache(ress, pages, heads, page, seed, scale_exp=None):
    """A pool of random codes and scales (no NaN codes)."""
    g = torch.Generator().manual_seed(seed)
    cache = ress.make_cache(pages, heads, page)
    for codes, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        codes.copy_((torch.randn(codes.shape, generator=g) * 100).clamp(-448, 448).to(FP8))
        e = torch.randint(-9, -5, scale.shape, generator=g) if scale_exp is None else \
            torch.full(scale.shape, scale_exp)
        scale.copy_(torch.exp2(e.float()))
    return cache


def _slots_of(starts, counts, page, ids):
    """Slots of runs: request r continues at position starts[r] with its own pages."""
    out = []
    for s, n in zip(starts, counts):
        own = {}
        for pos in range(s, s + n):
            if pos // page not in own:
                own[pos // page] = ids.pop()
            out.append(own[pos // page] * page + pos % page)
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page,heads,starts,counts", [
    (64, 1, [0], [1]), (64, 2, [0, 1, 63, 64, 65], [64, 1, 1, 1, 63]),
    (128, 3, [0, 127, 5, 64], [200, 2, 130, 64]), (64, 5, [3] * 40, [1] * 40),
    (64, 16, [0, 7, 30], [1374, 700, 64]), (128, 2, [10], [2000])])
def test_append_is_exact(page, heads, starts, counts, dtype, ress_gpu):
    rng = np.random.default_rng(sum(counts) + heads)
    pages = sum(-(-(s % page + n) // page) for s, n in zip(starts, counts)) + 2
    cache = _filled_cache(ress_gpu, pages, heads, page, seed=page + heads)
    ids = rng.permutation(pages).tolist()
    slots = _slots_of([s % page for s in starts], counts, page, ids)
    g = torch.Generator().manual_seed(1)
    x = [(torch.randn(len(slots), heads, 64, generator=g)
          * torch.exp2(torch.randint(-3, 6, (len(slots), heads, 1), generator=g).float())).to(dtype)
         for _ in range(2)]
    ref = [append_ref(np64(t), slots, np64(c), np64(s), page)
           for t, c, s in ((x[0], cache.k, cache.k_scale), (x[1], cache.v, cache.v_scale))]
    ress_gpu.ress_cache_append(x[0].cuda(), x[1].cuda(), _i32(slots), cache)
    _ok(ress_gpu)
    for (codes, scale), c, s in ((ref[0], cache.k, cache.k_scale), (ref[1], cache.v, cache.v_scale)):
        assert np.array_equal(np64(s), scale)
        assert np.array_equal(np64(c), codes)


def test_append_at_the_edges_of_its_number_range(ress_gpu):
    """Zeros, values below the smallest scale, exact multiples of 448, the
    smallest code, a page whose scale grows by more than e4m3 can hold, and
    NaN and infinity, which are flagged and stay in their own cells."""
    page, heads = 64, 4
    rows = torch.zeros(6, heads, 64)
    rows[0, 1] = 448.0
    rows[1, 1] = 449.0
    rows[0, 2] = 2.0 ** -120
    rows[1, 2] = -2.0 ** -108
    rows[0, 3] = 2.0 ** 100
    for i, slots in enumerate(([0, 1, 2, 3, 4, 5], [64, 65, 66, 67, 68, 69], [70, 71, 72, 73, 74, 75])):
        cache = _filled_cache(ress_gpu, 2, heads, page, seed=3, scale_exp=-8)
        x = rows * (2.0 ** -i)
        ref = append_ref(np64(x), slots, np64(cache.k), np64(cache.k_scale), page)
        ress_gpu.ress_cache_append(x.cuda(), x.cuda(), _i32(slots), cache)
        _ok(ress_gpu)
        assert np.array_equal(np64(cache.k_scale), ref[1]) and np.array_equal(np64(cache.k), ref[0])
    cache = _filled_cache(ress_gpu, 1, 1, page, seed=4)
    x = torch.ones(2, 1, 64)
    x[0, 0, 5], x[1, 0, 7] = float("nan"), float("nan")
    x[1, 0, 9] = float("-inf")
    ress_gpu.ress_cache_append(x.cuda(), x.cuda(), _i32([0, 1]), cache)
    status, detail = ress_gpu.ress_check_device_errors()
    assert status == ress_gpu.RESS_ERR_INVALID_ARG and detail == 105
    scale = np64(cache.k_scale)[0, 0]
    assert scale == 2.0 ** -8                    # of the ones among them
    got, want = np64(cache.k)[0, 0, :2] * scale, np64(x)[:, 0]
    assert np.array_equal(np.isnan(got), np.isnan(want))
    want[1, 9] = -448 * scale
    assert np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])


def test_append_skips_and_flags(ress_gpu):
    """Negative slots are skipped, slots behind the pool flagged, every other
    cell and scale is left as it was."""
    cache = _filled_cache(ress_gpu, 3, 2, 64, seed=8)
    before = [t.clone() for t in cache]
    slots = [-1, 64, 65, -1, 66, 192, 193, 2 ** 31 - 1, -5]
    x = torch.randn(len(slots), 2, 64, generator=torch.Generator().manual_seed(2))
    ress_gpu.ress_cache_append(x.cuda(), x.cuda(), _i32(slots), cache)
    status, detail = ress_gpu.ress_check_device_errors()
    assert status == ress_gpu.RESS_ERR_BAD_INDEX and detail == 104
    for page in (0, 2):
        for a, b in zip(cache, before):
            assert torch.equal(a[page].view(torch.uint8 if a.dtype == FP8 else a.dtype),
                               b[page].view(torch.uint8 if b.dtype == FP8 else b.dtype))
    assert torch.equal(cache.k[1, :, 3:].view(torch.uint8), before[0][1, :, 3:].view(torch.uint8))


def test_append_reads_slices_of_fused_rows(ress_gpu):
    g = torch.Generator().manual_seed(6)
    kv = torch.randn(150, 2, 3, 64, generator=g).to(torch.bfloat16).cuda()
    slots = _i32(list(range(150)))
    a, b = ress_gpu.make_cache(3, 3, 64), ress_gpu.make_cache(3, 3, 64)
    ress_gpu.ress_cache_append(kv[:, 0], kv[:, 1], slots, a)
    ress_gpu.ress_cache_append(kv[:, 0].contiguous(), kv[:, 1].contiguous(), slots, b)
    _ok(ress_gpu)
    for x, y in zip(a, b):
        assert torch.equal(x.float(), y.float())


# ------------------------------------------------------------------------------------------
# attention over the cache
# ------------------------------------------------------------------------------------------
def attn_ref(q, cache, table, lengths, offsets, step, page):
    qn = np64(q)
    vals = [np64(c) * np64(s)[:, :, None, None] for c, s in ((cache.k, cache.k_scale),
                                                           (cache.v, cache.v_scale))]
    t_all, h = qn.shape[:2]
    hk = vals[0].shape[1]
    out = np.zeros(qn.shape)
    lse = np.full((h, t_all), -np.inf)
    for r, n in enumerate(lengths):
        rows = range(offsets[r], offsets[r + 1])
        m = len(rows)
        ids = table[r][:-(-n // page)]
        keep = np.repeat(np.array([0 <= i < vals[0].shape[0] for i in ids], dtype=bool), page)[:n]
        k, v = (np.concatenate([x[i if 0 <= i < x.shape[0] else 0] for i in ids] or
                               [np.zeros((hk, 0, 64))], axis=1)[:, :n] for x in vals)
        for i, row in enumerate(rows):
            pos = n - m + i
            end = n if step == 0 else min(n, (pos // step + 1) * step) if pos >= 0 else 0
            ok = keep & (np.arange(n) < end)
            if not ok.any():
                continue
            for a in range(h):
                s = k[a // (h // hk)][ok] @ qn[row, a] / 8.0
                top = s.max()
                p = np.exp(s - top)
                lse[a, row] = top + math.log(p.sum())
                out[row, a] = p @ v[a // (h // hk)][ok] / p.sum()
    return out, lse, max(1e-30, np.abs(vals[1][np.isfinite(vals[1])]).max(initial=0.0))


def check_attn(out, lse, ref):
    ro, rl, top = ref
    o, l = np64(out), np64(lse)
    assert np.isfinite(o).all()
    assert np.abs(o - ro).max() <= 2.0 ** -7 * top, np.abs(o - ro).max() / top
    dead = np.isinf(rl)
    assert np.array_equal(np.isinf(l), dead) and (l[dead] < 0).all()
    err = np.abs(l[~dead] - rl[~dead])
    assert (err <= 1e-4 + 1e-5 * np.abs(rl[~dead])).all(), err.max()


def make_requests(ress, lengths, queries, page, heads, kv_heads, seed, spread=0):
    """A cache whose pages hold random tokens; cells behind a request's last
    token hold NaN codes."""
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lengths]
    width = max(max(need), 1) + 1
    pool = sum(need) + 2
    ids = rng.permutation(pool).tolist()
    table = [[ids.pop() for _ in range(m)] + [-3] * (width - m) for m in need]
    cache = ress.make_cache(pool, kv_heads, page)
    slots = [table[r][pos // page] * page + pos % page for r, n in enumerate(lengths)
             for pos in range(n)]
    x = [torch.randn(len(slots), kv_heads, 64, generator=g) for _ in range(2)]
    if spread:
        x = [t * torch.exp2(torch.randint(-spread, spread + 1, (len(slots), 1, 1),
                                          generator=g).float()) for t in x]
    for c in (cache.k, cache.v):
        c.view(torch.uint8).fill_(0x7F)
    for c in (cache.k_scale, cache.v_scale):
        c.fill_(1.0)
    if slots:
        ress.ress_cache_append(x[0].to(torch.bfloat16).cuda(), x[1].to(torch.bfloat16).cuda(),
                               _i32(slots), cache)
    q = torch.randn(sum(queries), heads, 64, generator=g).to(torch.bfloat16)
    return q, cache, table, np.concatenate([[0], np.cumsum(queries)]).tolist()


CASES = [
    # lengths, queries, page, heads, kv heads, step
    ([1], [1], 64, 1, 1, 0),
    ([0], [1], 64, 2, 1, 0),
    ([63, 64, 65, 1, 0, 128], [1] * 6, 64, 4, 4, 0),
    ([1500, 127, 129], [1, 1, 1], 128, 16, 2, 0),
    ([700, 3], [1, 0], 64, 6, 2, 1),
    ([900, 200, 64], [5, 3, 64], 64, 16, 16, 0),
    ([300, 77], [17, 77], 64, 8, 1, 1),
    ([300, 90], [33, 90], 128, 12, 4, 7),
    ([400, 30], [129, 31], 64, 4, 4, 1),       # more queries than tokens: rows before position 0
    ([1374 + 600], [600], 64, 4, 2, 1374),
    ([2000], [260], 128, 3, 3, 0),
    ([513, 1025], [300, 255], 64, 64, 8, 100),
]


@pytest.mark.parametrize("lengths,queries,page,heads,kv_heads,step", CASES)
def test_cache_attention(lengths, queries, page, heads, kv_heads, step, ress_gpu):
    q, cache, table, off = make_requests(ress_gpu, lengths, queries, page, heads, kv_heads,
                                         seed=sum(lengths) + heads)
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((heads, q.shape[0]), 7.0, device="cuda")
    ress_gpu.ress_cache_attn(q.cuda(), cache, _i32(table), _i32(lengths), _i32(off), step=step,
                             out=out, lse=lse)
    _ok(ress_gpu)
    check_attn(out, lse, attn_ref(q, cache, table, lengths, off, step, page))
    again, lse2 = ress_gpu.ress_cache_attn(q.cuda(), cache, _i32(table), _i32(lengths), _i32(off),
                                           step=step)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("queries", [1, 200])
def test_pages_whose_scales_lie_far_apart(queries, ress_gpu):
    """Page scales that differ by 2^40 and more: large values sit in pages of
    their own and dominate or vanish by their logits alone."""
    q, cache, table, off = make_requests(ress_gpu, [640], [queries], 64, 2, 1, seed=3)
    cache.v_scale.copy_(torch.exp2(torch.arange(cache.v_scale.numel()).float() * 6 - 40).view(
        cache.v_scale.shape))
    cache.k_scale.copy_(torch.exp2(-torch.arange(cache.k_scale.numel()).float() - 6).view(
        cache.k_scale.shape))
    out, lse = ress_gpu.ress_cache_attn(q.cuda(), cache, _i32(table), _i32([640]), _i32(off))
    _ok(ress_gpu)
    check_attn(out, lse, attn_ref(q, cache, table, [640], off, 0, 64))


@pytest.mark.parametrize("queries", [1, 150])
def test_bad_pages_lengths_and_offsets_are_flagged(queries, ress_gpu):
    lengths = [300, 200]
    q, cache, table, off = make_requests(ress_gpu, lengths, [queries] * 2, 64, 4, 2, seed=21)
    bad = [list(r) for r in table]
    bad[0][2] = 10 ** 6
    bad[1][0] = -1
    out, lse = ress_gpu.ress_cache_attn(q.cuda(), cache, _i32(bad), _i32(lengths), _i32(off))
    status, detail = ress_gpu.ress_check_device_errors()
    assert status == ress_gpu.RESS_ERR_BAD_INDEX and detail == 95
    check_attn(out, lse, attn_ref(q, cache, bad, lengths, off, 0, 64))
    # a negative length is taken as zero, one beyond the row as the row
    out, lse = ress_gpu.ress_cache_attn(q.cuda(), cache, _i32(table), _i32([-5, 200]), _i32(off))
    status, detail = ress_gpu.ress_check_device_errors()
    assert status == ress_gpu.RESS_ERR_BAD_INDEX and detail == 94
    assert (out[:queries] == 0).all() and torch.isinf(lse[:, :queries]).all()
    # offsets that descend make an empty request: its rows are not written
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    ress_gpu.ress_cache_attn(q.cuda(), cache, _i32(table), _i32(lengths),
                             _i32([queries, 0, queries]), out=out)
    status, detail = ress_gpu.ress_check_device_errors()
    assert status == ress_gpu.RESS_ERR_BAD_INDEX and detail == 90
    assert (out[queries:] == 7.0).all()


def test_rows_of_no_request_are_left_as_they_were(ress_gpu):
    lengths = [100, 200]
    q, cache, table, _ = make_requests(ress_gpu, lengths, [3, 2], 64, 2, 2, seed=31)
    big = torch.zeros(12, 2, 64, dtype=torch.bfloat16)
    big[4:9] = q
    out = torch.full(big.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((2, 12), 7.0, device="cuda")
    ress_gpu.ress_cache_attn(big.cuda(), cache, _i32(table), _i32(lengths), _i32([4, 7, 9]),
                             out=out, lse=lse)
    _ok(ress_gpu)
    ref = attn_ref(q, cache, table, lengths, [0, 3, 5], 0, 64)
    check_attn(out[4:9], lse[:, 4:9], ref)
    assert (out[:4] == 7).all() and (out[9:] == 7).all()
    assert (lse[:, :4] == 7).all() and (lse[:, 9:] == 7).all()


@pytest.mark.parametrize("queries", [1, 150])
def test_a_nan_query_comes_out(queries, ress_gpu):
    q, cache, table, off = make_requests(ress_gpu, [300, 90], [queries] * 2, 64, 4, 2, seed=41)
    args = cache, _i32(table), _i32([300, 90]), _i32(off)
    want, wlse = ress_gpu.ress_cache_attn(q.cuda(), *args)
    q[queries, 3, 17] = float("nan")
    out, lse = ress_gpu.ress_cache_attn(q.cuda(), *args)
    _ok(ress_gpu)
    assert out[queries, 3].isnan().all() and lse[3, queries].isnan()
    out[queries, 3], lse[3, queries] = want[queries, 3], wlse[3, queries]
    assert torch.equal(out, want) and torch.equal(lse, wlse)


@pytest.mark.parametrize("queries", [1, 200])
def test_pools_beyond_4_gb(queries, ress_gpu):
    """Pages whose byte offsets pass 2^32: the same tokens in the last pages of a
    large pool and in a small one."""
    pages, heads = 70000, 16                           # 4.6 GB of codes each
    big, small = ress_gpu.make_cache(pages, heads, 64), ress_gpu.make_cache(8, heads, 64)
    x = torch.randn(200, 2, heads, 64, generator=torch.Generator().manual_seed(2)).to(
        torch.bfloat16).cuda()
    ids = torch.tensor([[pages - 1, pages - 3, 5, pages - 2], [0, 1, 2, 3]])
    q = torch.randn(queries, heads, 64, generator=torch.Generator().manual_seed(3)).to(
        torch.bfloat16).cuda()
    got = []
    for cache, row in ((big, ids[0]), (small, ids[1])):
        t = torch.arange(200)
        ress_gpu.ress_cache_append(x[:, 0], x[:, 1], _i32((row[t // 64] * 64 + t % 64).tolist()),
                                   cache)
        got.append(ress_gpu.ress_cache_attn(q, cache, _i32([row.tolist()]), _i32([200]),
                                            _i32([0, queries])))
    _ok(ress_gpu)
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    for a, b in zip(big, small):
        assert torch.equal(a[ids[0].cuda()].float(), b[:4].float())


def test_threads_that_share_a_stream(ress_gpu):
    """Calls from several threads on one stream: each has its own workspace."""
    import threading
    data = [make_requests(ress_gpu, [3000, 500], [n] * 2, 64, 8, 4, seed=50 + n) for n in (1, 90)]
    dev = [(q.cuda(), c, _i32(t), _i32([3000, 500]), _i32(o)) for q, c, t, o in data]
    want = [ress_gpu.ress_cache_attn(*a) for a in dev]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        for _ in range(20):
            got[i].append(ress_gpu.ress_cache_attn(*dev[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    _ok(ress_gpu)
    for i in (0, 1):
        assert len(got[i]) == 20
        for o, l in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])


# ------------------------------------------------------------------------------------------
# the three together
# ------------------------------------------------------------------------------------------
def test_streaming_views_end_to_end(ress_gpu):
    """Scenes that grow view by view and then token by token: plan, append and
    attend, each step from the outputs of the last; the attention is checked
    against float64 over the codes that the cache stands for, and those
    against the tokens themselves (e4m3: half a step is 2^-4 relative, plus
    half the smallest code of the scale)."""
    page, heads, kv_heads, r = 64, 8, 4, 3
    g = torch.Generator().manual_seed(77)
    pool = 40
    cache = ress_gpu.make_cache(pool, kv_heads, page)
    free = torch.randperm(pool, generator=g).to(torch.int32).cuda()
    table = torch.full((r, 12), -1, dtype=torch.int32, device="cuda")
    lengths, cursor = _i32([0] * r), _i32([0])
    held = [[torch.zeros(0, kv_heads, 64)] for _ in range(r)]
    for added in ([100, 0, 37], [28, 65, 1], [1, 1, 1], [1, 200, 1], [1, 1, 1]):
        n = sum(added)
        off, slots, lengths, cursor = ress_gpu.ress_cache_plan(
            _i32(added), lengths, table, free, cursor, page, n, pages=pool)
        kv = torch.randn(n, 2, kv_heads, 64, generator=g).to(torch.bfloat16)
        at = 0
        for i, a in enumerate(added):
            held[i].append(kv[at:at + a, 0].float())
            at += a
        dev = kv.cuda()
        ress_gpu.ress_cache_append(dev[:, 0], dev[:, 1], slots, cache)
        q = torch.randn(n, heads, 64, generator=g).to(torch.bfloat16)
        for step in (0, 1):
            out, lse = ress_gpu.ress_cache_attn(q.cuda(), cache, table, lengths, off, step=step)
            _ok(ress_gpu)
            check_attn(out, lse, attn_ref(q, cache, table.tolist(), lengths.tolist(),
                                          off.tolist(), step, page))
    assert lengths.tolist() == [131, 267, 41] and int(cursor) == 3 + 5 + 1
    for i in range(r):
        want = torch.cat(held[i]).numpy()
        ids = table[i, :-(-want.shape[0] // page)].tolist()
        s = np64(cache.k_scale)[ids]
        got = (np64(cache.k)[ids] * s[:, :, None, None]).transpose(0, 2, 1, 3).reshape(-1, kv_heads, 64)
        unit = np.repeat(s, page, axis=0)[:want.shape[0], :, None]
        err = np.abs(got[:want.shape[0]] - want)
        assert (err <= 2.0 ** -4 * np.abs(want) + unit * 2.0 ** -10).all()


def test_a_captured_step_replays_on_new_contents(ress_gpu):
    """plan, append and attention captured into one graph: replays read what
    the buffers hold then, and a second graph with a workspace of its own does
    not disturb the first."""
    page, heads, kv_heads, r, pool = 64, 4, 2, 2, 16
    g = torch.Generator().manual_seed(5)
    cache = ress_gpu.make_cache(pool, kv_heads, page)
    free = torch.arange(pool, dtype=torch.int32, device="cuda")
    table = torch.full((r, 6), -1, dtype=torch.int32, device="cuda")
    added, lengths, cursor = _i32([60, 3]), _i32([0, 0]), _i32([0])
    kv = torch.randn(63, 2, kv_heads, 64, generator=g).to(torch.bfloat16).cuda()
    q = torch.randn(63, heads, 64, generator=g).to(torch.bfloat16).cuda()

    def step():
        off, slots, nl, nc = ress_gpu.ress_cache_plan(added, lengths, table, free, cursor, page, 63)
        ress_gpu.ress_cache_append(kv[:, 0], kv[:, 1], slots, cache)
        out, lse = ress_gpu.ress_cache_attn(q, cache, table, nl, off)
        lengths.copy_(nl)
        cursor.copy_(nc)
        return off, out, lse

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        off, out, lse = step()
    for new in ([1, 2], [4, 0], [30, 33]):
        added.copy_(_i32(new))
        kv.copy_(torch.randn(kv.shape, generator=g).to(torch.bfloat16))
        graph.replay()
        _ok(ress_gpu)
        n = sum(new)
        o = off.tolist()
        assert o == [0, new[0], n]
        check_attn(out[:n], lse[:, :n], attn_ref(q[:n].cpu(), cache, table.tolist(),
                                                 lengths.tolist(), o, 0, page))
    assert lengths.tolist() == [60 + 35, 3 + 35]


@pytest.mark.parametrize("queries", [1, 140])
def test_calls_on_another_stream_and_two_at_once(queries, ress_gpu):
    """The stream argument, with outputs and workspace made by the call."""
    args = [make_requests(ress_gpu, [3000, 500], [queries] * 2, 64, 8, 4, seed=s) for s in (1, 2)]
    want = [ress_gpu.ress_cache_attn(q.cuda(), c, _i32(t), _i32([3000, 500]), _i32(o))
            for q, c, t, o in args]
    dev = [(q.cuda(), c, _i32(t), _i32([3000, 500]), _i32(o)) for q, c, t, o in args]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for a, s in zip(dev, streams):
            got.append(ress_gpu.ress_cache_attn(*a, stream=s))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])
    _ok(ress_gpu)


@pytest.mark.parametrize("new", [1, 150])
@pytest.mark.parametrize("own_stream", [False, True])
def test_calls_in_a_row_wait_for_one_another(new, own_stream, ress_gpu):
    """Kernels start while the one before them ends.  Chains of calls, each on the
    outputs of the last, with buffers that are written over behind the calls that
    read them: queued behind a busy GPU they give the very bits that they give
    with a wait after each call."""
    page, heads, kv_heads, r, pool, steps = 64, 4, 2, 2, 40, 8
    g = torch.Generator().manual_seed(3)
    free = torch.randperm(pool, generator=g).to(torch.int32).cuda()
    first = torch.randn(r * new, 2 * heads, 64, generator=g).to(torch.bfloat16).cuda()
    noise = torch.randn(steps, r * new, heads, 64, generator=g).to(torch.bfloat16).cuda()
    added, total = _i32([new] * r), r * new

    def chain(wait):
        pause = torch.cuda.synchronize if wait else lambda: None
        cache = ress_gpu.make_cache(pool, kv_heads, page)
        table = torch.full((r, 20), -1, dtype=torch.int32, device="cuda")
        lengths, cursor = _i32([0] * r), _i32([0])
        x, got = first.clone(), []
        pause()
        if not wait:
            torch.cuda._sleep(20_000_000)
        for s in range(steps):
            off, slots, new_len, new_cur = ress_gpu.ress_cache_plan(
                added, lengths, table, free, cursor, page, total, pages=pool)
            pause()
            lengths.copy_(new_len)
            cursor.copy_(new_cur)
            q, k, v = x[:, :heads], x[:, heads:heads + kv_heads], x[:, heads + kv_heads:]
            ress_gpu.ress_cache_append(k, v, slots, cache)
            pause()
            out, lse = ress_gpu.ress_cache_attn(q, cache, table, new_len, off)
            pause()
            two, lse2 = ress_gpu.ress_cross_attn(out, k, v, off, off)
            pause()
            grads = ress_gpu.ress_cross_attn_bwd(out, k, v, two, lse2, out, off, off)
            pause()
            x[:, :heads] = two + noise[s]
            x[:, heads:heads + kv_heads] = grads[1].clamp(-4, 4)   # unbounded, the chain
            x[:, heads + kv_heads:] = grads[2].clamp(-4, 4)        # itself grows to infinity
            got += [off, slots, new_len, out.clone(), lse, two, lse2, *grads]
            out.zero_()
            pause()
        return got + list(cache) + [table]

    stream = torch.cuda.Stream() if own_stream else torch.cuda.current_stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        want = chain(True)
        runs = [chain(False) for _ in range(3)]
        torch.cuda.synchronize()
    _ok(ress_gpu)
    for got in runs:
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
