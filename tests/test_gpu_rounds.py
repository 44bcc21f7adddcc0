"""Items cut into pieces that take two rounds of the workers, where a worker leaves two
partial results and the joining kernel finds the second ones: forward, both walks of
the gradients, one sequence (planned on the host) and equal ones (on the device).

The plan's arithmetic stands here once more, and every case is checked to be cut and
to take two rounds, so that a change of the choices cannot leave the path untested.

Bounds as in test_gpu_cross.py: P enters its products rounded to bf16 (2^-8 + 2^-12
with exponentials and sums), dS as well, out is rounded (2^-8), and the magnitudes N
that cancel in dS leave 2^-13 of themselves."""

import pytest
import torch

GRID, CHUNK, MIN_SHARE = 148, 128, 512


def up(a, b):
    return -(-a // b)


def rounds_of(rows, cols, heads, tile_rows, mult, item_cost, seqs=1):
    """(pieces per item, rounds) of equal items, or None where the work stands on a line."""
    chunks, items = up(cols, CHUNK) * mult, up(rows, tile_rows) * heads * seqs
    fixed, units = up(item_cost, CHUNK), items * (item_cost + up(cols, CHUNK) * mult * CHUNK)
    tries = []
    for i in range(32):
        ns = max(1, min(i + 1 if i < 30 else (i - 29) * GRID // items, chunks))
        rounds = up(items * ns, GRID)
        if ns == 1 or rounds <= 2:
            tries.append((rounds * (fixed + up(chunks, ns)), ns, rounds))
    t, ns, rounds = min(tries)
    share = max(up(units, GRID), MIN_SHARE)
    return (ns, rounds) if t * CHUNK <= share + (share >> 4) + item_cost else None


def forward_plan(nq, nk, heads, kv_heads, seqs):
    group = heads // kv_heads
    rows = nq * group
    pair = up(rows, 256) * 2 * 100 <= up(rows, 128) * 118
    return rounds_of(nq, nk, kv_heads, 128 // group * (2 if pair else 1), 1, 256, seqs)


FORWARD = [  # query rows and keys of a sequence, heads, key heads, sequences
    (512, 20000, 48, 48, 1), (320, 4100, 32, 32, 1), (320, 4100, 16, 16, 2),
    (200, 4100, 32, 8, 3), (512, 9000, 24, 24, 2)]
QUERY_WALK = [(256, 20000, 48, 48, 1), (190, 20000, 64, 16, 1), (130, 20000, 24, 8, 3)]
KEY_WALK = [(20000, 256, 48, 48, 1), (3000, 700, 64, 16, 1), (4100, 130, 48, 16, 3)]


@pytest.mark.parametrize("case", FORWARD)
def test_forward_cases_take_two_rounds(case):
    plan = forward_plan(*case)
    assert plan and plan[0] > 1 and plan[1] == 2


@pytest.mark.parametrize("nq,nk,heads,kv_heads,seqs", QUERY_WALK)
def test_query_walks_take_two_rounds(nq, nk, heads, kv_heads, seqs):
    plan = rounds_of(nq, nk, kv_heads, 128 // (heads // kv_heads), 1, 5 * CHUNK, seqs)
    assert plan and plan[0] > 1 and plan[1] == 2


@pytest.mark.parametrize("nq,nk,heads,kv_heads,seqs", KEY_WALK)
def test_key_walks_take_two_rounds(nq, nk, heads, kv_heads, seqs):
    plan = rounds_of(nk, nq, kv_heads, 128, heads // kv_heads, 5 * CHUNK, seqs)
    assert plan and plan[0] > 1 and plan[1] == 2


def _make(nq, nk, heads, kv_heads, seqs, seed):
    g = torch.Generator().manual_seed(seed)
    q, do = (torch.randn(nq * seqs, heads, 64, generator=g).to(torch.bfloat16).cuda()
             for _ in range(2))
    k, v = (torch.randn(nk * seqs, kv_heads, 64, generator=g).to(torch.bfloat16).cuda()
            for _ in range(2))
    off = {} if seqs == 1 else {
        name: torch.arange(0, n * seqs + 1, n, dtype=torch.int32, device="cuda")
        for name, n in (("q_offsets", nq), ("kv_offsets", nk))}
    return q, k, v, do, off


def _within(got, want, bound):
    err = (got.double() - want).abs()
    assert (err <= bound + 1e-12).all(), float((err / (bound + 1e-12)).max())


def _parts(nq, nk, heads, seqs):
    """A few (query rows, key rows, head) of a batch."""
    for b in sorted({0, seqs - 1}):
        for h in sorted({0, heads // 3, heads - 1}):
            yield slice(b * nq, (b + 1) * nq), slice(b * nk, (b + 1) * nk), h


@pytest.mark.gpu
@pytest.mark.parametrize("nq,nk,heads,kv_heads,seqs", FORWARD)
def test_forward(nq, nk, heads, kv_heads, seqs, ress_gpu):
    q, k, v, _, off = _make(nq, nk, heads, kv_heads, seqs, nq + nk)
    out, lse = ress_gpu.ress_cross_attn(q, k, v, **off)
    assert ress_gpu.ress_check_device_errors() == (0, 0)
    for a, c, h in _parts(nq, nk, heads, seqs):
        K, V = (t[c, h * kv_heads // heads].double() for t in (k, v))
        s = q[a, h].double() @ K.T / 8.0
        want = torch.logsumexp(s, dim=1)
        p = torch.exp(s - want[:, None])
        ref = p @ V
        _within(out[a, h], ref, (2.0 ** -8 + 2.0 ** -12) * (p @ V.abs()) + 2.0 ** -8 * ref.abs())
        _within(lse[h, a], want, 1e-4 + 1e-5 * want.abs())
    again = ress_gpu.ress_cross_attn(q, k, v, **off)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("nq,nk,heads,kv_heads,seqs", QUERY_WALK + KEY_WALK)
def test_gradients(nq, nk, heads, kv_heads, seqs, ress_gpu):
    q, k, v, do, off = _make(nq, nk, heads, kv_heads, seqs, nq + nk)
    out, lse = ress_gpu.ress_cross_attn(q, k, v, **off)
    grads = ress_gpu.ress_cross_attn_bwd(q, k, v, out, lse, do, **off)
    assert ress_gpu.ress_check_device_errors() == (0, 0)
    group = heads // kv_heads
    for a, c, hk in _parts(nq, nk, kv_heads, seqs):
        K, V = (t[c, hk].double() for t in (k, v))
        sums = [torch.zeros_like(K) for _ in range(4)]      # dk, its bound, dv, its bound
        for h in range(hk * group, (hk + 1) * group):
            Q, D, O = (t[a, h].double() for t in (q, do, out))
            p = torch.exp(Q @ K.T / 8.0 - lse[h, a].double()[:, None])
            dS = p * (D @ V.T - (D * O).sum(1, keepdim=True))
            N = p * (D.abs() @ V.abs().T + (D * O).abs().sum(1, keepdim=True))
            W = (2.0 ** -8 + 2.0 ** -12) * dS.abs() + 2.0 ** -13 * N
            ref = dS @ K / 8.0
            _within(grads[0][a, h], ref, W @ K.abs() / 8.0 + 2.0 ** -8 * ref.abs())
            for at, x in zip(sums, (dS.T @ Q / 8.0, W.T @ Q.abs() / 8.0, p.T @ D,
                                    (2.0 ** -8 + 2.0 ** -12) * (p.T @ D.abs()))):
                at += x
        _within(grads[1][c, hk], sums[0], sums[1] + 2.0 ** -8 * sums[0].abs())
        _within(grads[2][c, hk], sums[2], sums[3] + 2.0 ** -8 * sums[2].abs())
    for x, y in zip(grads, ress_gpu.ress_cross_attn_bwd(q, k, v, out, lse, do, **off)):
        assert torch.equal(x, y)
