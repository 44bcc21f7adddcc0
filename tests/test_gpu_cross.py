"""Attention over keys of another length and its gradients on the GPU, against
float64.

Tolerances, derived before the first run.  Forward: a probability enters P V
rounded to bf16 (at most 2^-8 relative) while the normaliser is not rounded, so
|out - ref| <= 2^-8 * sum_t p_t |v_t| + 2^-8 |out| (the output's own rounding)
+ 2^-12 * sum_t p_t |v_t| (exponentials to 2^-14, float32 sums).  lse: logits are
float32 sums of 64 exact products (|error| <= 64 * 2^-24 * sum |q k| / 8, below
2^-14 for sums up to 64), and ex2 and lg2 are good to 2^-20: 1e-4 + 1e-5 |lse|.
Gradients: P and dS enter their products rounded to bf16, so
|dv - ref| <= (2^-8 + 2^-12) sum_i P |dout| + 2^-8 |dv|, and
|dk - ref| <= (2^-8 + 2^-12) sum_i |dS| |q| / 8 + 2^-8 |dk| + 2^-13 sum_i P N |q| / 8
where N = |dout| . (|v| + |out|) bounds the magnitudes that cancel in dS (float32
sums of 64 terms: 64 * 2^-24 each side, and the exponentials' 2^-14); dq the same
with k in the place of q."""

import math

import numpy as np
import pytest
import torch

from tests.parity import np64

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _off(v):
    return _i32(np.concatenate([[0], np.cumsum(v)]).astype(np.int64).tolist())


def _ok(ress):
    status, detail = ress.ress_check_device_errors()
    assert status == 0, (status, detail)


def make(nq, nk, heads, kv_heads, seed, qlen=None, klen=None, poison=True):
    """Packed q, k, v, dout; rows behind a sequence's data hold NaN."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(sum(nq), heads, 64, generator=g)
    k, v = (torch.randn(sum(nk), kv_heads, 64, generator=g) for _ in range(2))
    do = torch.randn(sum(nq), heads, 64, generator=g)
    q, k, v, do = (t.to(torch.bfloat16) for t in (q, k, v, do))
    if poison:
        for n, lens, ts in ((nq, qlen, (q, do)), (nk, klen, (k, v))):
            at = 0
            for b, m in enumerate(n):
                for t in ts:
                    if lens is not None:
                        t[at + lens[b]:at + m] = float("nan")
                at += m
    return q, k, v, do


def reference(q, k, v, nq, nk, qlen=None, klen=None, do=None, out=None, lse=None):
    """Outputs, lse, bounds (and gradients with theirs, given out, lse and dout) in float64."""
    qn, kn, vn = np64(q), np64(k), np64(v)
    heads, hk = qn.shape[1], kn.shape[1]
    g = heads // hk
    r = {"out": np.zeros(qn.shape), "lse": np.full((heads, qn.shape[0]), -np.inf),
         "bout": np.zeros(qn.shape)}
    for n, like in (("dq", qn), ("dk", kn), ("dv", kn)):
        r[n], r["b" + n] = np.zeros(like.shape), np.zeros(like.shape)
    q0 = k0 = 0
    for b in range(len(nq)):
        a = slice(q0, q0 + (nq[b] if qlen is None else qlen[b]))
        c = slice(k0, k0 + (nk[b] if klen is None else klen[b]))
        q0, k0 = q0 + nq[b], k0 + nk[b]
        if a.stop == a.start or c.stop == c.start:
            continue
        for h in range(heads):
            Q, K, V = qn[a, h], kn[c, h // g], vn[c, h // g]
            s = Q @ K.T / 8.0
            top = s.max(axis=1, keepdims=True)
            p = np.exp(s - top)
            z = p.sum(axis=1, keepdims=True)
            r["lse"][h, a] = (top + np.log(z))[:, 0]
            p /= z
            r["out"][a, h] = p @ V
            r["bout"][a, h] = (2.0 ** -8 + 2.0 ** -12) * (p @ np.abs(V)) + 2.0 ** -8 * np.abs(p @ V)
            if do is None:
                continue
            D, O = np64(do)[a, h], np64(out)[a, h]
            P = np.exp(s - np64(lse)[h, a][:, None])
            dS = P * (D @ V.T - (D * O).sum(axis=1)[:, None])
            N = P * (np.abs(D) @ np.abs(V).T + (np.abs(D) * np.abs(O)).sum(axis=1)[:, None])
            W = (2.0 ** -8 + 2.0 ** -12) * np.abs(dS) + 2.0 ** -13 * N
            r["dq"][a, h] = dS @ K / 8
            r["bdq"][a, h] = W @ np.abs(K) / 8
            r["dk"][c, h // g] += dS.T @ Q / 8
            r["bdk"][c, h // g] += W.T @ np.abs(Q) / 8
            r["dv"][c, h // g] += P.T @ D
            r["bdv"][c, h // g] += (2.0 ** -8 + 2.0 ** -12) * (P.T @ np.abs(D))
    for n in ("dq", "dk", "dv"):
        r["b" + n] += 2.0 ** -8 * np.abs(r[n])
    return r


def close(got, ref, name):
    x = np64(got)
    assert np.isfinite(x).all(), name
    err, bound = np.abs(x - ref[name]), ref["b" + name] + 1e-12
    assert (err <= bound).all(), (name, float((err / bound).max()))


def close_lse(got, ref):
    l, want = np64(got), ref["lse"]
    dead = np.isinf(want)
    assert np.array_equal(np.isinf(l), dead) and (l[dead] < 0).all()
    err = np.abs(l[~dead] - want[~dead])
    assert (err <= 1e-4 + 1e-5 * np.abs(want[~dead])).all(), err.max()


CASES = [
    # nq, nk, heads, kv heads, real queries, real keys
    ([1], [1], 1, 1, None, None),
    ([1], [300], 16, 16, None, None),
    ([5], [1374], 4, 1, None, None),
    ([129], [64], 2, 2, None, None),
    ([300], [127], 3, 1, None, None),
    ([128], [128], 64, 64, None, None),
    ([64, 0, 33, 1], [128, 7, 0, 65], 4, 2, None, None),
    ([200, 10], [500, 129], 6, 2, [150, 10], [400, 0]),
    ([513], [1025], 2, 1, [500], [1000]),
    ([700, 700], [900, 31], 12, 4, None, [899, 1]),
    ([40] * 30, [70] * 30, 8, 1, None, [69 - i for i in range(30)]),
    ([2], [5000], 64, 2, None, None),
    ([3000], [3], 2, 2, None, None),
    ([2000], [1700], 1, 1, None, None),
    ([600, 300, 129], [700, 50, 400], 16, 16, None, None),   # many items of several costs
    ([1500], [130], 64, 64, None, None),                     # more equal items than CTAs
]


@pytest.mark.parametrize("nq,nk,heads,kv_heads,qlen,klen", CASES)
def test_forward_and_gradients(nq, nk, heads, kv_heads, qlen, klen, ress_gpu):
    q, k, v, do = make(nq, nk, heads, kv_heads, seed=sum(nq) + sum(nk) + heads, qlen=qlen, klen=klen)
    dev = [t.cuda() for t in (q, k, v)]
    one = len(nq) == 1
    seqs = dict(q_offsets=None if one else _off(nq), kv_offsets=None if one else _off(nk),
                q_lens=None if qlen is None else _i32(qlen),
                kv_lens=None if klen is None else _i32(klen))
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((heads, q.shape[0]), 7.0, device="cuda")
    ress_gpu.ress_cross_attn(*dev, out=out, lse=lse, **seqs)
    _ok(ress_gpu)
    ref = reference(q, k, v, nq, nk, qlen, klen, do, out, lse)
    close(out, ref, "out")
    close_lse(lse, ref)
    grads = [torch.full(t.shape, 7.0, dtype=torch.bfloat16, device="cuda") for t in (q, k, v)]
    ress_gpu.ress_cross_attn_bwd(*dev, out, lse, do.cuda(), dq=grads[0], dk=grads[1], dv=grads[2],
                                 **seqs)
    _ok(ress_gpu)
    for name, t in zip(("dq", "dk", "dv"), grads):
        close(t, ref, name)
    # the same again: no result depends on the run
    again = ress_gpu.ress_cross_attn(*dev, **seqs)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    for a, b in zip(ress_gpu.ress_cross_attn_bwd(*dev, out, lse, do.cuda(), **seqs), grads):
        assert torch.equal(a, b)
    only, none = ress_gpu.ress_cross_attn(*dev, want_lse=False, **seqs)
    assert none is None and torch.equal(only, out)


def test_pieces_in_two_rounds(ress_gpu):
    """96 equal items, each cut into three pieces, two pieces per CTA: against
    float64 on the GPU, and against the same queries in calls of their own."""
    g = torch.Generator().manual_seed(13)
    q, k, v = (torch.randn(n, 48, 64, generator=g).to(torch.bfloat16).cuda()
               for n in (300, 20000, 20000))
    out, lse = ress_gpu.ress_cross_attn(q, k, v)
    _ok(ress_gpu)
    for h in (0, 17, 47):
        s = q[:, h].double() @ k[:, h].double().T / 8.0
        want = torch.logsumexp(s, dim=1)
        p = torch.exp(s - want[:, None])
        bound = (2.0 ** -8 + 2.0 ** -12) * (p @ v[:, h].double().abs())
        ref = p @ v[:, h].double()
        assert ((out[:, h].double() - ref).abs() <= bound + 2.0 ** -8 * ref.abs()).all()
        assert ((lse[h].double() - want).abs() <= 1e-4 + 1e-5 * want.abs()).all()


def test_compiled_and_python_calls_agree(ress_gpu):
    """The binding's C++ part and the Python code behind it make the same call, and
    raise the same errors."""
    q, k, v, do = (t.cuda() for t in make([50, 7], [90, 33], 4, 2, seed=21))
    seqs = dict(q_offsets=_off([50, 7]), kv_offsets=_off([90, 33]), kv_lens=_i32([80, 33]))
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    call = ress_gpu._call
    assert call is not None
    fast = call.cross_attn(q, k, v, seqs["q_offsets"], seqs["kv_offsets"], None, seqs["kv_lens"], True)
    slow = ress_gpu.ress_cross_attn(q, k, v, **seqs, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(fast, slow))
    args = (q, k, v, seqs["q_offsets"], seqs["kv_offsets"], None, seqs["kv_lens"])
    fast = call.cross_attn_bwd(*args, *slow, do)
    slow = ress_gpu.ress_cross_attn_bwd(q, k, v, *slow, do, **seqs, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(fast, slow))
    _ok(ress_gpu)
    with pytest.raises(TypeError, match="kv_lens must be"):
        ress_gpu.ress_cross_attn(q, k, v, kv_lens=torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="kv_offsets must have shape"):
        ress_gpu.ress_cross_attn(q, k, v, q_offsets=_off([50, 7]), kv_offsets=_off([90]))
    with pytest.raises(TypeError, match="k must be"):
        ress_gpu.ress_cross_attn(q, k.float(), v.float())
    with pytest.raises(ValueError, match="must be on"):
        ress_gpu.ress_cross_attn(q, k, v, kv_lens=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ress_gpu.RessError):
        ress_gpu.ress_cross_attn(q, k[:, :1].expand(-1, 3, -1).contiguous(),
                                 k[:, :1].expand(-1, 3, -1).contiguous())     # 3 does not divide 4


def test_gradients_against_differences(ress_gpu):
    """The directional derivative of sum(out * dout) along random directions of
    q, k and v: central differences of the float64 forward, whose own error is
    below 1e-6 here (third derivatives of order one times step^2 = 1e-8), against
    the kernel's gradients, each off by no more than its bound."""
    nq, nk, heads, hk = [37, 20], [90, 33], 4, 2
    q, k, v, do = make(nq, nk, heads, hk, seed=3)
    dev = [t.cuda() for t in (q, k, v)]
    seqs = dict(q_offsets=_off(nq), kv_offsets=_off(nk))
    out, lse = ress_gpu.ress_cross_attn(*dev, **seqs)
    grads = ress_gpu.ress_cross_attn_bwd(*dev, out, lse, do.cuda(), **seqs)
    ref = reference(q, k, v, nq, nk, do=do, out=out, lse=lse)
    rng = np.random.default_rng(4)
    base = [np64(t) for t in (q, k, v)]
    for i, name in enumerate(("dq", "dk", "dv")):
        d = rng.standard_normal(base[i].shape)
        d /= np.linalg.norm(d)
        vals = []
        for sign in (1, -1):
            x = [torch.from_numpy(t + (sign * 1e-4 * d if j == i else 0)) for j, t in enumerate(base)]
            vals.append((reference(*x, nq, nk)["out"] * np64(do)).sum())
        slope = (vals[0] - vals[1]) / 2e-4
        got = (np64(grads[i]) * d).sum()
        # the kernel's delta is dout . out with out in bf16: 2^-8 relative of each term
        slack = (ref["b" + name] * np.abs(d)).sum()
        assert abs(got - slope) <= slack + 1e-5, (name, got, slope, slack)


def test_rows_are_slices_of_fused_projections(ress_gpu):
    """q, k and v as views into wider token rows, against dense copies."""
    g = torch.Generator().manual_seed(8)
    qq = torch.randn(300, 5, 4, 64, generator=g).to(torch.bfloat16).cuda()
    kv = torch.randn(500, 2, 2, 64, generator=g).to(torch.bfloat16).cuda()
    args = (qq[:, 3], kv[:, 0], kv[:, 1])
    dense = tuple(t.contiguous() for t in args)
    out, lse = ress_gpu.ress_cross_attn(*args)
    want = ress_gpu.ress_cross_attn(*dense)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    do = torch.randn(300, 4, 64, generator=g).to(torch.bfloat16).cuda()
    for a, b in zip(ress_gpu.ress_cross_attn_bwd(*args, out, lse, do),
                    ress_gpu.ress_cross_attn_bwd(*dense, out, lse, do)):
        assert torch.equal(a, b)
    _ok(ress_gpu)


def test_rows_of_no_sequence_are_left_as_they_were(ress_gpu):
    q, k, v, do = make([20], [40], 2, 2, seed=5)
    dev = [t.cuda() for t in (q, k, v, do)]
    seqs = dict(q_offsets=_i32([3, 10, 15]), kv_offsets=_i32([5, 20, 33]))
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((2, 20), 7.0, device="cuda")
    ress_gpu.ress_cross_attn(*dev[:3], out=out, lse=lse, **seqs)
    assert (out[:3] == 7).all() and (out[15:] == 7).all()
    assert (lse[:, :3] == 7).all() and (lse[:, 15:] == 7).all()
    grads = [torch.full(t.shape, 7.0, dtype=torch.bfloat16, device="cuda") for t in (q, k, v)]
    ress_gpu.ress_cross_attn_bwd(*dev[:3], out, lse, dev[3], dq=grads[0], dk=grads[1], dv=grads[2],
                                 **seqs)
    _ok(ress_gpu)
    for t, a, b in zip(grads, (3, 5, 5), (15, 33, 33)):
        assert (t[:a] == 7).all() and (t[b:] == 7).all()
    ref = reference(q[3:15], k[5:33], v[5:33], [7, 5], [15, 13], do=do[3:15], out=out[3:15],
                    lse=lse[:, 3:15])
    close(out[3:15], ref, "out")
    close(grads[0][3:15], ref, "dq")
    close(grads[1][5:33], ref, "dk")
    close(grads[2][5:33], ref, "dv")


def test_infinities_and_nan_of_masked_keys_stay_there(ress_gpu):
    """A padded key row of NaN and one of infinities change nothing."""
    nq, nk = [150], [200]
    q, k, v, do = make(nq, nk, 2, 1, seed=6, klen=[170])
    k[180:190], v[180:190] = float("inf"), float("-inf")
    seqs = dict(kv_lens=_i32([170]))
    dev = [t.cuda() for t in (q, k, v)]
    out, lse = ress_gpu.ress_cross_attn(*dev, **seqs)
    grads = ress_gpu.ress_cross_attn_bwd(*dev, out, lse, do.cuda(), **seqs)
    _ok(ress_gpu)
    ref = reference(q, k, v, nq, nk, klen=[170], do=do, out=out, lse=lse)
    close(out, ref, "out")
    for name, t in zip(("dq", "dk", "dv"), grads):
        close(t, ref, name)
    assert (grads[1][170:] == 0).all() and (grads[2][170:] == 0).all()


@pytest.mark.parametrize("nq,nk", [(3, 20), (40, 3000), (700, 400)])
def test_nan_that_is_attended_to_comes_out(nq, nk, ress_gpu):
    """A NaN in a query row or in a key reaches every output that depends on it,
    and a NaN value its dimension of them; other heads and rows stay as they were."""
    q, k, v, _ = make([nq], [nk], 4, 2, seed=11)
    want, wlse = ress_gpu.ress_cross_attn(q.cuda(), k.cuda(), v.cuda())
    a, b, c = (t.clone() for t in (q, k, v))
    a[1, 1, 5] = float("nan")            # query head 1 of token 1
    b[nk - 2, 1, 60] = float("nan")      # key head 1: query heads 2 and 3
    c[7, 0, 9] = float("nan")            # value head 0: query heads 0 and 1
    out, lse = ress_gpu.ress_cross_attn(a.cuda(), b.cuda(), c.cuda())
    _ok(ress_gpu)
    bad = torch.zeros(out.shape, dtype=torch.bool)
    bad[1, 1] = True
    bad[:, 2:] = True
    bad[:, :2, 9] = True
    assert torch.equal(out.isnan().cpu(), bad)
    assert torch.equal(out.cpu()[~bad], want.cpu()[~bad])
    lbad = torch.zeros(lse.shape, dtype=torch.bool)
    lbad[1, 1] = True
    lbad[2:] = True
    assert torch.equal(lse.isnan().cpu(), lbad)
    assert torch.equal(lse.cpu()[~lbad], wlse.cpu()[~lbad])


def test_large_and_flat_logits(ress_gpu):
    """One key that takes all of a row, and rows whose keys are all the same."""
    q, k, v, do = make([130], [400], 1, 1, seed=9)
    k[7] = 0.0
    k[300] = (q[5, 0].float() * 8).to(torch.bfloat16)
    q[60:70] = 0.0
    dev = [t.cuda() for t in (q, k, v)]
    out, lse = ress_gpu.ress_cross_attn(*dev)
    grads = ress_gpu.ress_cross_attn_bwd(*dev, out, lse, do.cuda())
    _ok(ress_gpu)
    ref = reference(q, k, v, [130], [400], do=do, out=out, lse=lse)
    close(out, ref, "out")
    assert abs(float(lse[0, 60]) - math.log(400)) < 1e-4
    for name, t in zip(("dq", "dk", "dv"), grads):
        close(t, ref, name)


def test_bad_offsets_and_lengths_are_flagged(ress_gpu):
    q, k, v, do = make([100], [100], 1, 1, seed=10)
    dev = [t.cuda() for t in (q, k, v)]

    def flagged(detail, **seqs):
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        _, lse = ress_gpu.ress_cross_attn(*dev, out=out, **seqs)
        status, seen = ress_gpu.ress_check_device_errors()
        assert status == ress_gpu.RESS_ERR_BAD_INDEX and seen == detail, (status, seen)
        ress_gpu.ress_cross_attn_bwd(*dev, out, lse, do.cuda(), **seqs)
        status, seen = ress_gpu.ress_check_device_errors()
        assert status == ress_gpu.RESS_ERR_BAD_INDEX and seen == detail, (status, seen)
        return out

    out = flagged(90, q_offsets=_i32([0, 101]), kv_offsets=_i32([0, 100]))
    assert (out == 7).all()
    flagged(90, q_offsets=_i32([50, 20, 30]), kv_offsets=_i32([0, 50, 100]))
    flagged(91, q_offsets=_i32([0, 100]), kv_offsets=_i32([-4, 100]))
    flagged(92, q_lens=_i32([101]))
    out = flagged(93, kv_lens=_i32([-1]))
    assert (out == 0).all()


def test_no_queries_and_no_keys(ress_gpu):
    e = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    x = torch.ones(9, 2, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = ress_gpu.ress_cross_attn(e, x, x)
    assert out.shape == (0, 2, 64) and lse.shape == (2, 0)
    out, lse = ress_gpu.ress_cross_attn(x, e, e)
    assert (out == 0).all() and (lse == -math.inf).all()
    dq, dk, dv = ress_gpu.ress_cross_attn_bwd(x, e, e, out, lse, x)
    assert (dq == 0).all() and dk.shape == (0, 2, 64)
    dq, dk, dv = ress_gpu.ress_cross_attn_bwd(e, x, x, e, lse[:, :0].contiguous(), e)
    assert (dk == 0).all() and (dv == 0).all()
    _ok(ress_gpu)


@pytest.mark.parametrize("nq,nk", [(7, 3000), (600, 900)])
def test_streams_graphs_and_two_calls_at_once(nq, nk, ress_gpu):
    """Forward and backward captured into a graph and replayed on new inputs,
    with calls on another stream between the replays."""
    q, k, v, do = (t.cuda() for t in make([nq], [nk], 4, 2, seed=nq))

    def step():
        out, lse = ress_gpu.ress_cross_attn(q, k, v)
        return (out, lse) + ress_gpu.ress_cross_attn_bwd(q, k, v, out, lse, do)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (1, 2):
        for t, n in zip((q, k, v, do), make([nq], [nk], 4, 2, seed=seed)):
            t.copy_(n)
        torch.cuda.synchronize()
        graph.replay()
        out, lse = ress_gpu.ress_cross_attn(q, k, v, stream=side)
        rest = ress_gpu.ress_cross_attn_bwd(q, k, v, out, lse, do, stream=side)
        torch.cuda.synchronize()
        for a, b in zip(got, (out, lse) + rest):
            assert torch.equal(a, b)
    _ok(ress_gpu)


def test_offsets_beyond_32_bits(ress_gpu):
    """Token rows whose element offsets pass 2^31 (a slice of very wide rows)."""
    n, wide = 40, 1 << 26
    big = torch.empty(n * wide, dtype=torch.bfloat16, device="cuda").view(n, wide)
    x = torch.randn(n, 2, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    big[:, :128] = x.view(n, 128)
    rows = big[:, :128].unflatten(1, (2, 64))
    out, lse = ress_gpu.ress_cross_attn(rows, rows, rows)
    want = ress_gpu.ress_cross_attn(x, x, x)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    for a, b in zip(ress_gpu.ress_cross_attn_bwd(rows, rows, rows, out, lse, x),
                    ress_gpu.ress_cross_attn_bwd(x, x, x, out, lse, x)):
        assert torch.equal(a, b)
    _ok(ress_gpu)
