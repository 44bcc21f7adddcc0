"""Refusals of the cross-attention and cache operators: the C ABI and the
binding turn every argument that a kernel could not work on into an error
before any CUDA call (no GPU needed)."""

import ctypes

import pytest
import torch

from block_sparse_global_mean_b200 import build as ress_build

FAKE = 0x10000          # 16-byte aligned, never dereferenced
FAKE_WS = 0x20000       # 256-byte aligned

no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(),
                                 reason="placeholder-pointer cases run only without a GPU")


@pytest.fixture(scope="module")
def ress():
    ress_build.build()
    from block_sparse_global_mean_b200 import ress as mod
    return mod


def _cross(ress, **kw):
    a = dict(nq=100, nk=200, seqs=1, heads=4, kv_heads=2, head_dim=64, dtype=0, q_stride=0,
             k_stride=0, v_stride=0)
    a.update(kw)
    return ress.ress_cross_shape(**a)


SHAPES = [  # (changes to a valid shape, status)
    (dict(nq=-1), "INVALID_ARG"), (dict(nk=-1), "INVALID_ARG"), (dict(seqs=0), "INVALID_ARG"),
    (dict(heads=0), "INVALID_ARG"), (dict(kv_heads=3), "INVALID_ARG"),
    (dict(kv_heads=0), "INVALID_ARG"), (dict(heads=66), "UNSUPPORTED"),
    (dict(head_dim=32), "UNSUPPORTED"), (dict(head_dim=0), "INVALID_ARG"),
    (dict(dtype=1), "UNSUPPORTED"), (dict(dtype=9), "INVALID_ARG"),
    (dict(nq=2 ** 31), "UNSUPPORTED"), (dict(nk=2 ** 30 + 1), "UNSUPPORTED"),
    (dict(seqs=8193), "UNSUPPORTED"), (dict(q_stride=4 * 64 - 8), "INVALID_ARG"),
    (dict(k_stride=2 * 64 + 4), "INVALID_ARG"), (dict(v_stride=-256), "INVALID_ARG"),
    (dict(v_stride=2 ** 33), "INVALID_ARG"), (dict(seqs=2), "INVALID_ARG"),   # no offsets
]


@no_gpu_only
@pytest.mark.parametrize("change,status", SHAPES)
def test_cross_refuses_a_shape(change, status, ress):
    sh = ctypes.byref(_cross(ress, **change))
    want = getattr(ress, "RESS_ERR_" + status)
    assert ress.lib.ress_cross_attn(sh, FAKE, FAKE, FAKE, None, None, None, None, FAKE, FAKE,
                                    FAKE_WS, 1 << 40, None) == want
    assert ress.lib.ress_cross_attn_bwd(sh, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, None, None,
                                        None, FAKE, FAKE, FAKE, FAKE_WS, 1 << 40, None) == want
    if change != dict(seqs=2):
        assert ress.lib.ress_cross_workspace_bytes(sh) == 0
        assert ress.lib.ress_cross_bwd_workspace_bytes(sh) == 0


@no_gpu_only
def test_cross_refuses_pointers(ress):
    sh = ctypes.byref(_cross(ress))
    bad = ress.RESS_ERR_INVALID_ARG
    good = [FAKE, FAKE, FAKE, None, None, None, None, FAKE, FAKE]
    for i, p in ((0, None), (1, None), (2, None), (7, None), (0, FAKE + 8), (1, FAKE + 2),
                 (2, FAKE + 8), (7, FAKE + 8), (8, FAKE + 2), (3, FAKE), (4, FAKE), (5, FAKE + 1),
                 (6, FAKE + 2)):
        a = list(good)
        a[i] = p
        assert ress.lib.ress_cross_attn(sh, *a, FAKE_WS, 1 << 40, None) == bad, (i, p)
    good = [FAKE] * 6 + [None] * 4 + [FAKE] * 3
    for i in (0, 1, 2, 3, 4, 5, 10, 11, 12):
        for p in (None, FAKE + 2):
            a = list(good)
            a[i] = p
            assert ress.lib.ress_cross_attn_bwd(sh, *a, FAKE_WS, 1 << 40, None) == bad, (i, p)
    need = ress.lib.ress_cross_bwd_workspace_bytes(sh)
    assert need > 0
    for ws, size, want in ((None, 0, ress.RESS_ERR_WORKSPACE),
                           (FAKE_WS, need - 1, ress.RESS_ERR_WORKSPACE), (FAKE_WS + 16, need, bad)):
        assert ress.lib.ress_cross_attn_bwd(sh, *good, ws, size, None) == want
    need = ress.lib.ress_cross_workspace_bytes(sh)
    good = [FAKE, FAKE, FAKE, None, None, None, None, FAKE, FAKE]
    if need:
        assert ress.lib.ress_cross_attn(sh, *good, FAKE_WS, need - 1, None) == \
            ress.RESS_ERR_WORKSPACE
        assert ress.lib.ress_cross_attn(sh, *good, FAKE_WS + 16, need, None) == bad
    assert ress.lib.ress_cross_attn(None, *good, FAKE_WS, 1 << 40, None) == bad
    empty = ctypes.byref(_cross(ress, nq=0))
    assert ress.lib.ress_cross_attn(empty, *[None] * 9, None, 0, None) == ress.RESS_OK
    empty = ctypes.byref(_cross(ress, nq=0, nk=0))
    assert ress.lib.ress_cross_attn_bwd(empty, *[None] * 13, None, 0, None) == ress.RESS_OK


def _cache(ress, **kw):
    a = dict(pages=10, page=64, kv_heads=2, head_dim=64, requests=3, max_pages=5)
    a.update(kw)
    return ress.ress_cache_shape(**a)


@no_gpu_only
@pytest.mark.parametrize("change,status", [
    (dict(pages=0), "INVALID_ARG"), (dict(page=0), "INVALID_ARG"), (dict(page=32), "UNSUPPORTED"),
    (dict(page=256), "UNSUPPORTED"), (dict(kv_heads=0), "INVALID_ARG"),
    (dict(kv_heads=65), "UNSUPPORTED"), (dict(head_dim=128), "UNSUPPORTED"),
    (dict(pages=2 ** 25, page=64), "UNSUPPORTED")])
def test_cache_refuses_a_pool(change, status, ress):
    sh = ctypes.byref(_cache(ress, **change))
    want = getattr(ress, "RESS_ERR_" + status)
    assert ress.lib.ress_cache_append(sh, FAKE, FAKE, 0, 0, 0, FAKE, 5, FAKE, FAKE, FAKE, FAKE,
                                      None) == want
    heads = 4 if change.get("kv_heads", 2) == 2 else change["kv_heads"] * 2
    assert ress.lib.ress_cache_attn(sh, heads, 3, FAKE, 0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                                    FAKE, 0, FAKE, FAKE, FAKE_WS, 1 << 40, None) == want
    assert ress.lib.ress_cache_attn_workspace_bytes(sh, heads, 3) == 0


@no_gpu_only
@pytest.mark.parametrize("change,status", [
    (dict(requests=0), "INVALID_ARG"), (dict(max_pages=0), "INVALID_ARG"),
    (dict(requests=8193), "UNSUPPORTED"), (dict(max_pages=2 ** 25), "UNSUPPORTED")])
def test_cache_refuses_a_table(change, status, ress):
    sh = ctypes.byref(_cache(ress, **change))
    want = getattr(ress, "RESS_ERR_" + status)
    assert ress.lib.ress_cache_plan(sh, FAKE, FAKE, FAKE, FAKE, 5, FAKE, 5, FAKE + 64, FAKE + 64,
                                    FAKE + 64, FAKE + 64, None) == want
    assert ress.lib.ress_cache_attn(sh, 4, 3, FAKE, 0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0,
                                    FAKE, FAKE, FAKE_WS, 1 << 40, None) == want


@no_gpu_only
def test_cache_calls_refuse_arguments(ress):
    lib, bad = ress.lib, ress.RESS_ERR_INVALID_ARG
    sh = ctypes.byref(_cache(ress))

    def plan(ptrs=None, n_free=5, tokens=5):
        a = [FAKE, FAKE, FAKE, FAKE, FAKE] + [FAKE + 64] * 4
        for i, p in (ptrs or {}).items():
            a[i] = p
        return lib.ress_cache_plan(sh, a[0], a[1], a[2], a[3], n_free, a[4], tokens, *a[5:], None)
    for i in range(9):
        assert plan({i: None}) == bad and plan({i: FAKE + 2}) == bad, i
    assert plan(n_free=-1) == bad and plan(tokens=-1) == bad
    for i in (5, 6, 7, 8):
        assert plan({i: FAKE}) == bad        # an output on an input

    def append(ptrs=None, dtype=0, ks=0, vs=0, tokens=5):
        a = [FAKE] * 7
        for i, p in (ptrs or {}).items():
            a[i] = p
        return lib.ress_cache_append(sh, a[0], a[1], dtype, ks, vs, a[2], tokens, *a[3:], None)
    for i in range(7):
        assert append({i: None}) == bad and append({i: FAKE + 2}) == bad, i
    assert append(dtype=2) == bad and append(tokens=-1) == bad
    assert append(tokens=2 ** 29 + 1) == ress.RESS_ERR_UNSUPPORTED
    assert append(ks=64) == bad and append(vs=2 * 64 + 4) == bad
    assert append({i: None for i in range(7)}, tokens=0) == ress.RESS_OK

    def attn(ptrs=None, heads=4, tokens=3, qs=0, step=0, ws=FAKE_WS, size=1 << 40):
        a = [FAKE] * 10
        for i, p in (ptrs or {}).items():
            a[i] = p
        return lib.ress_cache_attn(sh, heads, tokens, a[0], qs, *a[1:8], step, a[8], a[9], ws, size,
                                   None)
    for i in range(9):
        assert attn({i: None}) == bad and attn({i: FAKE + 2}) == bad, i
    assert attn({9: FAKE + 2}) == bad
    assert attn(heads=3) == bad and attn(heads=0) == bad and attn(step=-1) == bad
    assert attn(tokens=-1) == bad and attn(qs=4 * 64 - 8) == bad and attn(qs=4 * 64 + 4) == bad
    assert attn(heads=128) == ress.RESS_ERR_UNSUPPORTED
    assert attn(tokens=2 ** 30 + 1) == ress.RESS_ERR_UNSUPPORTED
    assert attn(tokens=0) == ress.RESS_OK
    need = lib.ress_cache_attn_workspace_bytes(sh, 4, 3)
    if need:
        assert attn(size=need - 1) == ress.RESS_ERR_WORKSPACE
        assert attn(ws=FAKE_WS + 16, size=need) == bad


def test_binding_refuses_mismatched_tensors(ress):
    bf, i32 = torch.bfloat16, torch.int32
    q, k = torch.zeros(10, 4, 64, dtype=bf), torch.zeros(20, 2, 64, dtype=bf)
    off = torch.zeros(3, dtype=i32)
    with pytest.raises(ValueError, match="CUDA device"):
        ress.ress_cross_attn(q, k, k)
    with pytest.raises(TypeError, match="q must be"):
        ress.ress_cross_attn(q.float(), k, k)
    with pytest.raises(ValueError, match="q must be"):
        ress.ress_cross_attn(q[0], k, k)

    class Fake(torch.Tensor):
        """A host tensor that says it is on a device, to reach the later checks."""
        is_cuda = True

    q, k, off = (t.as_subclass(Fake) for t in (q, k, off))
    with pytest.raises(ValueError, match="v has shape"):
        ress.ress_cross_attn(q, k, k[:19])
    with pytest.raises(ValueError, match="come together"):
        ress.ress_cross_attn(q, k, k, q_offsets=off)
    with pytest.raises(ValueError, match="kv_offsets must have shape"):
        ress.ress_cross_attn(q, k, k, q_offsets=off, kv_offsets=off[:2])
    with pytest.raises(TypeError, match="kv_lens must be"):
        ress.ress_cross_attn(q, k, k, kv_lens=torch.zeros(1))
    with pytest.raises(ValueError, match="stand together"):
        ress.ress_cross_attn(q.transpose(0, 1).contiguous().transpose(0, 1), k, k)
    with pytest.raises(ValueError, match="out must have shape"):
        ress.ress_cross_attn(q, k, k, out=k)
    with pytest.raises(ValueError, match="dout must have shape"):
        ress.ress_cross_attn_bwd(q, k, k, q, torch.zeros(4, 10).as_subclass(Fake), k)
    with pytest.raises(ValueError, match="lse must have shape"):
        ress.ress_cross_attn_bwd(q, k, k, q, torch.zeros(10, 4).as_subclass(Fake), q)

    cache = ress.ress_cache(*(t.as_subclass(Fake)
                              for t in ress.make_cache(4, 2, 64, device="cpu")))
    slots = torch.zeros(20, dtype=i32).as_subclass(Fake)
    with pytest.raises(ValueError, match="heads"):
        ress.ress_cache_append(q, q, slots, cache)
    with pytest.raises(ValueError, match="slots must have shape"):
        ress.ress_cache_append(k, k, slots[:3], cache)
    with pytest.raises(TypeError, match="k must be"):
        ress.ress_cache_append(k.half(), k.half(), slots, cache)
    with pytest.raises(TypeError, match="v must be"):
        ress.ress_cache_append(k, k.float(), slots, cache)
    with pytest.raises(ValueError, match="cache.v must have shape"):
        ress.ress_cache_append(k, k, slots, cache._replace(v=cache.v[:3]))
    with pytest.raises(TypeError, match="cache.k must be"):
        ress.ress_cache_append(k, k, slots, cache._replace(k=cache.k.to(bf)))
    table = torch.zeros(2, 3, dtype=i32).as_subclass(Fake)
    with pytest.raises(ValueError, match="offsets must have shape"):
        ress.ress_cache_attn(q, cache, table, off[:2], off[:2])
    with pytest.raises(ValueError, match="table must be"):
        ress.ress_cache_attn(q, cache, torch.zeros(2, dtype=i32), torch.zeros(2, dtype=i32),
                             torch.zeros(3, dtype=i32))
    table = torch.zeros(3, 4, dtype=i32).as_subclass(Fake)
    with pytest.raises(ValueError, match="lengths must have shape"):
        ress.ress_cache_plan(off, off[:2], table, off, off[:1], 64, 9)
    with pytest.raises(ValueError, match="cursor must have shape"):
        ress.ress_cache_plan(off, off, table, off, off, 64, 9)


def test_compiled_calls_leave_to_python_what_is_not_common(ress):
    """The C++ part of the binding takes CUDA tensors of the right kind alone, and
    says None to everything else, whatever it is given."""
    assert ress._call is not None
    q, k = torch.zeros(10, 4, 64, dtype=torch.bfloat16), torch.zeros(20, 2, 64, dtype=torch.bfloat16)
    cache = ress.make_cache(4, 2, 64, device="cpu")
    i32 = torch.zeros(3, dtype=torch.int32)
    for f, args in ((ress._call.cross_attn, (q, k, k, None, None, None, None, True)),
                    (ress._call.cross_attn_bwd, (q, k, k, None, None, None, None, q, q, q)),
                    (ress._call.cache_plan, (i32, i32, i32[:, None], i32, i32[:1], 64, 5, None)),
                    (ress._call.cache_append, (k, k, i32, *cache)),
                    (ress._call.cache_attn, (q, *cache, i32[:, None], i32, i32, 0, True))):
        assert f(*args) is None
        assert f() is None and f(*args[:-1]) is None and f(*args, 1) is None
        for i in range(len(args)):
            for x in (None, 3, -1, 2 ** 70, "x", q.numpy if i % 2 else [q]):
                assert f(*args[:i], x, *args[i + 1:]) is None
