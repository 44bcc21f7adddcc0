"""Sizes and numbers at the ends of what the cache operators take, refused on the
host before any CUDA call (no GPU needed)."""

import ctypes

import pytest
import torch

from block_sparse_global_mean_b200 import build as ress_build

FAKE = 0x10000          # 16-byte aligned, never dereferenced

no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(),
                                 reason="placeholder-pointer cases run only without a GPU")


@pytest.fixture(scope="module")
def ress():
    ress_build.build()
    from block_sparse_global_mean_b200 import ress as mod
    return mod


@no_gpu_only
@pytest.mark.parametrize("tokens", [2 ** 30 + 1, 2 ** 31 - 1])
def test_plan_refuses_a_slot_map_beyond_its_limit(tokens, ress):
    """Beyond 2^30 tokens no attention call takes the rows, and positions that step
    by the size of the grid come near 2^31."""
    sh = ctypes.byref(ress.ress_cache_shape(10, 64, 1, 64, 3, 5))
    assert ress.lib.ress_cache_plan(sh, FAKE, FAKE, FAKE, FAKE, 5, FAKE, tokens, FAKE + 64,
                                    FAKE + 64, FAKE + 64, FAKE + 64,
                                    None) == ress.RESS_ERR_UNSUPPORTED


class Fake(torch.Tensor):
    """A host tensor that says it is on a device, to reach the later checks."""
    is_cuda = True


def _on_device(*ts):
    return [t.as_subclass(Fake) for t in ts]


@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32 + 1, 2 ** 32 + 64, -2 ** 31 - 1])
def test_binding_refuses_numbers_beyond_32_bits(big, ress):
    """ctypes would cut them: a step of 2^32 + 1 to a causal mask, a page of 2^32 + 64
    to one of 64 tokens."""
    i32 = torch.int32
    cache = ress.ress_cache(*_on_device(*ress.make_cache(4, 2, 64, device="cpu")))
    q, table, one, two = _on_device(torch.zeros(3, 2, 64, dtype=torch.bfloat16),
                                    torch.zeros(1, 3, dtype=i32), torch.zeros(1, dtype=i32),
                                    torch.zeros(2, dtype=i32))
    with pytest.raises(ValueError, match="step must fit"):
        ress.ress_cache_attn(q, cache, table, one, two, step=big)
    with pytest.raises(ValueError, match="page must fit"):
        ress.ress_cache_plan(one, one, table, two, one, big, 5)
    with pytest.raises(ValueError, match="tokens must fit"):
        ress.ress_cache_plan(one, one, table, two, one, 64, big)
    if big > 0:
        with pytest.raises(ValueError, match="pages must fit"):
            ress.ress_cache_plan(one, one, table, two, one, 64, 5, pages=big)
        with pytest.raises(ValueError, match="pages must fit"):
            ress._cache_shape(big, 64, 2, 64, 1, 1)
        with pytest.raises(ValueError, match="max_pages must fit"):
            ress._cache_shape(4, 64, 2, 64, 1, big)
        with pytest.raises(ValueError, match="sequences must fit"):
            ress._cross_shape(1, 1, big, 2, 2, 64, 0, 0, 0)


def test_binding_refuses_numbers_that_are_no_integers(ress):
    i32 = torch.int32
    cache = ress.ress_cache(*_on_device(*ress.make_cache(4, 2, 64, device="cpu")))
    q, table, one, two = _on_device(torch.zeros(3, 2, 64, dtype=torch.bfloat16),
                                    torch.zeros(1, 3, dtype=i32), torch.zeros(1, dtype=i32),
                                    torch.zeros(2, dtype=i32))
    with pytest.raises(TypeError):
        ress.ress_cache_attn(q, cache, table, one, two, step=1.5)
    with pytest.raises(TypeError):
        ress.ress_cache_plan(one, one, table, two, one, 64.5, 5)


def test_binding_refuses_a_negative_slot_map(ress):
    table, one, two = _on_device(torch.zeros(1, 3, dtype=torch.int32),
                                 torch.zeros(1, dtype=torch.int32),
                                 torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="tokens must not be negative"):
        ress.ress_cache_plan(one, one, table, two, one, 64, -5)
