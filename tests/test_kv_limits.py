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
