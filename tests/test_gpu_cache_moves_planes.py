"""Compaction of caches without elements: lengths only, as for any other cache."""
import pytest
import torch

import paged_kv_cache_267_gb300 as pa
from test_gpu_cache_moves import ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(0, 8, 2, 16, 64), (3, 8, 0, 16, 64), (3, 8, 2, 16, 0), (8, 0, 16, 64), (8, 2, 16, 0)])
def test_compact_without_elements(shape):
    """Lists with a gap over caches of no layers, no heads, no elements: nothing to move, nothing to flag."""
    kc, vc = (torch.empty(shape, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    tokens = ints([-1, -1])
    args = (ints([20, 30]), ints([0, 6, 12]), ints([[1, 3], [0, 5]]), ints([2, 2]))
    lens = pa.compact_cache(kc, vc, ints([[1, 2], [4, 5]]), *args, block_size=16, kept_tokens=tokens)
    assert pa.check_device_error() == 0
    assert lens.tolist() == [16, 26] and tokens.tolist() == [16, 32]
    # a list or a table that is wrong is flagged all the same
    lens = pa.compact_cache(kc, vc, ints([[1, 2], [4, 5]]), ints([20, 30]), ints([0, 6, 12]), ints([[3, 1], [0, 5]]), ints([2, 2]),
                            block_size=16)
    assert pa.check_device_error() == pa.DEVERR_QUERY and lens.tolist() == [20, 26]
    lens = pa.compact_cache(kc, vc, ints([[1, 8], [4, 5]]), *args, block_size=16)
    assert pa.check_device_error() == pa.DEVERR_BLOCK_ID and lens.tolist() == [16, 26]


def test_compact_in_an_empty_pool():
    """No blocks: every entry of a table is outside of the pool."""
    kc, vc = (torch.empty(0, 2, 16, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    lens = pa.compact_cache(kc, vc, ints([[0, 1]]), ints([20]), ints([0, 6]), ints([[1, 3]]), ints([2]), block_size=16)
    assert pa.check_device_error() == pa.DEVERR_BLOCK_ID and lens.tolist() == [16]
    lens = pa.compact_cache(kc, vc, ints([[-1, -1]]), ints([20]), ints([0, 6]), ints([[0, 1]]), ints([2]), block_size=16)
    assert pa.check_device_error() == 0 and lens.tolist() == [16]
