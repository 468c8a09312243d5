"""Calls of the block-sparse decode at the ends of what they accept."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B(lib):
    from paged_kv_cache_317_gb300 import binding
    return binding


@pytest.mark.parametrize("width", [40, 20000])
def test_the_longest_list(B, width):
    """2^31 - 1 places for a few blocks: the index over the places must not wrap."""
    most = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of free device memory")
    lens = torch.tensor([5], dtype=torch.int32, device="cuda")
    out = torch.zeros((1, 1, most), dtype=torch.int32, device="cuda")
    B.paged_block_select(torch.zeros((1, 1, width), device="cuda"), lens, 1, most, out=out)
    torch.cuda.synchronize()
    assert out[0, 0, :5].tolist() == [0, 1, 2, 3, 4]
    for part in out[0, 0, 5:].split(1 << 28):
        assert bool((part == -1).all())
