"""Rope and append at the most tokens that a call may have."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def splash():
    from block_sparse_flash_gb300 import build as b
    b.build()
    import block_sparse_flash_gb300 as m
    return m


@pytest.mark.parametrize("d", [16, 48])
def test_the_most_tokens_of_a_call(splash, d):
    """2^31 - 1 tokens, all padding and all the same row: nothing to store, so
    that they need no memory; the last value of the range that is accepted."""
    B = 2 ** 31 - 1
    k = torch.ones(1, 1, 1, d, dtype=torch.bfloat16, device="cuda").expand(B, 1, 1, d)
    cache = torch.zeros(1, 1, 16, d, dtype=torch.bfloat16, device="cuda")
    bt = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    pos = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    splash.paged_append(k, k, cache, cache.clone(), bt, pos, seq_ids=torch.zeros_like(pos))
    splash.check_device_error()
    assert not cache.any()
