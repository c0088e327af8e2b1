"""new_paged_carry."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("default", [torch.float32, torch.bfloat16, torch.float64])
def test_carries_are_fp32_whatever_the_default_type(lib, default):
    cache = lib.new_paged_cache(3, 2, 4, Hq=4, Hkv=2, d=64, page=16, dtype=torch.bfloat16, fox=True)
    before = torch.get_default_dtype()
    torch.set_default_dtype(default)
    try:
        carry, gates = lib.new_paged_carry(cache)
    finally:
        torch.set_default_dtype(before)
    assert carry.dtype == gates.dtype == torch.float32
    assert torch.equal(carry, torch.eye(64, device="cuda").expand(3, 2, 64, 64)) and carry.is_contiguous()
    assert torch.equal(gates, torch.zeros((3, 4), device="cuda"))
