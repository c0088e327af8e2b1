"""The page calls at their largest counts and sizes."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_reserve_of_more_pages_than_an_int_counts(lib):
    """2^31 missing slots in all: more than any pool has, so nothing changes."""
    seqs, slots = 8192, 1 << 18
    c = lib.new_paged_cache(seqs, slots, 16, Hq=1, page=16)
    ws = lib.new_paged_workspace(c)
    extra = torch.full((seqs,), slots * 16, dtype=torch.int32, device="cuda")
    lib.path_paged_reserve(extra, c, workspace=ws)
    assert lib.path_check_workspace(ws) == lib.ERR_CAPACITY
    assert not c.k_ref.any() and not c.v_ref.any()
    assert int(c.k_table.max()) == -1 and int(c.v_table.max()) == -1
