"""The page calls at their largest counts and sizes."""
import pytest
import torch

from tests import paged_cases as pc

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


def test_fork_of_a_page_of_two_gigabytes(lib):
    """A page of 2^31 bytes: 16,384 heads of 256 positions."""
    H, d, page = 16384, 128, 256
    c = lib.new_paged_cache(2, 1, 2, 1, Hq=H, d=d, page=page, dtype=torch.float32)
    c.k_pages[0].normal_()
    c.k_pages[1].fill_(float("nan"))
    c.k_table[0, 0] = c.v_table[0, 0] = 0
    c.k_ref[0] = c.v_ref[0] = 1
    c.lens[0] = page
    ws = lib.new_paged_workspace(c)
    lib.path_paged_fork([0], [1], c, workspace=ws)
    assert lib.path_check_workspace(ws) == lib.OK
    assert c.k_table.tolist() == [[0], [1]] and c.v_table.tolist() == [[0], [0]]
    assert torch.equal(c.k_pages[1], c.k_pages[0])


def test_long_lists_of_rows(lib):
    """Lists past the short form of the page calls' parameters."""
    n = 300
    c = lib.new_paged_cache(2 * n, 3, 5 * n, Hq=1, page=16, d=64)
    ws = lib.new_paged_workspace(c)
    lens = torch.tensor([1 + (7 * s) % 40 for s in range(n)] + [0] * n, dtype=torch.int32, device="cuda")
    lib.path_paged_reserve(lens, c, workspace=ws)
    c.lens.copy_(lens)
    c.k_pages.normal_()
    c.v_pages.normal_()
    lib.path_paged_fork(list(range(n)), list(range(2 * n - 1, n - 1, -1)), c, workspace=ws)
    assert lib.path_check_workspace(ws) == lib.OK
    for s in (0, 1, 31, 32, 33, n - 1):
        t, m = 2 * n - 1 - s, int(lens[s])
        assert int(c.lens[t]) == m
        for pool, table in ((c.k_pages, c.k_table), (c.v_pages, c.v_table)):
            assert torch.equal(pc.rows_of(pool, table[s], m), pc.rows_of(pool, table[t], m))
    lib.path_paged_free(list(range(n)), c, workspace=ws)
    assert int((c.v_ref > 0).sum()) == int((c.v_table[n:] >= 0).sum()) and (c.k_table[:n] == -1).all()
    lib.path_paged_free(list(range(n, 2 * n)), c, workspace=ws)
    assert not c.k_ref.any() and not c.v_ref.any() and lib.path_check_workspace(ws) == lib.OK
