"""Workspaces of the paged calls, on the GPU: what is refused, and who learns of their status."""
import pytest
import torch

from tests import paged_cases as pc

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def test_workspaces_that_are_not_the_calls(lib):
    x = pc.make([20, 5], [1, 1], 2, 2, 64, 16, BF, False, seed=45)
    c = pc.cache_of(lib, x)
    n = lib.path_paged_workspace_bytes(c, 2, 1, Hq=2)
    for ws in (torch.zeros(n, dtype=torch.uint8), torch.zeros(n, dtype=torch.uint8).pin_memory()):
        with pytest.raises(TypeError, match="workspace"):
            pc.step(lib, x, c, workspace=ws)
        with pytest.raises(TypeError, match="workspace"):
            lib.path_paged_compact(c, workspace=ws)


def test_page_calls_without_a_workspace_raise(lib):
    """Without a workspace whose status word the caller could read, what the device finds is raised."""
    c = lib.new_paged_cache(3, 8, 4, Hq=1, page=16)
    lib.path_paged_reserve(torch.tensor([40, 0, 0], dtype=torch.int32, device="cuda"), c)
    c.lens[0] = 40
    with pytest.raises(lib.PathError) as e:
        lib.path_paged_reserve(torch.tensor([0, 32, 0], dtype=torch.int32, device="cuda"), c)
    assert e.value.code == lib.ERR_CAPACITY
    with pytest.raises(lib.PathError) as e:
        lib.path_paged_fork([0], [1], c)
    assert e.value.code == lib.ERR_CAPACITY
    c.k_table[0, 7] = 99
    with pytest.raises(lib.PathError) as e:
        lib.path_paged_compact(c)
    assert e.value.code == lib.ERR_CACHE
    with pytest.raises(lib.PathError) as e:
        lib.path_paged_free([0], c)
    assert e.value.code == lib.ERR_CACHE
    assert not c.k_ref.any() and not c.v_ref.any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("chunks", [[1, 1], [70, 3]])
def test_a_step_without_a_workspace_raises(lib, dtype, chunks):
    x = pc.make([20, 5], chunks, 2, 2, 64, 16, dtype, False, seed=46)
    x["v_table"][1, 0] = -1  # a page that was never mapped
    with pytest.raises(lib.PathError) as e:
        pc.step(lib, x)
    assert e.value.code == lib.ERR_CACHE


def test_a_captured_page_call_gives_its_workspace(lib):
    """In a capture nothing can be waited for: the call's workspace is returned, and its status word
    holds what the last replay found."""
    c = lib.new_paged_cache(1, 4, 2, Hq=1, page=16)
    extra = torch.tensor([16], dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ws = lib.path_paged_reserve(extra, c)
        c.lens += extra
    for turn in range(2):
        g.replay()
        assert lib.path_check_workspace(ws) == lib.OK
    g.replay()
    assert lib.path_check_workspace(ws) == lib.ERR_CAPACITY
