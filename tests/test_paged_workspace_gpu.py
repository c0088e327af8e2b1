"""Workspaces of the paged calls, on the GPU."""
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
