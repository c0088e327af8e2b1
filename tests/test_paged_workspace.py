"""The paged calls' workspaces, on the CPU."""
import pytest
import torch

import dependent_position_encoded_gb300 as pa
from tests.test_paged_checks import _cache, _step


@pytest.mark.parametrize("ws", [
    object(), torch.zeros(1 << 20), torch.zeros(2, 1 << 20, dtype=torch.uint8).t(),
    torch.zeros(1 << 20, dtype=torch.uint8),
])
def test_workspaces_are_checked(ws):
    for call in (lambda: pa.path_fox_paged_extend(*_step().values(), _cache(), 2, workspace=ws),
                 lambda: pa.path_paged_compact(_cache(), workspace=ws),
                 lambda: pa.path_paged_free([0], _cache(), workspace=ws),
                 lambda: pa.path_paged_fork([0], [1], _cache(), workspace=ws)):
        with pytest.raises((TypeError, ValueError), match="workspace"):
            call()
