"""The paged calls' workspaces, on the CPU."""
import pytest
import torch

import dependent_position_encoded_gb300 as pa
from tests.test_paged_checks import _c, _cache, _step


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


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (4, 1), (8, 1), (3, 1), (16, 2), (48, 16)])
def test_a_workspace_serves_every_smaller_step(lib, dtype, hq, hkv):
    so = lib._load()
    sizes = (1, 2, 3, 16, 17, 32, 33, 63, 64, 65, 128, 129, 512, 513, 1000, 20000)
    for d in (64, 128):
        for seqs in (1, 5, 300):
            for slots in (0, 1, 40, 2048):
                c = _c(dtype=dtype, Hq=hq, Hkv=hkv, seqs=seqs, max_pages=slots, d=d)
                bytes_of = {(n, t): so.path_paged_workspace_bytes(c, n, t)
                            for n in sizes for t in sizes if t <= n}
                # running maxima over the chunks, then over the tokens
                most = {}
                for (n, t) in sorted(bytes_of):
                    i, j = sizes.index(n), sizes.index(t)
                    below = [most.get((sizes[i - 1], t), 0) if i else 0, most[n, sizes[j - 1]] if j else 0]
                    assert bytes_of[n, t] > 256 and bytes_of[n, t] >= max(below), (d, seqs, slots, n, t)
                    most[n, t] = max(below + [bytes_of[n, t]])
                big = so.path_paged_workspace_bytes(c, 1000, 513)
                assert big >= so.path_paged_workspace_bytes(c, 0, 0)
