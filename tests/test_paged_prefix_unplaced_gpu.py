"""Steps behind shared prefixes whose cu_tokens falls, with a sequence that gets no place among its
prefix's tokens: what a workspace held before the call has no part in any result, and the sequence's
carry stays as it was."""
import pytest
import torch

from tests import paged_cases as pc
from tests import paged_prefix_cases as px
from tests.paged_window_cases import same_bits

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(params=[
    ([0, 0, 5, 2, 3], 1),        # the last sequence: one token, from before an earlier one's end
    ([0, 0, 50, 20, 30], 12),    # ten of them
    ([0, 0, 200, 20, 120], 130),
], ids=["one", "ten", "blocks"])
def unplaced(request):
    """Row 1 brings more tokens than the step takes, row 2's range falls, row 3 lies behind both, so that no
    row has a place: (inputs, cache, workspace, the step)."""
    cu, most = request.param

    def build(lib, dtype, fox, d):
        x = px.make([300, 40, 0, 129], [0, 1, 1, most], [-1, 0, 0, 0], 4, 2, d, 16, dtype, fox, seed=1,
                    tail=max(cu), width=-(-(300 + most) // 16))
        cache = pc.cache_of(lib, x)
        ws = lib.new_paged_workspace(cache, x["q"].shape[0], most, Hq=4, prefix=True)
        x["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        return x, cache, ws, lambda **kw: px.step(lib, dict(x, chunks=[most]), cache, workspace=ws, **kw)

    return build


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_outputs_without_a_place(lib, unplaced, dtype, fox, d):
    x, _, ws, step = unplaced(lib, dtype, fox, d)
    before, first = px.snapshot(x), None
    for fill in (0, 0x3F, 0xFF):  # 0.75 and NaN in fp32
        for n in before:
            if x[n] is not None:
                x[n].copy_(before[n])
        ws[256:] = fill
        out = torch.full_like(x["q"], 7.0)
        step(out=out)
        assert lib.path_check_workspace(ws) == lib.ERR_CACHE
        first = out.clone() if first is None else first
        assert same_bits(out, first)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_carries_without_a_place(lib, unplaced, dtype, fox, d):
    x, _, ws, step = unplaced(lib, dtype, fox, d)
    before = px.snapshot(x)
    step()
    assert lib.path_check_workspace(ws) == lib.ERR_CACHE
    assert torch.equal(x["carry"], before["carry"])
    assert not fox or torch.equal(x["gate_carry"], before["gate_carry"])
