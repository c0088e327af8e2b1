"""NaN in cached and in new keys."""
import pytest
import torch

from tests import paged_cases as pc

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("Hq,Hkv,chunks", [
    (2, 2, [1, 1]),        # one pass
    (3, 1, [1, 1]),        # block kernels
    (2, 2, [5, 1]),
    (4, 2, [150, 70]),     # several blocks
])
@pytest.mark.parametrize("at", [0, 77])
def test_a_nan_in_a_cached_key_reaches_the_outputs(lib, dtype, fox, Hq, Hkv, chunks, at):
    """A key that is not a number makes its head's rows NaN, as the formula does, and leaves the other
    heads and sequences as they are."""
    x = pc.make([90, 40], chunks, Hq, Hkv, 64, 16, dtype, fox, seed=41)
    x["k_pages"][x["k_table"][0, at // 16].long(), 0, at % 16, 3] = NAN
    ref = pc.reference(x)[0]
    out = pc.step(lib, x)
    G = Hq // Hkv
    assert out[:chunks[0], :G].isnan().all()
    for a, b in ((out[:chunks[0], G:], ref[:chunks[0], G:]), (out[chunks[0]:], ref[chunks[0]:])):
        pc.close(a, b, dtype, "out")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fox", [False, True])
def test_a_nan_in_a_new_key_reaches_the_rows_behind_it(lib, dtype, fox):
    x = pc.make([30], [200], 4, 2, 64, 16, dtype, fox, seed=42)
    x["k"][20, 1, 5] = NAN
    if fox:
        x["log_f"][40:, 2:] = -3.0  # closed long before the last rows
    ref = pc.reference(x)[0]
    out = pc.step(lib, x)
    assert out[20:, 2:].isnan().all()
    pc.close(out[:, :2], ref[:, :2], dtype, "out")
    pc.close(out[:20, 2:], ref[:20, 2:], dtype, "out")
