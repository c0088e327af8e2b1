"""Numbers that no C int holds, whose low bits a call would take, on the CPU: refused before any launch."""
import pytest
import torch

import dependent_position_encoded_gb300 as pa
from tests.test_paged_checks import D, HKV, HQ, S, _cache, _step


def _calls(most):
    gated, plain = list(_step().values()), [x for n, x in _step().items() if n != "log_f"]
    prefix = (torch.full((S,), -1, dtype=torch.int32), torch.zeros(S, HKV, D, D))
    return [lambda: pa.path_paged_extend(*plain, _cache(), most),
            lambda: pa.path_fox_paged_extend(*gated, _cache(), most),
            lambda: pa.path_paged_window_extend(*plain, _cache(), most, 8, 1),
            lambda: pa.path_fox_paged_window_extend(*gated, _cache(), most, 8, 1),
            lambda: pa.path_paged_prefix_extend(*plain, _cache(), *prefix, most),
            lambda: pa.path_fox_paged_prefix_extend(*gated, _cache(), *prefix, torch.zeros(S, HQ), most)]


@pytest.mark.parametrize("most", [2 ** 32 + 1, 2 ** 31, -2 ** 32 + 2, -2 ** 31 - 1])
@pytest.mark.parametrize("call", range(6))
def test_max_chunk(most, call):
    with pytest.raises(ValueError, match="32-bit"):
        _calls(most)[call]()


@pytest.mark.parametrize("call", range(6))
def test_numbers_that_fit_go_on_to_the_next_check(call):
    with pytest.raises(TypeError, match="CUDA"):
        _calls(2)[call]()
