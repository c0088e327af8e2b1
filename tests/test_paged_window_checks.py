"""What the window calls and trimming refuse, on the CPU: all before any launch."""
import pytest
import torch

import dependent_position_encoded_gb300 as pa
from tests.test_paged_checks import FAKE, HQ, N, S, _c, _cache, _step, no_gpu


@pytest.mark.parametrize("kw,exc", [
    (dict(q=torch.zeros(N, HQ, 64)), TypeError),
    (dict(beta=torch.zeros(N, HQ)), ValueError),
    (dict(log_f=None), TypeError),
    (dict(cu_tokens=torch.zeros(S, dtype=torch.int32)), ValueError),
])
def test_step_errors_raise_before_any_call(kw, exc):
    with pytest.raises(exc):
        pa.path_fox_paged_window_extend(*_step(**kw).values(), _cache(), 2, 8, 1)


def test_host_tensors_need_a_gpu():
    with pytest.raises(TypeError, match="CUDA"):
        pa.path_fox_paged_window_extend(*_step().values(), _cache(), 2, 8, 1)
    with pytest.raises(TypeError, match="CUDA"):
        pa.path_paged_trim(_cache(), 8, 1)
    with pytest.raises(TypeError):
        pa.path_fox_paged_window_extend(*_step().values(), _cache(g_pages=None), 2, 8, 1)


@pytest.fixture(scope="module")
def so():
    pa.ensure_built()
    return pa._load()


def _window(so, cache, fox, window, sinks, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, w=FAKE, beta=FAKE, log_f=FAKE, cu=FAKE, N=N, chunk=2,
             scale=0.125, out=FAKE, st=None, ws=FAKE, bytes=1 << 30, stream=None)
    a.update(kw)
    args = [a[n] for n in ("q", "k", "v", "w", "beta")] + ([a["log_f"]] if fox else [])
    fn = so.path_fox_paged_window_extend if fox else so.path_paged_window_extend
    return fn(cache, *args, a["cu"], a["N"], a["chunk"], window, sinks, a["scale"], a["out"], a["st"],
              a["ws"], a["bytes"], a["stream"])


@no_gpu
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("window,sinks,kw,code", [
    (0, 0, {}, pa.ERR_ARG),
    (-3, 0, {}, pa.ERR_ARG),
    (8, -1, {}, pa.ERR_ARG),
    ((1 << 22) + 1, 0, {}, pa.ERR_ARG),
    (8, (1 << 22) + 1, {}, pa.ERR_ARG),
    (1, 4, {}, pa.ERR_ARG),                      # a chunk longer than the window
    (8, 4, dict(chunk=0), pa.ERR_SHAPE),
    (8, 4, dict(q=None), pa.ERR_NULL),
    (8, 4, dict(q=FAKE + 2), pa.ERR_ALIGN),
    (8, 4, dict(ws=None), pa.ERR_NULL),
    (8, 4, dict(bytes=256), pa.ERR_WORKSPACE),
    (8, 4, dict(N=0, chunk=0), pa.OK),
])
def test_window_arguments(so, fox, window, sinks, kw, code):
    assert _window(so, _c(), fox, window, sinks, **kw) == code


@no_gpu
@pytest.mark.parametrize("window,sinks,cache,code", [
    (0, 0, {}, pa.ERR_ARG),
    (8, -1, {}, pa.ERR_ARG),
    (8, 0, dict(k_ref=None), pa.ERR_NULL),
    (8, 0, dict(page=24), pa.ERR_SHAPE),
    (8, 0, dict(v_ref=FAKE + 4), pa.ERR_ALIGN),
    (8, 0, dict(seqs=0), pa.OK),
    (8, 0, dict(max_pages=0), pa.OK),
])
def test_trim_arguments(so, window, sinks, cache, code):
    assert so.path_paged_trim(_c(**cache), window, sinks, FAKE, 1 << 30, None) == code


@no_gpu
def test_trim_needs_the_page_calls_workspace(so):
    need = so.path_paged_workspace_bytes(_c(), 0, 0)
    assert so.path_paged_trim(_c(), 8, 0, FAKE, need - 1, None) == pa.ERR_WORKSPACE
    assert so.path_paged_trim(_c(), 8, 0, None, need, None) == pa.ERR_NULL


@pytest.mark.parametrize("window,sinks", [(2 ** 32 + 8, 1), (8, 2 ** 32 + 1), (2 ** 40, 0), (-2 ** 33 + 8, 0)])
def test_numbers_that_no_int_holds(window, sinks):
    with pytest.raises(ValueError, match="32-bit"):
        pa.path_paged_window_extend(*[x for n, x in _step().items() if n != "log_f"], _cache(), 2, window, sinks)
    with pytest.raises(ValueError, match="32-bit"):
        pa.path_fox_paged_window_extend(*_step().values(), _cache(), 2, window, sinks)
    with pytest.raises(ValueError, match="32-bit"):
        pa.path_paged_trim(_cache(), window, sinks)
