"""Trimming of named rows: what it refuses (on the CPU, before any launch), and that the rows which it does
not name keep everything."""
import ctypes

import pytest
import torch

import dependent_position_encoded_gb300 as pa
from tests import paged_cases as pc
from tests import paged_prefix_cases as px
from tests import paged_window_cases as wc
from tests.test_paged_checks import FAKE, _c, _cache, no_gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def so():
    pa.ensure_built()
    return pa._load()


@no_gpu
@pytest.mark.parametrize("rows,count,window,sinks,cache,code", [
    ([1, 1], 2, 8, 0, {}, pa.ERR_ARG),
    ([3], 1, 8, 0, {}, pa.ERR_ARG),               # no row of the cache
    ([-1], 1, 8, 0, {}, pa.ERR_ARG),
    ([0] * 1025, 1025, 8, 0, {}, pa.ERR_SHAPE),
    (None, 1, 8, 0, {}, pa.ERR_NULL),
    ([0], -1, 8, 0, {}, pa.ERR_SHAPE),
    ([0], 1, 0, 0, {}, pa.ERR_ARG),
    ([0], 1, 8, -1, {}, pa.ERR_ARG),
    (None, 0, 0, 0, {}, pa.ERR_ARG),
    ([0], 1, 8, 0, dict(k_ref=None), pa.ERR_NULL),
    ([0], 1, 8, 0, dict(v_ref=FAKE + 4), pa.ERR_ALIGN),
    ([0], 1, 8, 0, dict(page=24), pa.ERR_SHAPE),
    (None, 0, 8, 0, {}, pa.OK),
    ([0], 1, 8, 0, dict(max_pages=0), pa.OK),
])
def test_arguments(so, rows, count, window, sinks, cache, code):
    a = None if rows is None else (ctypes.c_int * len(rows))(*rows)
    assert so.path_paged_trim_rows(_c(**cache), a, count, window, sinks, FAKE, 1 << 30, None) == code


@no_gpu
def test_workspace(so):
    need, a = so.path_paged_workspace_bytes(_c(), 0, 0), (ctypes.c_int * 1)(0)
    assert so.path_paged_trim_rows(_c(), a, 1, 8, 0, FAKE, need - 1, None) == pa.ERR_WORKSPACE
    assert so.path_paged_trim_rows(_c(), a, 1, 8, 0, None, need, None) == pa.ERR_NULL


def test_the_package_refuses():
    with pytest.raises(TypeError, match="CUDA"):
        pa.path_paged_trim(_cache(), 8, 1, rows=[0])
    with pytest.raises(ValueError, match="32-bit"):
        pa.path_paged_trim(_cache(), 2 ** 32 + 8, 1, rows=[0])


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("count", [0, 1, 3, 32, 33, 200])
def test_other_rows_keep_everything(lib, page, count):
    lens = [(37 * i) % 700 for i in range(300)]
    x = pc.make(lens, [0] * 300, 1, 1, 64, page, BF, False, seed=1)
    cache = pc.cache_of(lib, x)
    names = ("k_table", "v_table", "k_ref", "v_ref", "lens")
    before = {n: getattr(cache, n).clone() for n in names}
    rows = torch.randperm(300, generator=torch.Generator().manual_seed(2))[:count].tolist()
    lib.path_paged_trim(cache, 100, 4, rows=rows)
    for a in "kv":
        table, lens2, left = before[a + "_table"].tolist(), list(lens), []
        for s in rows:
            (row,), (n,), gone = wc.trimmed([table[s]], [lens[s]], 100, 4, page)
            table[s], lens2[s], left = row, n, left + gone
        ref = before[a + "_ref"].clone()
        ref[torch.tensor(left, dtype=torch.long, device="cuda")] = 0
        assert getattr(cache, a + "_table").tolist() == table
        assert torch.equal(getattr(cache, a + "_ref"), ref)
    assert cache.lens.tolist() == lens2


@pytest.mark.gpu
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("T", [1, 9])
def test_streams_beside_prefixes(lib, dtype, fox, T):
    """A stream that is trimmed beside a prefix and a sequence behind it, both longer than the window, in one
    captured graph: the other two give the reference's outputs."""
    x = px.make([500, 300, 400], [0, T, 0], [-1, 0, -1], 4, 2, 64, 16, dtype, fox, seed=3)
    before, cache = px.snapshot(x), pc.cache_of(lib, x)
    was = {n: getattr(cache, n).clone() for n in ("k_table", "v_table", "k_ref", "v_ref", "lens")}
    ws = lib.new_paged_workspace(cache, T, T, Hq=4, prefix=True)
    lib.path_paged_trim(cache, 100, 4, workspace=ws, rows=[])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.path_paged_trim(cache, 100, 4, workspace=ws, rows=[2])
    g.replay()
    gone = (401 - 100) // 16 - 1
    assert cache.lens.tolist() == [500, 300, 400 - 16 * gone]
    for n in ("k_table", "v_table"):
        assert torch.equal(getattr(cache, n)[:2], was[n][:2])
    for n in ("k_ref", "v_ref"):
        assert int(getattr(cache, n).sum()) == int(was[n].sum()) - gone
    out = px.step(lib, x, cache, workspace=ws)
    assert lib.path_check_workspace(ws) == lib.OK
    x["k_table"].copy_(was["k_table"])  # (the check reads the stream's row too, whose pages nobody has taken)
    x["v_table"].copy_(was["v_table"])
    px.check(x, before, out)
