"""Steps behind prefixes: idle rows that name anything, prefixes with a page that is not mapped; chunks on
pools past 2^31 elements, behind prefixes and through windows."""
import pytest
import torch

from tests import paged_cases as pc
from tests import paged_prefix_cases as px
from tests import paged_window_cases as wc

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 5, 70])
@pytest.mark.parametrize("name", [1 << 30, 2 ** 31 - 1, 6, 1, 0, -2 ** 31])
def test_idle_rows_that_name_anything(lib, dtype, T, name):
    # rows 1, 3 and 5 have no tokens and are nobody's prefix
    x = px.make([100, 20, 30, 0, 5, 17], [0, 0, T, 0, T, 0], [-1, name, 0, name, -1, name], 4, 2, 64, 16, dtype, True,
                seed=1)
    before = px.snapshot(x)
    ws = lib.new_paged_workspace(pc.cache_of(lib, x), 2 * T, T, Hq=4, prefix=True)
    out = px.step(lib, x, workspace=ws)
    assert lib.path_check_workspace(ws) == lib.OK
    px.check(x, before, out)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("T", [1, 3, 80])
@pytest.mark.parametrize("d,page,slot", [(64, 16, 3), (64, 64, 0), (128, 128, 1)])
@pytest.mark.parametrize("pools", ["k", "v", "kv"])
def test_positions_of_a_page_that_is_not_mapped_are_absent(lib, dtype, fox, T, d, page, slot, pools):
    """Logits with a prefix's keys go by the carry alone, whatever their positions, so what is left of it counts
    as a prefix that is shorter by that page."""
    n = 5 * page + 9
    x = px.make([n, 9, 70, 0], [0, T, T, T], [-1, 0, -1, 0], 4, 2, d, page, dtype, fox, seed=2)
    y = {a: b.clone() if isinstance(b, torch.Tensor) else b for a, b in x.items()}
    y["n"] = [n - page] + x["n"][1:]
    for a in "kv":
        row = y[a + "_table"][0]
        row[slot:-1] = x[a + "_table"][0, slot + 1:]
        row[-1] = -1
        if a in pools:
            x[a + "_table"][0, slot] = -1
    ws = lib.new_paged_workspace(pc.cache_of(lib, x), 3 * T, T, Hq=4, prefix=True)
    out = px.step(lib, x, workspace=ws)
    assert lib.path_check_workspace(ws) == lib.ERR_CACHE
    ref = px.reference(y)
    pc.close(out, ref[0], dtype, "out")
    for s in (1, 3):
        # as paged_prefix_cases.check has it
        err = (x["carry"][s].double() - ref[4][s]).norm(dim=-1) / y["carry"][s].double().norm(dim=-1).clamp(min=1e-3)
        assert float(err.max()) <= 8 * 2.0 ** -24 * T ** 0.5 + 2.0 ** -22


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["prefix", "window"])
@pytest.mark.parametrize("chunks", [[3, 7, 0], [70, 1, 130]])
def test_chunks_on_pools_past_2_31_elements(lib, dtype, kind, chunks):
    page, Hkv, d, far = 64, 16, 64, 34000  # 65,536 elements a page
    if kind == "prefix":
        x = px.make([500, 3, 0, 90], [0] + chunks, [-1, 0, 0, 0], 16, Hkv, d, page, dtype, True, seed=3, width=12)
    else:
        x = pc.make([500, 3, 900], chunks, 16, Hkv, d, page, dtype, True, seed=3, width=18)
    for a in "kv":
        n = x[a + "_pages"].shape[0]
        for name in (a + "_pages", "g_pages") if a == "k" else (a + "_pages",):
            big = torch.empty((far + n, *x[name].shape[1:]), dtype=x[name].dtype, device="cuda")
            big[far:] = x[name]
            big[:far] = 7.0
            x[name] = big
        t = x[a + "_table"]
        t[t >= 0] += far
        x[a + "_ref"] = torch.cat([x[a + "_ref"].new_zeros(far), x[a + "_ref"]])
    assert x["k_pages"].numel() > 2 ** 31
    if kind == "prefix":
        before = px.snapshot(x)
        out = px.step(lib, x)
        torch.cuda.synchronize()
        px.check(x, before, out)
    else:
        before = wc.snapshot(x)
        out = wc.window_step(lib, x, pc.cache_of(lib, x), 200, 4)
        torch.cuda.synchronize()
        wc.check_window(x, before, out, 200, 4)
    del x, before, out
    torch.cuda.empty_cache()
