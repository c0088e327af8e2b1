"""Steps over caches one of whose pools has no pages."""
import ctypes

import pytest
import torch

from tests import paged_cases as pc

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("chunks", [[1, 1], [70, 3]])
@pytest.mark.parametrize("Hq", [2, 6])
@pytest.mark.parametrize("empty", ["num_k_pages", "num_v_pages"])
def test_positions_of_an_empty_pool_are_absent(lib, dtype, chunks, Hq, empty):
    """A pool of no pages: every position counts as absent, whatever the tables say, and the status
    word says so; the new tokens still attend to each other."""
    x = pc.make([300, 40], chunks, Hq, 2, 64, 16, dtype, False, seed=43)
    so = lib._load()
    ws = lib.new_paged_workspace(pc.cache_of(lib, x), sum(chunks), max(chunks), Hq=Hq)
    ws[256:] = 0x3f  # what an earlier call may have left: parts of ordinary size
    c = lib._CPagedCache(*[x[n].data_ptr() if x[n] is not None else None
                           for n in ("k_pages", "v_pages", "g_pages", "k_table", "v_table", "k_ref",
                                     "v_ref", "lens")], 2, x["k_table"].shape[1], 16,
                         x["k_pages"].shape[0], x["v_pages"].shape[0], Hq, 2, 64,
                         lib.BF16 if dtype == BF else lib.F32)
    setattr(c, empty, 0)
    before = pc.snapshot(x)
    out = torch.full_like(x["q"], 7.0)
    assert so.path_paged_extend(
        ctypes.byref(c), *[x[n].data_ptr() for n in ("q", "k", "v", "w", "beta", "cu")], sum(chunks),
        max(chunks), 0.125, out.data_ptr(), None, ws.data_ptr(), ws.numel(),
        torch.cuda.current_stream().cuda_stream) == lib.OK
    assert lib.path_check_workspace(ws) == lib.ERR_CACHE
    ref = pc.reference(dict(x, n=[0, 0], **before))[0]
    pc.close(out, ref, dtype, "out")
    pool = "k_pages" if empty == "num_k_pages" else "v_pages"
    assert torch.equal(x[pool].nan_to_num(nan=7.0), before[pool].nan_to_num(nan=7.0))
