"""Window and prefix steps where their kernels change hands: row tiles of every filling, more sequences
than find their places beside the plan, more query heads than a row tile holds, token ranges that
fall, pools past 2^31 elements, several graphs and streams."""
import pytest
import torch

from tests import paged_cases as pc
from tests import paged_prefix_cases as px
from tests import paged_window_cases as wc

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def prefix_run(lib, x, **kw):
    before = px.snapshot(x)
    out = px.step(lib, x, **kw)
    torch.cuda.synchronize()
    px.check(x, before, out)


def window_run(lib, x, window, sinks):
    wc.hide(x, window, sinks)
    before = wc.snapshot(x)
    out = wc.window_step(lib, x, pc.cache_of(lib, x), window, sinks)
    torch.cuda.synchronize()
    wc.check_window(x, before, out, window, sinks)


@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("d,Hq,Hkv", [(64, 8, 1), (128, 8, 1), (128, 4, 2)])
@pytest.mark.parametrize("members", [4, 5, 8, 9, 16, 17, 32, 33, 64, 65])
def test_rows_of_a_tile(lib, fox, d, Hq, Hkv, members):
    # 8 to 520 rows: four copies of them in the tile, two, one, a full tile, one more
    x = px.make([700] + [i % 5 for i in range(members)], [0] + [1] * members, [-1] + [0] * members, Hq, Hkv, d, 64,
                BF, fox, seed=1)
    prefix_run(lib, x)


@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("most", [1, 2])
@pytest.mark.parametrize("width", [4, 40])
def test_more_sequences_than_find_their_places_alone(lib, fox, most, width):
    S = 1100
    g = torch.Generator().manual_seed(2)
    of = [-1] * 20 + torch.randint(-1, 20, (S - 20,), generator=g).tolist()
    chunks = [0] * 20 + torch.randint(0, most + 1, (S - 20,), generator=g).tolist()
    x = px.make([1 + 3 * i for i in range(20)] + [i % 4 for i in range(S - 20)], chunks, of, 2, 1, 64, 16, BF, fox,
                seed=2, width=width)
    prefix_run(lib, x)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("d,Hq", [(64, 128), (64, 130), (128, 129)])
def test_more_query_heads_than_rows_of_a_tile(lib, dtype, fox, d, Hq):
    x = pc.make([300, 0, 129], [1, 1, 1], Hq, 1, d, 32, dtype, fox, seed=3)
    window_run(lib, x, 150, 3)
    x = px.make([300, 0, 129, 7], [0, 1, 1, 1], [-1, 0, 0, -1], Hq, 1, d, 32, dtype, fox, seed=4)
    prefix_run(lib, x)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("G", [12, 40])
@pytest.mark.parametrize("T", [1, 3])
def test_more_gated_heads_than_the_ring_holds(lib, dtype, G, T):
    x = pc.make([1000, 33, 0], [T, T, T], 2 * G, 2, 128, 64, dtype, True, seed=5)
    window_run(lib, x, 400, 5)
    x = px.make([1000, 33, 0], [0, T, T], [-1, 0, 0], 2 * G, 2, 64, 64, dtype, True, seed=6)
    prefix_run(lib, x)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("chunks,cu", [
    ([0, 1, 1, 1], [0, 0, 3, 1, 2]),
    ([0, 30, 100, 70], [0, 0, 200, 100, 200]),
    ([0, 20, 20, 20], [0, 0, 60, 0, 60]),  # the same tokens for two sequences
])
def test_token_ranges_that_fall(lib, dtype, fox, chunks, cu):
    """cu_tokens that falls is reported, the prefix and the pages of none stay as they were, and the next
    step is right."""
    most = max(max(chunks), max(b - a for a, b in zip(cu, cu[1:])))
    x = px.make([300, 40, 0, 129], chunks, [-1, 0, 0, 0], 4, 2, 64, 16, dtype, fox, seed=7,
                tail=max(cu) - sum(chunks) + 5, width=-(-(300 + most) // 16))
    cache = pc.cache_of(lib, x)
    before = px.snapshot(x)
    ws = lib.new_paged_workspace(cache, x["q"].shape[0], most, Hq=4, prefix=True)
    good, x["cu"] = x["cu"], torch.tensor(cu, dtype=torch.int32, device="cuda")
    out = torch.full_like(x["q"], 3.0)
    px.step(lib, dict(x, chunks=[most]), cache, out=out, workspace=ws)
    assert lib.path_check_workspace(ws) == lib.ERR_CACHE
    assert (out[max(cu):] == 3).all()
    for n, t in (("k_pages", "k_table"), ("v_pages", "v_table"), ("g_pages", "k_table")):
        if x[n] is not None:
            other = torch.ones(x[n].shape[0], dtype=torch.bool, device="cuda")
            mine = x[t][1:]
            other[mine[mine >= 0].long()] = False
            assert wc.same_bits(x[n][other], before[n][other])
    for n in before:
        if x[n] is not None:
            x[n].copy_(before[n])
    x["cu"] = good
    got = px.step(lib, x, cache, workspace=ws)
    assert lib.path_check_workspace(ws) == lib.OK
    px.check(x, before, got)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("pool", ["k", "v"])
def test_prefix_page_that_is_not_mapped(lib, dtype, T, pool):
    """A prefix that lacks a page is reported; what else there is counts as if its positions were absent."""
    x = px.make([100, 9, 70], [0, T, T], [-1, 0, -1], 4, 2, 64, 16, dtype, True, seed=8)
    x[pool + "_table"][0, 3] = -1
    before = px.snapshot(x)
    cache = pc.cache_of(lib, x)
    ws = lib.new_paged_workspace(cache, 2 * T, T, prefix=True)
    out = px.step(lib, x, cache, workspace=ws)
    assert lib.path_check_workspace(ws) == lib.ERR_CACHE
    assert torch.isfinite(out.float()).all()
    y = dict(x, **before)  # the sequence without a prefix
    pc.close(out[T:], pc.reference(y)[0][T:], dtype, "out")


@pytest.mark.parametrize("fox", [False, True])
def test_pools_past_2_31_elements(lib, fox):
    page, Hkv, d, far = 64, 16, 64, 34000  # 65,536 elements a page
    for prefix in (False, True):
        if prefix:
            x = px.make([500, 3, 0], [0, 1, 1], [-1, 0, 0], 16, Hkv, d, page, BF, fox, seed=9, width=300)
        else:
            x = pc.make([500, 3, 900], [1, 1, 1], 16, Hkv, d, page, BF, fox, seed=9, width=300)
        for a in "kv":
            n = x[a + "_pages"].shape[0]
            pools = (a + "_pages", "g_pages") if a == "k" else (a + "_pages",)
            for name in pools:
                if x[name] is not None:
                    big = torch.empty((far + n, *x[name].shape[1:]), dtype=x[name].dtype, device="cuda")
                    big[far:] = x[name]
                    big[:far] = 7.0
                    x[name] = big
            t = x[a + "_table"]
            t[t >= 0] += far
            x[a + "_ref"] = torch.cat([x[a + "_ref"].new_zeros(far), x[a + "_ref"]])
        assert x["k_pages"].numel() > 2 ** 31
        if prefix:
            prefix_run(lib, x)
        else:
            before = wc.snapshot(x)
            out = wc.window_step(lib, x, pc.cache_of(lib, x), 200, 4)
            torch.cuda.synchronize()
            wc.check_window(x, before, out, 200, 4)
        del x
        torch.cuda.empty_cache()


def test_graphs_of_both_kinds_share_a_workspace(lib):
    a = px.make([600, 20, 0], [0, 1, 1], [-1, 0, 0], 8, 2, 128, 64, BF, True, seed=10, width=60)
    b = pc.make([900, 130], [1, 1], 8, 2, 128, 64, BF, True, seed=11, width=60)
    c = px.make([300, 20, 0], [0, 30, 70], [-1, 0, 0], 8, 2, 128, 64, BF, True, seed=12, width=60)
    ca, cb, cc = (pc.cache_of(lib, x) for x in (a, b, c))
    ws = lib.new_paged_workspace(cc, 100, 70, prefix=True)
    was = [px.snapshot(a), wc.snapshot(b), px.snapshot(c)]
    outs = [torch.zeros_like(x["q"]) for x in (a, b, c)]

    def steps():
        return [lambda: px.step(lib, a, ca, workspace=ws, out=outs[0]),
                lambda: wc.window_step(lib, b, cb, 300, 4, workspace=ws, out=outs[1]),
                lambda: px.step(lib, c, cc, workspace=ws, out=outs[2])]

    for s in steps():
        s()
    for x, before in zip((a, b, c), was):
        for n in before:
            if x[n] is not None:
                x[n].copy_(before[n])
    graphs = []
    for s in steps():
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s()
        graphs.append(g)
    for order in ((2, 0, 1), (1, 2, 0)):
        for x, before in zip((a, b, c), was):
            for n in before:
                if x[n] is not None:
                    x[n].copy_(before[n])
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        px.check(a, was[0], outs[0])
        wc.check_window(b, was[1], outs[1], 300, 4)
        px.check(c, was[2], outs[2])
    assert lib.path_check_workspace(ws) == lib.OK


def test_two_streams_at_once(lib):
    """Steps on two other streams, each with its own workspace and cache."""
    xs = [px.make([2000, 20, 0, 5], [0, 1, 1, 1], [-1, 0, 0, 0], 8, 2, 128, 64, BF, True, seed=13, width=70),
          px.make([1500, 20, 0], [0, 30, 70], [-1, 0, 0], 8, 8, 64, 64, BF, False, seed=14)]
    was = [px.snapshot(x) for x in xs]
    caches = [pc.cache_of(lib, x) for x in xs]
    spaces = [lib.new_paged_workspace(c, sum(x["chunks"]), max(x["chunks"]), Hq=8, prefix=True)
              for c, x in zip(caches, xs)]
    streams = [torch.cuda.Stream() for _ in xs]
    outs = [torch.empty_like(x["q"]) for x in xs]
    torch.cuda.synchronize()
    for _ in range(3):
        for x, before in zip(xs, was):
            for n in before:
                if x[n] is not None:
                    x[n].copy_(before[n])
        torch.cuda.synchronize()
        for x, c, ws, s, out in zip(xs, caches, spaces, streams, outs):
            px.step(lib, x, c, workspace=ws, out=out, stream=s)
        torch.cuda.synchronize()
        for x, before, out in zip(xs, was, outs):
            px.check(x, before, out)


@pytest.mark.parametrize("page", [16, 256])
def test_trim_twice_and_reserve(lib, page):
    """A second trim finds nothing, and the pages that left can be had again."""
    x = pc.make([1000, 5, 700], [0, 0, 0], 2, 2, 64, page, BF, False, seed=15, spare=0)
    cache = pc.cache_of(lib, x)
    lib.path_paged_trim(cache, 100, 4)
    first = [getattr(cache, n).clone() for n in ("k_table", "v_table", "k_ref", "v_ref", "lens")]
    lib.path_paged_trim(cache, 100, 4)
    for a, n in zip(first, ("k_table", "v_table", "k_ref", "v_ref", "lens")):
        assert torch.equal(a, getattr(cache, n)), n
    free = int((cache.k_ref == 0).sum())
    assert free == sum(max(0, (n - 99) // page - (4 + page - 1) // page) for n in (1000, 5, 700))
    room = pc.pages(int(cache.lens[1]), page) * page - int(cache.lens[1])
    most = min(free, cache.k_table.shape[1] - 1)
    new = torch.tensor([0, room + most * page, 0], dtype=torch.int32, device="cuda")
    lib.path_paged_reserve(new, cache)
    assert int((cache.k_ref == 0).sum()) == free - most
