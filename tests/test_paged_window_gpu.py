"""Steps through a sliding window with sinks (path_paged_window_extend, its gated form) and
path_paged_trim: against the fp64 reference, with everything out of sight poisoned."""
import pytest
import torch

from tests import paged_cases as pc
from tests import paged_window_cases as wc

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def run(lib, x, window, sinks, hide=True, **kw):
    if hide:
        wc.hide(x, window, sinks)
    before = wc.snapshot(x)
    cache = pc.cache_of(lib, x)
    out = wc.window_step(lib, x, cache, window, sinks, **kw)
    torch.cuda.synchronize()
    wc.check_window(x, before, out, window, sinks)
    return out


# a window of one; one inside a page, at its border, over several; sinks that end in a page, at its
# border, inside the window
SIGHTS = [(1, 0), (1, 5), (20, 0), (16, 16), (65, 3), (200, 130), (2000, 4)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("d,Hq,Hkv,page", [(64, 2, 2, 16), (128, 4, 1, 32), (64, 3, 1, 16), (128, 8, 1, 64)])
@pytest.mark.parametrize("window,sinks", SIGHTS)
def test_single_tokens(lib, dtype, fox, d, Hq, Hkv, page, window, sinks):
    x = pc.make([0, 1, 15, 16, 65, 127, 300, 1100, 40], [1] * 8 + [0], Hq, Hkv, d, page, dtype, fox, seed=1)
    run(lib, x, window, sinks)


@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("d,Hq,Hkv,page", [(64, 8, 8, 64), (128, 16, 4, 128), (128, 4, 4, 256)])
@pytest.mark.parametrize("window,sinks", [(100, 4), (1500, 40), (4000, 0)])
def test_single_tokens_of_large_caches(lib, fox, d, Hq, Hkv, page, window, sinks):
    # tables wide enough for the block kernels where the window is large
    lens = [5000 - 37 * i for i in range(20)]
    x = pc.make(lens, [1] * 20, Hq, Hkv, d, page, BF, fox, seed=2)
    run(lib, x, window, sinks)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("d,Hq,Hkv,page", [(64, 2, 2, 16), (64, 6, 2, 256), (128, 2, 2, 64), (128, 4, 1, 128)])
@pytest.mark.parametrize("lens,chunks", [
    ([0, 0, 0], [1, 64, 65]),
    ([5, 64, 200], [3, 0, 17]),
    ([63, 130, 400], [64, 128, 200]),
    ([700, 0, 333], [2, 130, 1]),
])
@pytest.mark.parametrize("more,sinks", [(0, 0), (1, 4), (90, 70), (1000, 1)])
def test_chunks(lib, dtype, fox, d, Hq, Hkv, page, lens, chunks, more, sinks):
    x = pc.make(lens, chunks, Hq, Hkv, d, page, dtype, fox, seed=3)
    run(lib, x, max(chunks) + more, sinks)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("chunks", [[1, 1, 1], [70, 1, 9]])
def test_strides_and_rows_behind_the_last_sequence(lib, dtype, chunks):
    x = pc.make([20, 0, 350], chunks, 4, 2, 64, 32, dtype, True, seed=4, head_major=True, tail=7)
    N = x["q"].shape[0]
    out = torch.full((4, N, 64), 7.0, dtype=dtype, device="cuda").transpose(0, 1)
    run(lib, x, 80, 5, out=out)
    assert (out[sum(chunks):] == 7).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("chunks", [[1, 1, 1], [7, 1, 90]])
def test_a_window_that_hides_nothing_is_the_plain_step(lib, dtype, chunks):
    a = pc.make([300, 0, 77], chunks, 4, 2, 64, 32, dtype, True, seed=5)
    b = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in a.items()}
    one = pc.step(lib, a)
    two = wc.window_step(lib, b, pc.cache_of(lib, b), 1 << 22, 0)
    torch.cuda.synchronize()
    for n in ("k_pages", "v_pages", "g_pages"):
        assert wc.same_bits(a[n], b[n]), n
    assert wc.same_bits(one, two)


@pytest.mark.parametrize("chunks", [[1, 1], [3, 70]])
def test_repeats_and_a_replayed_graph_give_the_same_bits(lib, chunks):
    x = pc.make([900, 1300], chunks, 8, 2, 128, 64, BF, True, seed=6)
    before = wc.snapshot(x)
    cache = pc.cache_of(lib, x)
    ws = lib.new_paged_workspace(cache, sum(chunks), max(chunks))
    out = torch.empty_like(x["q"])
    wc.window_step(lib, x, cache, 300, 4, workspace=ws, out=out)
    torch.cuda.synchronize()
    first = [out.clone()] + [x[n].clone() for n in before]
    wc.check_window(x, before, out, 300, 4)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        wc.window_step(lib, x, cache, 300, 4, workspace=ws, out=out)
    for _ in range(2):
        for n in before:
            x[n].copy_(before[n])
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(first, [out] + [x[n] for n in before]):
            assert wc.same_bits(a, b)
    assert lib.path_check_workspace(ws) == lib.OK


def test_one_workspace_serves_every_window(lib):
    x = pc.make([2000 + i for i in range(6)], [1] * 6, 8, 4, 64, 16, BF, False, seed=7)
    cache = pc.cache_of(lib, x)
    need = lib.path_paged_workspace_bytes(cache, 6, 1, 8)
    ws = torch.zeros(need + 4096, dtype=torch.uint8, device="cuda")
    ws[need:] = 77
    for window in (1, 3, 63, 64, 65, 500, 1000, 1500, 2001, 4000):
        wc.window_step(lib, x, cache, window, 4, workspace=ws[:need])
    torch.cuda.synchronize()
    assert (ws[need:] == 77).all() and lib.path_check_workspace(ws[:need]) == lib.OK


def test_page_in_sight_that_is_not_mapped(lib):
    x = pc.make([200], [1], 2, 2, 64, 16, BF, False, seed=8)
    wc.hide(x, 40, 4)
    x["k_table"][0, 11] = -1
    cache = pc.cache_of(lib, x)
    ws = lib.new_paged_workspace(cache, 1, 1)
    wc.window_step(lib, x, cache, 40, 4, workspace=ws)
    assert lib.path_check_workspace(ws) == lib.ERR_CACHE


# ---------------------------------------------------------------- trim

@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 40), (100, 0), (64, 64), (300, 17), (5000, 4)])
def test_trim(lib, page, window, sinks):
    lens = [0, 1, page, page + 1, 200, 640, 1000, 3000]
    x = pc.make(lens, [0] * 7 + [page * 3], 2, 1, 64, page, BF, True, seed=9, width=60 * 64 // page)
    cache = pc.cache_of(lib, x)
    # shared value pages, and a row of the table that is full to its end
    cache.v_ref += (cache.v_ref > 0).int() * (torch.arange(cache.v_ref.numel(), device="cuda") % 3 == 0)
    before = {n: getattr(cache, n).clone() for n in ("k_table", "v_table", "k_ref", "v_ref", "lens")}
    lib.path_paged_trim(cache, window, sinks)
    for a in "kv":
        rows, lens2, left = wc.trimmed(before[a + "_table"].tolist(), lens, window, sinks, page)
        ref = before[a + "_ref"].clone()
        ref.index_add_(0, torch.tensor(left, dtype=torch.long, device="cuda"),
                       -torch.ones(len(left), dtype=torch.int32, device="cuda"))
        assert getattr(cache, a + "_table").tolist() == rows
        assert torch.equal(getattr(cache, a + "_ref"), ref)
    assert cache.lens.tolist() == lens2


def test_trim_of_a_table_wider_than_a_round(lib):
    x = pc.make([5000 * 16 + 3, 30], [0, 0], 1, 1, 64, 16, BF, False, seed=10, width=5100)
    cache = pc.cache_of(lib, x)
    before = cache.k_table.tolist()
    lib.path_paged_trim(cache, 333, 20)
    rows, lens, _ = wc.trimmed(before, [5000 * 16 + 3, 30], 333, 20, 16)
    assert cache.k_table.tolist() == rows and cache.lens.tolist() == lens


def test_trim_leaves_a_length_that_does_not_fit(lib):
    x = pc.make([100, 100], [0, 0], 1, 1, 64, 16, BF, False, seed=11)
    cache = pc.cache_of(lib, x)
    cache.lens[0] = 16 * cache.k_table.shape[1] + 1
    before = cache.k_table.clone()
    with pytest.raises(lib.PathError) as e:
        lib.path_paged_trim(cache, 16, 0)
    assert e.value.code == lib.ERR_CACHE
    assert torch.equal(cache.k_table[0], before[0]) and cache.lens[1] == 100 - 16 * 5


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fox", [False, True])
def test_streams_that_reserve_step_and_trim(lib, dtype, fox):
    """Two streams run far past their pools' size: reserved, stepped and trimmed in one captured
    graph; outputs against those of an untrimmed fp64 stream."""
    window, sinks, page, Hq, Hkv, d, S = 50, 5, 16, 4, 2, 64, 2
    steps, chunk = 24, 9
    cache = lib.new_paged_cache(S, 8, 16, Hq=Hq, Hkv=Hkv, d=d, page=page, dtype=dtype, fox=fox)
    whole = pc.make([0] * S, [steps * chunk] * S, Hq, Hkv, d, page, dtype, fox, seed=12)
    ref, *_ = wc.window_reference(whole, window, sinks)
    ws = lib.new_paged_workspace(cache, S * chunk, chunk, Hq=Hq)
    new = torch.full((S,), chunk, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, chunk, 2 * chunk], dtype=torch.int32, device="cuda")
    x = {n: whole[n][:S * chunk].clone() for n in ("q", "k", "v", "w", "beta", "log_f")
         if whole[n] is not None}
    x.update(log_f=x.get("log_f"), cu=cu, chunks=[chunk] * S)
    out = torch.empty_like(x["q"])

    def one():
        lib.path_paged_reserve(new, cache, workspace=ws)
        wc.window_step(lib, x, cache, window, sinks, workspace=ws, out=out)
        cache.lens += new
        lib.path_paged_trim(cache, window, sinks, workspace=ws)

    g = None
    for step in range(steps):
        at = torch.cat([torch.arange(chunk) + s * steps * chunk + step * chunk for s in range(S)]).cuda()
        for n in ("q", "k", "v", "w", "beta", "log_f"):
            if x[n] is not None:
                x[n].copy_(whole[n][at])
        if step == 1:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                one()
        if g is None:
            one()
        else:
            g.replay()
        torch.cuda.synchronize()
        err = (out.double() - ref[at]).norm() / ref[at].norm()
        # bf16 keys are rounded (2^-8 / sqrt 3 = 2.3e-3 at most, as a logit's error) once more in each
        # step that advances them, 7 times for the 50 in the window and 24 for the 5 sinks:
        # 2.3e-3 sqrt((50 * 7 + 5 * 24) / 55) = 6.6e-3, beside the 4.5e-3 of a step alone 8e-3
        assert float(err) <= (8e-3 if dtype == BF else 1e-5), (step, float(err))
    assert lib.path_check_workspace(ws) == lib.OK
    assert cache.lens.max() <= window + sinks + 2 * page
    assert int((cache.k_ref > 0).sum()) <= 2 * 8
