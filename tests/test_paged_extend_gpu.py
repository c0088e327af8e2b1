"""Steps of new tokens over a paged cache (path_paged_extend, path_fox_paged_extend) against
the fp64 reference: head layouts, page sizes, ragged chunks and lengths from 0, strides, gates,
repeated and captured calls, and what the device finds wrong."""
import pytest
import torch

from tests import paged_cases as pc

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def run(lib, x, scale=None, **kw):
    before = pc.snapshot(x)
    out = pc.step(lib, x, scale=scale, **kw)
    torch.cuda.synchronize()
    pc.check(x, before, out, scale)
    return out


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (4, 2), (4, 1), (3, 1)])
def test_single_tokens(lib, dtype, fox, d, Hq, Hkv):
    # lengths around a page's and a split's border, and an empty cache; the last sequence idles
    lens = [0, 1, 15, 16, 65, 127, 300, 1100, 40]
    x = pc.make(lens, [1] * 8 + [0], Hq, Hkv, d, 16, dtype, fox, seed=1)
    run(lib, x)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("d,Hq,Hkv,page", [(64, 2, 2, 16), (64, 6, 2, 32), (128, 2, 2, 64),
                                           (128, 4, 1, 128)])
@pytest.mark.parametrize("lens,chunks", [
    ([0, 0, 0], [1, 64, 65]),               # nothing cached: one block, a full one, one more
    ([5, 64, 200], [3, 0, 17]),             # short chunks, an idle sequence between
    ([63, 130, 1], [64, 128, 200]),         # several blocks
    ([700, 0, 33], [2, 130, 1]),            # several splits; one token among longer chunks
])
def test_chunks(lib, dtype, fox, d, Hq, Hkv, page, lens, chunks):
    x = pc.make(lens, chunks, Hq, Hkv, d, page, dtype, fox, seed=2)
    run(lib, x)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("chunks", [[1, 1, 1], [70, 1, 9]])
def test_strides_and_rows_behind_the_last_sequence(lib, dtype, fox, chunks):
    x = pc.make([20, 0, 150], chunks, 4, 2, 64, 32, dtype, fox, seed=3, head_major=True, tail=7)
    N = x["q"].shape[0]
    out = torch.full((4, N, 64), 7.0, dtype=dtype, device="cuda").transpose(0, 1)
    run(lib, x, out=out)
    assert (out[sum(chunks):] == 7).all()


@pytest.mark.parametrize("chunks", [[1, 1], [150, 40]])
def test_other_scales(lib, chunks):
    for scale in (0.0, -0.2, 0.3):
        x = pc.make([90, 40], chunks, 2, 1, 64, 64, F32, False, seed=4)
        run(lib, x, scale=scale)


@pytest.mark.parametrize("chunks", [[1, 1], [150, 40]])
@pytest.mark.parametrize("G", [1, 3])
def test_scales_that_turn_the_order(lib, chunks, G):
    """Logits of unit size, as the bar of bf16 supposes, and none."""
    for scale in (0.0, -0.125):
        x = pc.make([90, 340], chunks, 2 * G, 2, 64, 64, BF, G == 3, seed=4)
        run(lib, x, scale=scale)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d,page,chunks", [
    (5, 1, 128, 256, [1, 9, 40]),
    (16, 2, 64, 256, [1, 1, 1]),
    (128, 1, 128, 16, [1, 0, 1]),   # a tile's rows are one token's
    (256, 1, 64, 32, [1, 1, 0]),    # more rows for one token than a tile has
    (200, 2, 128, 64, [2, 1, 70]),
])
def test_many_heads_to_a_key(lib, dtype, fox, Hq, Hkv, d, page, chunks):
    x = pc.make([700, 0, 255], chunks, Hq, Hkv, d, page, dtype, fox, seed=19)
    run(lib, x)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("chunks", [[1, 1], [70, 3]])
def test_inputs_broadcast_over_heads_and_nan_behind(lib, dtype, chunks):
    """One transition and gate for all heads, given with a stride of 0; NaN in the rows behind
    the last sequence."""
    x = pc.make([50, 300], chunks, 4, 2, 64, 16, dtype, True, seed=20, tail=3)
    for n in ("w", "beta", "log_f"):
        x[n] = x[n][:, :1].expand(x[n].shape)
    for n in ("q", "k", "v"):
        x[n][sum(chunks):] = float("nan")
    run(lib, x)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("chunks", [[1, 1], [70, 3]])
def test_two_streams_at_once(lib, dtype, chunks):
    """Two caches stepped on two streams, each with its own workspace, give what they give one
    after the other."""
    xs = [pc.make([900, 130], chunks, 4, 2, 64, 16, dtype, True, seed=21 + i) for i in range(2)]
    caches = [pc.cache_of(lib, x) for x in xs]
    ws = [lib.new_paged_workspace(c, sum(chunks), max(chunks), Hq=4) for c in caches]
    starts = [pc.snapshot(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    ends = []
    for apart in (True, False):
        for x, s in zip(xs, starts):
            for n in s:
                x[n].copy_(s[n])
        outs = [[], []]
        torch.cuda.synchronize()
        for _ in range(10):
            for i, x in enumerate(xs):
                with torch.cuda.stream(streams[i]):
                    outs[i].append(pc.step(lib, x, caches[i], workspace=ws[i]))
                if apart:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        ends.append([t.clone() for o in outs for t in o] +
                    [x[n].nan_to_num(nan=7.0) for x in xs for n in starts[0]])
    assert all(torch.equal(a, b) for a, b in zip(*ends))
    assert all(lib.path_check_workspace(w) == lib.OK for w in ws)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fox", [False, True])
def test_beta_zero_and_two(lib, dtype, fox):
    # beta = 0 leaves keys as they are; beta near 2 is a reflection
    for beta in (0.0, 1.99):
        x = pc.make([70, 10], [80, 5], 2, 2, 64, 16, dtype, fox, seed=5)
        x["beta"].fill_(beta)
        run(lib, x)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("chunks", [[1, 1], [90, 3]])
def test_gates_that_close(lib, dtype, chunks):
    """Gates so small that everything before one vanishes, among gates of ordinary size."""
    x = pc.make([300, 40], chunks, 4, 2, 64, 32, dtype, True, seed=6)
    x["log_f"][0] = -1e6
    if chunks[0] > 1:
        x["log_f"][66, :2] = -3e8
    run(lib, x)


def far_key(lens, chunks, at, Hq, Hkv, d, page, dtype=BF):
    """Steps whose gates close fast, exp(-0.35) a token, so that nothing a few hundred positions
    back should count, but one key far back points along every query with a logit of 260: at
    most 180 of gates lie on it, so it takes all the weight (the logits of the others are of
    unit size). `at`: its position per sequence."""
    x = pc.make(lens, chunks, Hq, Hkv, d, page, dtype, True, seed=22)
    q = torch.randn(d, device="cuda")
    q = (q * d ** 0.5 / q.norm()).to(dtype)
    x["q"][:] = q
    x["beta"].zero_()
    x["log_f"].fill_(-0.35)
    first = 0
    for s, (n, T, j) in enumerate(zip(lens, chunks, at)):
        dist = torch.arange(n - 1, -1, -1, device="cuda", dtype=torch.float32)
        pc.put(x["g_pages"], x["k_table"][s], 0, (-0.35 * dist)[:, None].expand(n, Hq).contiguous())
        key = (q.double() * 260 / d ** 0.5).to(dtype)[None, None].expand(1, Hkv, d)
        if j is not None and j < n:
            pc.put(x["k_pages"], x["k_table"][s], j, key.contiguous())
        elif j is not None:
            x["k"][first + j - n] = key[0]
        first += T
    return x


@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (8, 2), (3, 1)])
@pytest.mark.parametrize("lens,chunks,at", [
    ([900, 600, 300], [1, 1, 1], [500, 100, None]),      # single tokens; far keys of two of them
    ([700, 200, 400], [30, 3, 65], [280, None, 5]),      # one row tile, or two
    ([500, 0], [190, 3], [300, None]),                   # the chunk's own blocks, and cached keys
    ([0, 0], [450, 500], [10, 63]),                      # a chunk's first block
])
def test_far_keys_behind_closed_gates(lib, d, page, Hq, Hkv, lens, chunks, at):
    x = far_key(lens, chunks, at, Hq, Hkv, d, page)
    run(lib, x)


@pytest.mark.parametrize("Hq,chunk", [(2, 1), (8, 40)])
def test_far_key_beside_an_absent_page(lib, Hq, chunk):
    x = far_key([900], [chunk], [550], Hq, 2, 64, 16)
    ids = x["v_table"][0]
    want = x["v_pages"][int(ids[550 // 16]), :, 550 % 16].float()
    ids[550 // 16 + 1] = -1
    x["k_table"][0, 550 // 16 - 1] = 1 << 20
    cache = pc.cache_of(lib, x)
    ws = lib.new_paged_workspace(cache, chunk, chunk, Hq=Hq)
    out = pc.step(lib, x, cache, workspace=ws)
    assert lib.path_check_workspace(ws) == lib.ERR_CACHE
    # all the weight is the far key's, and its value is a bf16 number already
    assert torch.equal(out.float(), want.repeat_interleave(Hq // 2, 0).expand(chunk, Hq, 64))


def test_one_call_equals_single_steps(lib):
    """A chunk and its tokens one by one end in the same cache and outputs, in fp32 within the
    roundings of either."""
    x = pc.make([33, 0], [70, 12], 2, 2, 64, 16, F32, True, seed=7)
    y = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}
    out = run(lib, x)
    cache = pc.cache_of(lib, y)
    outs = torch.empty_like(out)
    for t in range(70):
        idx = [b for b in range(2) if t < y["chunks"][b]]
        at = [sum(y["chunks"][:b]) + t for b in idx]
        cu = torch.tensor([0, 1, len(idx)], dtype=torch.int32, device="cuda")
        rows = {n: y[n][at].contiguous() for n in ("q", "k", "v", "w", "beta", "log_f")}
        outs[at] = lib.path_fox_paged_extend(rows["q"], rows["k"], rows["v"], rows["w"],
                                             rows["beta"], rows["log_f"], cu, cache, 1)
        cache.lens += cu[1:] - cu[:-1]
    for b in range(2):
        n = y["n"][b] + y["chunks"][b]
        for p in ("k_pages", "g_pages"):
            u, v = (pc.rows_of(z[p], z["k_table"][b], n) for z in (x, y))
            assert float((u - v).norm() / v.norm()) < 2e-5
    assert float((out - outs).norm() / out.norm()) < 2e-5


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("chunks", [[1, 1, 1], [5, 66, 1]])
def test_runs_repeat_bit_for_bit(lib, dtype, chunks):
    got = []
    for _ in range(2):
        x = pc.make([900, 17, 64], chunks, 4, 2, 64, 64, dtype, True, seed=8)
        out = pc.step(lib, x)
        got.append([out, x["k_pages"], x["v_pages"], x["g_pages"]])
    for a, b in zip(*got):
        assert torch.equal(a.nan_to_num(nan=7.0), b.nan_to_num(nan=7.0))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("chunks", [[1, 1], [67, 2]])
def test_another_stream_and_a_captured_step(lib, dtype, chunks):
    """A captured step advances through replays whose lengths and tokens change on the device,
    two graphs sharing one workspace."""
    x = pc.make([40, 130], chunks, 2, 2, 64, 16, dtype, True, seed=9, width=32)
    for name in ("k", "v"):  # room for four steps
        t, ref = x[name + "_table"], x[name + "_ref"]
        more = 32 * 2
        pool = x[name + "_pages"]
        base = pool.shape[0]
        grown = torch.full((base + more,) + tuple(pool.shape[1:]), float("nan"), dtype=pool.dtype,
                           device="cuda")
        grown[:base] = pool
        x[name + "_pages"] = grown
        if name == "k":
            g = torch.full((base + more,) + tuple(x["g_pages"].shape[1:]), float("nan"), device="cuda")
            g[:base] = x["g_pages"]
            x["g_pages"] = g
        x[name + "_ref"] = torch.cat([ref, torch.zeros(more, dtype=torch.int32, device="cuda")])
        free = iter(range(base, base + more))
        for s in range(2):
            for i in range(32):
                if int(t[s, i]) < 0:
                    t[s, i] = next(free)
    cache = pc.cache_of(lib, x)
    ws = lib.new_paged_workspace(cache, x["q"].shape[0], max(chunks))
    out = torch.empty_like(x["q"])
    T = x["cu"][1:] - x["cu"][:-1]
    start = pc.snapshot(x)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        pc.step(lib, x, cache, out=out, workspace=ws)  # warm-up
        stream.synchronize()
        graphs = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                pc.step(lib, x, cache, out=out, workspace=ws)
                cache.lens += T
            graphs.append(g)
    for n in start:
        x[n].copy_(start[n])
    cache.lens.copy_(torch.tensor([40, 130], dtype=torch.int32))
    torch.cuda.synchronize()
    for turn in range(3):
        x["n"] = cache.lens.tolist()
        before = pc.snapshot(x)
        y = pc.make([40, 130], chunks, 2, 2, 64, 16, dtype, True, seed=20 + turn)
        for n in ("q", "k", "v", "w", "beta", "log_f"):
            x[n].copy_(y[n])
        graphs[turn % 2].replay()
        torch.cuda.synchronize()
        pc.check(x, before, out)
    assert lib.path_check_workspace(ws) == lib.OK


def test_stream_argument(lib):
    x = pc.make([400, 3], [1, 1], 2, 2, 64, 16, BF, False, seed=10)
    before = pc.snapshot(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = pc.step(lib, x, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    pc.check(x, before, out)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("chunks", [[1, 1, 1, 1], [70, 3, 2, 80]])
def test_what_the_device_finds_wrong(lib, dtype, chunks):
    """A length past the table, a negative one and chunks out of order leave their sequence as
    it was and set the status word; the others are served."""
    x = pc.make([30, 20, 50, 10], chunks, 2, 2, 64, 16, dtype, True, seed=11)
    x["lens"][1] = 5000
    x["lens"][2] = -1
    cache = pc.cache_of(lib, x)
    ws = lib.new_paged_workspace(cache, x["q"].shape[0], max(chunks))
    before = pc.snapshot(x)
    out = torch.full_like(x["q"], 3.0)
    pc.step(lib, x, cache, out=out, workspace=ws)
    assert lib.path_check_workspace(ws) == lib.ERR_CACHE
    assert lib.path_check_workspace(ws) == lib.OK
    a, b = sum(chunks[:1]), sum(chunks[:3])
    assert (out[a:b] == 3).all()
    ref, Ks, _, _ = pc.reference(dict(x, **before))
    pc.close(torch.cat([out[:a], out[b:]]), torch.cat([ref[:a], ref[b:]]), dtype, "out")
    for s in (1, 2):
        for n, t in (("k_pages", "k_table"), ("v_pages", "v_table"), ("g_pages", "k_table")):
            ids = x[t][s][x[t][s] >= 0].long()
            assert torch.equal(x[n][ids].nan_to_num(nan=7.0), before[n][ids].nan_to_num(nan=7.0))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("chunks", [[1, 1], [70, 3]])
def test_pages_outside_the_pool_are_absent(lib, dtype, chunks):
    """Page numbers below 0 or past the pool: their positions take no part, nothing is written
    for them, and the status word says so."""
    x = pc.make([100, 90], chunks, 2, 1, 64, 16, dtype, False, seed=12)
    good = {n: x[n].clone() for n in ("k_table", "v_table")}
    x["k_table"][0, 2] = x["k_pages"].shape[0]
    x["v_table"][0, 2] = -5
    x["k_table"][0, 4] = -1
    x["v_table"][0, 4] = 1 << 30
    cache = pc.cache_of(lib, x)
    ws = lib.new_paged_workspace(cache, x["q"].shape[0], max(chunks), Hq=2)
    before = pc.snapshot(x)
    out = pc.step(lib, x, cache, workspace=ws)
    assert lib.path_check_workspace(ws) == lib.ERR_CACHE
    # the same cache without those 32 positions
    y = dict(x, **before)
    keep = [p for p in range(100) if p // 16 not in (2, 4)]
    K, V = (pc.rows_of(before[n + "_pages"], good[n + "_table"][0], 100)[keep].to(dtype) for n in "kv")
    z = pc.make([68, 90], chunks, 2, 1, 64, 16, dtype, False, seed=12)
    for n in ("q", "k", "v", "w", "beta"):
        z[n] = x[n]
    for n, rows in (("k", K), ("v", V)):
        pc.put(z[n + "_pages"], z[n + "_table"][0], 0, rows)
        pc.put(z[n + "_pages"], z[n + "_table"][1], 0,
               pc.rows_of(y[n + "_pages"], good[n + "_table"][1], 90).to(dtype))
    ref = pc.reference(z)[0]
    pc.close(out, ref, dtype, "out")
    bad = [int(good["k_table"][0, i]) for i in (2, 4)]
    for i in bad:
        assert torch.equal(x["k_pages"][i].nan_to_num(nan=7.0), before["k_pages"][i].nan_to_num(nan=7.0))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d,new", [
    (3, 1, 64, {0: 1, 17: 1, 39: 1}),       # single tokens
    (8, 1, 128, {3: 2, 38: 20}),            # more rows than a tile of 128: the key update's own pass
    (2, 2, 64, {20: 1}),                    # one token in all
])
def test_more_sequences_than_tokens(lib, dtype, fox, Hq, Hkv, d, new):
    """Most sequences idle, so that the step has fewer tokens than the cache sequences."""
    lens = [(37 * s) % 300 for s in range(40)]
    x = pc.make(lens, [new.get(s, 0) for s in range(40)], Hq, Hkv, d, 16, dtype, fox, seed=17)
    run(lib, x)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("Hq,Hkv,chunks,cu", [
    (8, 2, [100, 0, 100, 100], [0, 200, 100, 300, 300]),
    (2, 2, [1] * 6, [0, 5, 1, 6, 2, 7, 3]),
    (4, 2, [700, 20], [300, 0, 720]),
    (2, 1, [64] * 12, [0, 768] * 6 + [768]),  # the same tokens for every other sequence
])
def test_token_ranges_that_fall(lib, dtype, fox, Hq, Hkv, chunks, cu):
    """cu_tokens that falls is reported, only the step's own sequences' pages and rows change,
    and the next step is right."""
    lens = [(130 * s) % 400 for s in range(len(chunks))]
    N, most = max(cu), max(max(chunks), max(b - a for a, b in zip(cu, cu[1:])))
    width = max(-(-(n + most) // 16) for n in lens)
    x = pc.make(lens, chunks, Hq, Hkv, 64, 16, dtype, fox, seed=18, tail=N + 5 - sum(chunks), width=width)
    cache = pc.cache_of(lib, x)
    before, tables = pc.snapshot(x), [x[n].clone() for n in ("k_table", "v_table", "lens")]
    ws = lib.new_paged_workspace(cache, x["q"].shape[0], most, Hq=Hq)
    args = [x[n] for n in ("q", "k", "v", "w", "beta")] + ([x["log_f"]] if fox else [])
    call = lib.path_fox_paged_extend if fox else lib.path_paged_extend
    out = torch.full_like(x["q"], 3.0)
    call(*args, torch.tensor(cu, dtype=torch.int32, device="cuda"), cache, most, out=out, workspace=ws)
    assert lib.path_check_workspace(ws) == lib.ERR_CACHE
    assert (out[N:] == 3).all()
    for n, t in (("k_pages", "k_table"), ("v_pages", "v_table"), ("g_pages", "k_table")):
        if x[n] is not None:
            spare = torch.ones(x[n].shape[0], dtype=torch.bool, device="cuda")
            spare[x[t][x[t] >= 0].long()] = False
            assert torch.equal(x[n][spare].nan_to_num(nan=7.0), before[n][spare].nan_to_num(nan=7.0))
            x[n].copy_(before[n])
    assert all(torch.equal(a, x[n]) for a, n in zip(tables, ("k_table", "v_table", "lens")))
    got = pc.step(lib, x, cache, workspace=ws)
    assert lib.path_check_workspace(ws) == lib.OK
    pc.check(x, before, got)


def test_a_workspace_for_chunks_serves_smaller_steps(lib):
    x = pc.make([200, 100], [300, 20], 2, 2, 64, 16, BF, True, seed=13)
    cache = pc.cache_of(lib, x)
    ws = lib.new_paged_workspace(cache, 320, 300)
    before = pc.snapshot(x)
    out = pc.step(lib, x, cache, workspace=ws)
    pc.check(x, before, out)
    for chunks in ([1, 1], [0, 65], [2, 0]):
        y = pc.make([200, 100], chunks, 2, 2, 64, 16, BF, True, seed=14, width=x["k_table"].shape[1])
        before = pc.snapshot(y)
        out = pc.step(lib, y, workspace=ws)
        pc.check(y, before, out)
    assert lib.path_check_workspace(ws) == lib.OK


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 4, 64), (4, 1, 128), (3, 1, 64)])
@pytest.mark.parametrize("chunks", [[3, 1, 1, 0, 1, 2], [1, 1, 70, 1, 1, 1, 1, 1], [1, 2]])
def test_single_tokens_among_chunks(lib, dtype, fox, Hq, Hkv, d, chunks):
    x = pc.make([(90 * s) % 400 for s in range(len(chunks))], chunks, Hq, Hkv, d, 16, dtype, fox, seed=23)
    run(lib, x)


@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("Hq,chunk", [(16, 3), (32, 25), (64, 40)])
def test_many_key_tiles(lib, d, page, fox, Hq, chunk):
    """Long caches: many key tiles for every resident CTA, so that its rings and barriers turn
    many times, and stretches that begin and end inside an item; 3, 50 and 160 rows a key
    head."""
    x = pc.make([20000, 3000], [chunk, 1], Hq, 16, d, page, BF, fox, seed=16)
    run(lib, x)


def test_long_cache_offsets_past_32_bits(lib):
    """Pages whose byte and element offsets pass 2^31 and 2^32."""
    pages, page, H, d = 36000, 64, 16, 128  # 4.7e9 elements a pool
    kp = torch.empty((pages, H, page, d), dtype=BF, device="cuda")
    vp = torch.empty_like(kp)
    for chunks in ([1], [70]):
        x = pc.make([100], chunks, H, H, d, page, BF, False, seed=15)
        ids = torch.tensor([[pages - 1, 0, pages // 2, pages - 2]], dtype=torch.int32, device="cuda")
        m = x["k_table"].shape[1]
        for n, big in (("k", kp), ("v", vp)):
            old = x[n + "_table"][0].long()
            big[ids[0, :m].long()] = x[n + "_pages"][old]
        before = pc.snapshot(x)
        ref, Ks, _, _ = pc.reference(dict(x, **before))
        cache = lib.PathPagedCache(k_pages=kp, v_pages=vp, k_table=ids[:, :m].contiguous(),
                                   v_table=ids[:, :m].contiguous(), lens=x["lens"])
        out = lib.path_paged_extend(x["q"], x["k"], x["v"], x["w"], x["beta"], x["cu"], cache,
                                    chunks[0])
        pc.close(out, ref, BF, "out")
        pc.close(pc.rows_of(kp, ids[0], 100 + chunks[0]), Ks[0], BF, "keys")
