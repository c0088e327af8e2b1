"""The page calls of the paged cache (reserve, fork, free, compact) against a plain model of
the pools, and a run of them together with steps."""
import random

import pytest
import torch

from tests import paged_cases as pc

pytestmark = pytest.mark.gpu


def state(c):
    return {n: getattr(c, n).clone() for n in ("k_pages", "v_pages", "g_pages", "k_table", "v_table",
                                               "k_ref", "v_ref", "lens")
            if getattr(c, n) is not None}


def same(c, s):
    for n, t in s.items():
        assert torch.equal(getattr(c, n).nan_to_num(nan=7.0) if t.is_floating_point() else getattr(c, n),
                           t.nan_to_num(nan=7.0) if t.is_floating_point() else t), n


class Model:
    """The pools as Python lists: lowest free page first, in the order of the requests."""

    def __init__(self, c):
        s = {n: t.cpu() for n, t in state(c).items()}
        self.t = [s["k_table"].tolist(), s["v_table"].tolist()]
        self.ref = [s["k_ref"].tolist(), s["v_ref"].tolist()]
        self.lens = s["lens"].tolist()
        self.page = c.k_pages.shape[2]
        self.data = [s["k_pages"], s["v_pages"]]
        self.g = s.get("g_pages")

    def take(self, p):
        i = self.ref[p].index(0)
        self.ref[p][i] = 1
        return i

    def reserve(self, extra):
        for p in (0, 1):
            for s, row in enumerate(self.t[p]):
                for i in range(pc.pages(self.lens[s] + extra[s], self.page)):
                    if row[i] < 0:
                        row[i] = self.take(p)

    def free(self, rows):
        for p in (0, 1):
            for s in rows:
                for i, x in enumerate(self.t[p][s]):
                    if x >= 0:
                        self.ref[p][x] -= 1
                    self.t[p][s][i] = -1
        for s in rows:
            self.lens[s] = 0

    def copy(self, p, new, old, rows):
        self.data[p][new][:, :rows] = self.data[p][old][:, :rows]
        if p == 0 and self.g is not None:
            self.g[new][:, :rows] = self.g[old][:, :rows]

    def fork(self, src, dst):
        for p in (0, 1):
            for a, b in zip(src, dst):
                n = self.lens[a]
                for i in range(pc.pages(n, self.page)):
                    rows = min(self.page, n - i * self.page)
                    if p == 1 and rows == self.page:
                        self.t[p][b][i] = self.t[p][a][i]
                        self.ref[p][self.t[p][a][i]] += 1
                    else:
                        self.t[p][b][i] = self.take(p)
                        self.copy(p, self.t[p][b][i], self.t[p][a][i], rows)
        for a, b in zip(src, dst):
            self.lens[b] = self.lens[a]

    def compact(self):
        for p in (0, 1):
            ref = self.ref[p]
            live = sum(r > 0 for r in ref)
            holes = [i for i in range(live) if ref[i] <= 0]
            moves = [i for i in range(live, len(ref)) if ref[i] > 0]
            to = dict(zip(moves, holes))
            for a, b in to.items():
                self.copy(p, b, a, self.page)
                ref[b], ref[a] = ref[a], 0
            self.t[p] = [[to.get(x, x) for x in row] for row in self.t[p]]

    def check(self, c):
        assert c.k_table.tolist() == self.t[0] and c.v_table.tolist() == self.t[1]
        assert c.k_ref.tolist() == self.ref[0] and c.v_ref.tolist() == self.ref[1]
        assert c.lens.tolist() == self.lens
        for a, b in ((c.k_pages, self.data[0]), (c.v_pages, self.data[1]), (c.g_pages, self.g)):
            if a is not None:
                assert torch.equal(a.cpu().nan_to_num(nan=7.0), b.nan_to_num(nan=7.0))


def cache(lib, lens, page=16, Hq=4, Hkv=2, d=64, dtype=torch.bfloat16, fox=True, spare=40, width=24,
          seed=0):
    x = pc.make(lens, [0] * len(lens), Hq, Hkv, d, page, dtype, fox, seed=seed, spare=spare, width=width)
    return pc.cache_of(lib, x)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("page,d", [(16, 64), (32, 128), (128, 64)])
def test_calls_follow_the_model(lib, dtype, fox, page, d):
    rng = random.Random(page + d)
    lens = [0, 1, page - 1, page, page + 1, 3 * page + 5, 0, 7 * page, 0, 0]
    c = cache(lib, lens, page, 4, 2, d, dtype, fox, spare=60, seed=3)
    m = Model(c)
    ws = lib.new_paged_workspace(c)
    for turn in range(4):
        extra = [rng.choice([0, 0, 1, page, page + 3]) for _ in lens]
        lib.path_paged_reserve(torch.tensor(extra, dtype=torch.int32, device="cuda"), c, workspace=ws)
        m.reserve(extra)
        m.check(c)
        rows = rng.sample(range(len(lens)), 4)
        lib.path_paged_free(rows, c, workspace=ws)
        m.free(rows)
        m.check(c)
        src = [s for s in range(len(lens)) if s not in rows and m.lens[s] > 0]
        if src:
            pairs = [(rng.choice(src), r) for r in rows[:3]]
            lib.path_paged_fork([a for a, _ in pairs], [b for _, b in pairs], c, workspace=ws)
            m.fork([a for a, _ in pairs], [b for _, b in pairs])
            m.check(c)
        if turn % 2:
            lib.path_paged_compact(c, workspace=ws)
            m.compact()
            m.check(c)
    assert lib.path_check_workspace(ws) == lib.OK


def test_large_pools(lib):
    """Pools of more pages than one round of the planning loops takes, with odd counts."""
    nk, nv, S, width = 20011, 9001, 40, 300
    c = lib.new_paged_cache(S, width, nk, nv, Hq=1, Hkv=1, page=16, d=64)
    c.k_pages.normal_()
    c.v_pages.normal_()
    g = torch.Generator(device="cuda").manual_seed(1)
    c.k_ref.copy_(torch.rand(nk, generator=g, device="cuda") < 0.3)
    c.v_ref.copy_(torch.rand(nv, generator=g, device="cuda") < 0.2)
    kept = [c.k_ref.clone(), c.v_ref.clone()]
    extra = [(37 * s) % (16 * 180) for s in range(S)]
    lib.path_paged_reserve(torch.tensor(extra, dtype=torch.int32, device="cuda"), c)
    want = sum(pc.pages(e, 16) for e in extra)
    for t, ref, old in ((c.k_table, c.k_ref, kept[0]), (c.v_table, c.v_ref, kept[1])):
        free = (old == 0).nonzero()[:, 0][:want]
        assert torch.equal(t[t >= 0].long(), free)
        assert torch.equal(ref, old.index_fill(0, free, 1))
    c.lens.copy_(torch.tensor(extra, dtype=torch.int32))
    rows = [pc.rows_of(c.k_pages, c.k_table[s], extra[s]) for s in range(S)]
    lib.path_paged_compact(c)
    for s in range(S):
        assert torch.equal(rows[s], pc.rows_of(c.k_pages, c.k_table[s], extra[s]))
    for ref in (c.k_ref, c.v_ref):
        live = int((ref > 0).sum())
        assert (ref[:live] > 0).all() and (ref[live:] == 0).all()


def test_nothing_changes_when_pages_run_out(lib):
    c = cache(lib, [20, 40, 0], spare=2)
    ws = lib.new_paged_workspace(c)
    before = state(c)
    many = torch.tensor([0, 0, 16 * 10], dtype=torch.int32, device="cuda")
    for call in (lambda: lib.path_paged_reserve(many, c, workspace=ws),
                 lambda: lib.path_paged_fork([1], [2], c, workspace=ws),
                 lambda: lib.path_paged_reserve(torch.full_like(many, 16 * 24), c, workspace=ws)):
        call()
        assert lib.path_check_workspace(ws) == lib.ERR_CAPACITY
        same(c, before)


def test_rows_that_are_not_as_they_must_be(lib):
    c = cache(lib, [20, 40, 0, 5])
    ws = lib.new_paged_workspace(c)
    before = state(c)
    for src, dst in (([0], [3]),):  # the destination is not empty
        lib.path_paged_fork(src, dst, c, workspace=ws)
        assert lib.path_check_workspace(ws) == lib.ERR_CACHE
        same(c, before)
    c.k_table[0, 1] = 1 << 29  # a source page outside the pool
    before = state(c)
    lib.path_paged_fork([0], [2], c, workspace=ws)
    assert lib.path_check_workspace(ws) == lib.ERR_CACHE
    same(c, before)
    lib.path_paged_compact(c, workspace=ws)
    assert lib.path_check_workspace(ws) == lib.ERR_CACHE
    assert int(c.k_table[0, 1]) == 1 << 29
    c.lens[2] = -1
    lib.path_paged_reserve(torch.zeros(4, dtype=torch.int32, device="cuda"), c, workspace=ws)
    assert lib.path_check_workspace(ws) == lib.ERR_CAPACITY


def test_compact_of_empty_and_full_pools(lib):
    c = lib.new_paged_cache(3, 4, 10, 7, Hq=2, page=16)
    lib.path_paged_compact(c)
    assert not c.k_ref.any() and not c.v_ref.any()
    lib.path_paged_reserve(torch.tensor([48, 32, 16], dtype=torch.int32, device="cuda"), c)
    before = [c.k_table.clone(), c.v_table.clone()]
    lib.path_paged_compact(c)
    assert torch.equal(c.k_table, before[0]) and torch.equal(c.v_table, before[1])


def test_serving_run(lib):
    """Prompt, fork, decode, free, compact, decode: every output against the reference, with two
    sequences that share value pages and go different ways."""
    Hq, Hkv, d, page = 4, 2, 64, 16
    c = lib.new_paged_cache(4, 16, 64, Hq=Hq, Hkv=Hkv, d=d, page=page, dtype=torch.float32, fox=True)
    c.k_pages.fill_(float("nan"))
    c.v_pages.fill_(float("nan"))
    c.g_pages.fill_(float("nan"))
    ws = lib.new_paged_workspace(c, 400, 100)
    seed = [0]

    def advance(chunks):
        seed[0] += 1
        lib.path_paged_reserve(torch.tensor(chunks, dtype=torch.int32, device="cuda"), c, workspace=ws)
        x = pc.make([0] * 4, chunks, Hq, Hkv, d, page, torch.float32, True, seed=seed[0])
        for n in ("k_pages", "v_pages", "g_pages", "k_table", "v_table", "lens"):
            x[n] = getattr(c, n)
        x["n"] = c.lens.tolist()
        ref, Ks, Vs, Gs = pc.reference(dict(x, **pc.snapshot(x)))
        out = pc.step(lib, x, c, workspace=ws)
        pc.close(out, ref, torch.float32, "out")
        c.lens += x["cu"][1:] - x["cu"][:-1]
        for s in range(4):
            n = int(c.lens[s])
            pc.close(pc.rows_of(c.k_pages, c.k_table[s], n), Ks[s], torch.float32, "keys")
            assert torch.equal(pc.rows_of(c.v_pages, c.v_table[s], n), Vs[s])

    advance([70, 0, 35, 0])
    lib.path_paged_fork([0, 0], [1, 3], c, workspace=ws)
    assert int((c.v_ref > 1).sum()) == 4  # the 64 tokens of four full value pages
    for _ in range(3):
        advance([1, 1, 1, 1])
    lib.path_paged_free([0, 2], c, workspace=ws)
    lib.path_paged_compact(c, workspace=ws)
    advance([20, 1, 0, 1])
    advance([1, 66, 1, 1])
    lib.path_paged_free([0, 1, 2, 3], c, workspace=ws)
    assert not c.k_ref.any() and not c.v_ref.any()
    assert lib.path_check_workspace(ws) == lib.OK


def test_captured_page_calls(lib):
    """A captured step that reserves its pages itself, replayed until the cache is full."""
    c = lib.new_paged_cache(2, 4, 20, Hq=2, page=16, d=64)
    ws = lib.new_paged_workspace(c, 10, 5)
    x = pc.make([0, 0], [5, 5], 2, 2, 64, 16, torch.bfloat16, False, seed=2)
    extra = torch.tensor([5, 5], dtype=torch.int32, device="cuda")
    out = torch.empty_like(x["q"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        lib.path_paged_reserve(extra, c, workspace=ws)
        pc.step(lib, x, c, out=out, workspace=ws)
        c.lens += extra
    for turn in range(12):
        g.replay()
    assert lib.path_check_workspace(ws) == lib.OK
    assert c.lens.tolist() == [60, 60]
    assert int(c.k_ref.sum()) == 8
    g.replay()  # 65 tokens do not fit four pages of 16
    assert lib.path_check_workspace(ws) == lib.ERR_CAPACITY


def test_captured_fork_free_and_compact(lib):
    """One graph that forks a sequence twice, steps all three, drops the first fork and packs the
    pools; each replay leaves what the calls made one by one leave, and the lists of rows may
    change after the capture."""
    def fresh():
        c = cache(lib, [40, 0, 0, 90], page=16, Hq=4, Hkv=2, d=64, dtype=torch.bfloat16, fox=True, spare=40, seed=5)
        return c, lib.new_paged_workspace(c, 16, 8, Hq=4)

    x = pc.make([0] * 4, [3, 1, 8, 4], 4, 2, 64, 16, torch.bfloat16, True, seed=6)
    extra = x["cu"][1:] - x["cu"][:-1]
    src, dst, gone = [0, 3], [1, 2], [1, 2]

    def turn(c, ws):
        lib.path_paged_fork(src, dst, c, workspace=ws)
        lib.path_paged_reserve(extra, c, workspace=ws)
        out = pc.step(lib, x, c, workspace=ws)
        c.lens += extra
        lib.path_paged_free(gone, c, workspace=ws)
        lib.path_paged_compact(c, workspace=ws)
        return out

    def contents(c):
        live_k, live_v = c.k_ref > 0, c.v_ref > 0
        return [c.k_table, c.v_table, c.k_ref, c.v_ref, c.lens, c.k_pages[live_k].nan_to_num(nan=7.0),
                c.v_pages[live_v].nan_to_num(nan=7.0), c.g_pages[live_k].nan_to_num(nan=7.0)]

    a, wa = fresh()
    outs = [turn(a, wa) for _ in range(3)]
    b, wb = fresh()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = turn(b, wb)
    for lists in (src, dst, gone):
        lists[:] = [0, 0]
    for out in outs:
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, out)
    assert lib.path_check_workspace(wa) == lib.OK and lib.path_check_workspace(wb) == lib.OK
    assert all(torch.equal(p, q) for p, q in zip(contents(a), contents(b)))
