"""Steps of sequences that continue a shared prefix (path_paged_prefix_extend, its gated form) against
the fp64 reference, and against copies of the prompt that take path_paged_extend."""
import pytest
import torch

from tests import paged_cases as pc
from tests import paged_prefix_cases as px
from tests.paged_window_cases import same_bits

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def run(lib, x, **kw):
    before = px.snapshot(x)
    out = px.step(lib, x, **kw)
    torch.cuda.synchronize()
    px.check(x, before, out)
    return out


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("d,Hq,Hkv,page", [(64, 2, 2, 16), (128, 4, 1, 32), (64, 3, 1, 16), (128, 8, 1, 64),
                                           (128, 20, 1, 128), (64, 8, 2, 256)])
def test_single_tokens(lib, dtype, fox, d, Hq, Hkv, page):
    # prefixes of many lengths, one of none, one that nobody continues, sequences without a prefix, an
    # idle one; rows in any order
    lens = [300, 0, 5, 128, 17, 1, 129, 40, 0, 65, 700]
    of = [-1, 0, 0, -1, 3, 3, -1, 0, 8, -1, -1]
    of[8] = -1
    of[9] = 8
    chunks = [0, 1, 1, 0, 1, 1, 1, 0, 0, 1, 0]
    x = px.make(lens, chunks, of, Hq, Hkv, d, page, dtype, fox, seed=1)
    run(lib, x)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("d,Hq,Hkv,page", [(64, 2, 2, 16), (64, 6, 2, 256), (128, 2, 2, 64), (128, 4, 1, 128)])
@pytest.mark.parametrize("lens,chunks,of", [
    ([100, 0, 0, 0], [0, 1, 64, 65], [-1, 0, 0, 0]),
    ([5, 64, 200, 300], [3, 17, 0, 0], [2, 3, -1, -1]),       # two prefixes, behind their sequences
    ([63, 1000, 130, 1], [64, 0, 128, 200], [1, -1, 1, -1]),  # a sequence without a prefix among them
    ([700, 0, 33, 1], [0, 130, 1, 2], [-1, 0, 0, 0]),
])
def test_chunks(lib, dtype, fox, d, Hq, Hkv, page, lens, chunks, of):
    x = px.make(lens, chunks, of, Hq, Hkv, d, page, dtype, fox, seed=2)
    run(lib, x)


@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("d,Hq,Hkv", [(64, 4, 4), (128, 16, 2)])
@pytest.mark.parametrize("members", [3, 33, 70, 140])
def test_many_sequences_of_one_prefix(lib, fox, d, Hq, Hkv, members):
    # row tiles of one and two, with copies of the rows and without
    x = px.make([1500] + [i % 7 for i in range(members)], [0] + [1] * members, [-1] + [0] * members, Hq, Hkv, d, 64,
                BF, fox, seed=3)
    run(lib, x)


def test_more_sequences_than_a_round_of_the_plan(lib):
    S = 600
    g = torch.Generator().manual_seed(4)
    of = [-1] * 20 + torch.randint(-1, 20, (S - 20,), generator=g).tolist()
    chunks = [0] * 20 + torch.randint(0, 3, (S - 20,), generator=g).tolist()
    x = px.make([30 + i for i in range(20)] + [i % 3 for i in range(S - 20)], chunks, of, 2, 1, 64, 16, BF, False, seed=4)
    run(lib, x)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("chunks", [[1, 0, 1], [70, 0, 9]])
def test_strides_and_rows_behind_the_last_sequence(lib, dtype, chunks):
    x = px.make([20, 350, 0], chunks, [1, -1, 1], 4, 2, 64, 32, dtype, True, seed=5, head_major=True, tail=7)
    N = x["q"].shape[0]
    out = torch.full((4, N, 64), 7.0, dtype=dtype, device="cuda").transpose(0, 1)
    run(lib, x, out=out)
    assert (out[sum(chunks):] == 7).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("chunks", [[0, 1, 1], [0, 66, 9]])
def test_out_in_the_place_of_an_input(lib, dtype, chunks):
    for name in ("q", "w"):
        x = px.make([200, 3, 0], chunks, [-1, 0, 0], 2, 2, 64, 32, dtype, True, seed=6)
        before = px.snapshot(x)
        ref = px.reference(x)
        out = px.step(lib, x, out=x[name])
        torch.cuda.synchronize()
        pc.close(out, ref[0], dtype, "out")
        assert float((x["carry"].double() - ref[4]).abs().max()) <= 1e-5
        assert not torch.equal(x["carry"], before["carry"])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("chunks", [[0, 1, 1], [0, 66, 9]])
def test_no_prefix_at_all_is_the_plain_step(lib, dtype, chunks):
    a = px.make([300, 0, 77], chunks, [-1, -1, -1], 4, 2, 64, 32, dtype, True, seed=7)
    b = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in a.items()}
    one, two = pc.step(lib, a), px.step(lib, b)
    torch.cuda.synchronize()
    for n in ("k_pages", "v_pages", "g_pages"):
        assert same_bits(a[n], b[n]), n
    assert same_bits(one, two) and torch.equal(a["carry"], b["carry"])


@pytest.mark.parametrize("chunks", [[0, 1, 1, 1], [0, 3, 70, 1]])
def test_repeats_and_a_replayed_graph_give_the_same_bits(lib, chunks):
    x = px.make([900, 30, 100, 0], chunks, [-1, 0, 0, 0], 8, 2, 128, 64, BF, True, seed=8)
    before = px.snapshot(x)
    cache = pc.cache_of(lib, x)
    ws = lib.new_paged_workspace(cache, sum(chunks), max(chunks), prefix=True)
    out = torch.empty_like(x["q"])
    px.step(lib, x, cache, workspace=ws, out=out)
    torch.cuda.synchronize()
    first = [out.clone()] + [x[n].clone() for n in before]
    px.check(x, before, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        px.step(lib, x, cache, workspace=ws, out=out)
    for _ in range(2):
        for n in before:
            x[n].copy_(before[n])
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(first, [out] + [x[n] for n in before]):
            assert same_bits(a, b)
    # the same graph with the sequences behind another prefix, the device's lists alone changed
    for n in before:
        x[n].copy_(before[n])
    x["prefix_of"].copy_(torch.tensor([-1, 0, -1, 0], dtype=torch.int32))
    x["of"] = [-1, 0, -1, 0]
    g.replay()
    torch.cuda.synchronize()
    px.check(x, before, out)
    assert lib.path_check_workspace(ws) == lib.OK


@pytest.mark.parametrize("of,chunks,bad", [
    ([-1, 1, 0], [0, 1, 1], 1),       # its own prefix
    ([-1, 3, 0], [0, 1, 1], 1),       # no row of the cache
    ([-1, 2, -1], [0, 1, 1], 1),      # a row with tokens of its own
    ([2, -1, 0], [0, 1, 1], 2),       # a prefix behind a prefix
])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 5])
def test_what_cannot_be_a_prefix(lib, dtype, of, chunks, bad, T):
    chunks = [c * T for c in chunks]
    x = px.make([100, 20, 30], chunks, of, 4, 2, 64, 16, dtype, False, seed=9)
    before = px.snapshot(x)
    cache = pc.cache_of(lib, x)
    ws = lib.new_paged_workspace(cache, sum(chunks), T, Hq=4, prefix=True)
    out = torch.full_like(x["q"], 7.0)
    px.step(lib, x, cache, workspace=ws, out=out)
    assert lib.path_check_workspace(ws) == lib.ERR_CACHE
    # as if it had had no tokens
    cu = x["cu"].tolist()
    assert (out[cu[bad]:cu[bad + 1]] == 7).all()
    assert torch.equal(x["carry"][bad], before["carry"][bad])
    ids = x["k_table"][bad]
    ids = ids[ids >= 0].long()
    assert same_bits(x["k_pages"][ids], before["k_pages"][ids])
    others = [s for s in range(3) if s != bad and chunks[s]]
    for s in others:
        assert torch.isfinite(out[cu[s]:cu[s + 1]].float()).all()


def test_idle_rows_may_name_anything(lib):
    x = px.make([100, 20, 30], [0, 0, 1], [1 << 30, 1, 0], 4, 2, 64, 16, BF, False, seed=10)
    x["prefix_of"][0] = -7
    x["of"][0] = -7
    run(lib, x)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("T", [1, 3, 80])
def test_samples_of_a_prompt(lib, dtype, fox, T):
    """A prompt is read once; samples continue it behind a prefix, and, beside them, in forks that
    copy its keys: both give the same outputs, the fp64 reference's."""
    page, Hq, Hkv, d, S, n, steps = 32, 4, 2, 64, 3, 333, 4
    g = torch.Generator(device="cuda").manual_seed(11)

    def tokens(N):
        r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        w = r(N, Hkv, d)
        return dict(q=r(N, Hq, d).to(dtype), k=r(N, Hkv, d).to(dtype), v=r(N, Hkv, d).to(dtype),
                    w=(w / w.norm(dim=-1, keepdim=True)).to(dtype),
                    beta=(2 * r(N, Hkv).sigmoid()).clamp(max=1.99),
                    log_f=torch.nn.functional.logsigmoid(r(N, Hq) + 2) if fox else None)

    prompt, parts = tokens(n), [[tokens(T) for _ in range(S)] for _ in range(steps)]
    rows = 1 + 2 * S  # the prompt, samples behind it, forks of it
    width = pc.pages(n + steps * T, page)
    cache = lib.new_paged_cache(rows, width, (rows + 1) * width, Hq=Hq, Hkv=Hkv, d=d, page=page, dtype=dtype, fox=fox)
    carry, gates = lib.new_paged_carry(cache, Hq=Hq)
    most = max(n, 2 * S * T)
    ws = lib.new_paged_workspace(cache, most, max(n, T), Hq=Hq, prefix=True)
    prefix_of = torch.tensor([-1] + [0] * S + [-1] * S, dtype=torch.int32, device="cuda")

    def go(x, counts):
        new = torch.tensor(counts, dtype=torch.int32, device="cuda")
        cu = torch.cat([new.new_zeros(1), new.cumsum(0).int()])
        lib.path_paged_reserve(new, cache, workspace=ws)
        a = (x["q"], x["k"], x["v"], x["w"], x["beta"])
        if fox:
            out = lib.path_fox_paged_prefix_extend(*a, x["log_f"], cu, cache, prefix_of, carry, gates, max(counts),
                                                   workspace=ws)
        else:
            out = lib.path_paged_prefix_extend(*a, cu, cache, prefix_of, carry, max(counts), workspace=ws)
        cache.lens += new
        return out

    go(prompt, [n] + [0] * (2 * S))
    kept = cache.k_pages[cache.k_table[0, :pc.pages(n, page)].long()].clone()
    lib.path_paged_fork([0] * S, [1 + S + i for i in range(S)], cache, workspace=ws)
    whole = [{k: (None if prompt[k] is None else prompt[k]) for k in prompt} for _ in range(S)]
    for step in range(steps):
        x = {k: None if prompt[k] is None else torch.cat([parts[step][i][k] for i in range(S)] * 2) for k in prompt}
        out = go(x, [0] + [T] * (2 * S))
        assert lib.path_check_workspace(ws) == lib.OK
        for i in range(S):
            whole[i] = {k: None if whole[i][k] is None else torch.cat([whole[i][k], parts[step][i][k]])
                        for k in prompt}
            y = dict(whole[i], n=[0], chunks=[n + (step + 1) * T], Hq=Hq, Hkv=Hkv, d=d,
                     k_pages=cache.k_pages, v_pages=cache.v_pages, g_pages=cache.g_pages,
                     k_table=cache.k_table[:1], v_table=cache.v_table[:1])
            ref = pc.reference(y)[0][-T:]
            behind, forked = out[i * T:(i + 1) * T], out[(S + i) * T:(S + i + 1) * T]
            if dtype == F32:
                pc.close(behind, ref, dtype, "out")
                pc.close(forked, ref, dtype, "out")
            else:
                # of a key the prompt's own rounding and one more for each step that advances it (none behind
                # the prefix, up to 4 of the fork's), 2.3e-3 of its logit at most each, beside a step's 4.5e-3
                for o, k in ((behind, 1), (forked, 1 + step)):
                    err = float((o.double() - ref).norm() / ref.norm())
                    assert err <= (4.5e-3 ** 2 + k * 2.3e-3 ** 2) ** 0.5, (step, i, k, err)
    assert same_bits(cache.k_pages[cache.k_table[0, :pc.pages(n, page)].long()], kept)
