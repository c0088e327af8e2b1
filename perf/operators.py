"""The paged-cache operators of PaTH attention as measurable cases.

Each case is one call that a serving program makes: a step of new tokens through
path_paged_extend / path_fox_paged_extend (attention of every sequence's new tokens over its
paged cache, whose keys take the new tokens' transitions in place), or the calls that manage
the cache's pages (path_paged_free, path_paged_fork, path_paged_reserve, path_paged_compact).
With `own` false the same results are formed with elementary torch operations in 32 bits.

Per sequence with n cached tokens and T new ones, and H_s = I - beta_s w_s w_s^T:
    u_t = beta_t (w_t - sum_{s<t} (w_s . w_t) u_s),  so that H_1 ... H_i = I - sum_{s<=i} u_s w_s^T
    cached key j:   logit scale * k_j . (H_1 ... H_i q_i) (+ g_j + sum_{s<=i} log f_s)
    new key j <= i: logit scale * k_j . (H_{j+1} ... H_i q_i) (+ sum_{j<s<=i} log f_s)
    keys after the step: (H_1 ... H_T)^T k_j, or (H_{j+1} ... H_T)^T k_j for a new one.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- the cases

def listed():
    e, f, c = {"op": "extend"}, {"op": "fork"}, {"op": "compact"}
    return [
        # one user, one short conversation, one token: what a step costs at the least
        dict(e, name="one token", B=1, Hq=8, Hkv=8, d=64, page=16, n=300, T=1, mix="one",
             fox=False, dtype="bf16"),
        # a batch of conversations, one token each
        dict(e, name="decode batch", B=32, Hq=16, Hkv=16, d=64, page=64, n=8192, T=1, mix="one",
             fox=False, dtype="bf16"),
        # the same with forget gates, and four query heads to a key head
        dict(e, name="decode gates shared", B=16, Hq=32, Hkv=8, d=128, page=64, n=16384, T=1,
             mix="one", fox=True, dtype="bf16"),
        # a few tokens each: a short user turn, or several tokens taken at once
        dict(e, name="few tokens", B=8, Hq=16, Hkv=4, d=64, page=32, n=6000, T=7, mix="ragged",
             fox=False, dtype="bf16"),
        # a step that mixes one prompt's chunk with many single tokens
        dict(e, name="mixed batch", B=32, Hq=16, Hkv=16, d=64, page=64, n=4096, T=512, mix="mixed",
             fox=False, dtype="bf16"),
        # first chunks of prompts: nothing is cached yet
        dict(e, name="first chunks", B=4, Hq=16, Hkv=8, d=64, page=64, n=0, T=1500, mix="ragged",
             fox=True, dtype="bf16"),
        # a long chunk late in a long document
        dict(e, name="long chunk", B=1, Hq=32, Hkv=8, d=128, page=128, n=32768, T=2048, mix="even",
             fox=False, dtype="bf16"),
        # a reference run in full precision
        dict(e, name="fp32 chunk", B=2, Hq=4, Hkv=4, d=64, page=32, n=1000, T=130, mix="ragged",
             fox=True, dtype="fp32"),
        # a beam of one request takes over from its best member
        dict(f, name="fork beam", S=8, pairs=3, Hq=8, Hkv=8, d=64, page=16, n=700, extra=1,
             fox=False, dtype="bf16"),
        # samples drawn from several long prompts
        dict(f, name="fork prompts", S=24, pairs=16, Hq=16, Hkv=8, d=128, page=64, n=12000,
             extra=64, fox=True, dtype="bf16"),
        # a small pool after a few requests have ended
        dict(c, name="compact small", S=6, Hq=4, Hkv=4, d=64, page=16, pages=300, live=0.5,
             fox=True, dtype="bf16"),
        # a large pool after many have
        dict(c, name="compact large", S=48, Hq=8, Hkv=8, d=128, page=64, pages=9000, live=0.6,
             fox=False, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["extend", "extend", "extend", "extend", "fork", "compact"])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    hkv = rng.choice([1, 2, 4, 8, 16])
    hq = hkv * rng.choice([1, 1, 2, 4, 8] if hkv <= 4 else [1, 2, 4] if hkv == 8 else [1, 2])
    fox = rng.random() < 0.5
    dtype = "fp32" if rng.random() < 0.2 else "bf16"
    base = dict(op=kind, Hq=hq, Hkv=hkv, d=d, page=page, fox=fox, dtype=dtype)
    if kind == "extend":
        mix = rng.choice(["one", "ragged", "ragged", "even", "mixed"])
        T = 1 if mix == "one" else _log_int(rng, 2, 300 if dtype == "fp32" else 2000)
        n = 0 if rng.random() < 0.1 else _log_int(rng, 1, 2000 if dtype == "fp32" else 30000)
        # batch: bounded by the cache's bytes and by the logits of the step
        per_cache = (n + T) * hkv * d
        per_logit = hq * T * (n + T)
        most = int(max(1, min(48, 1.0e8 / per_cache, 1.2e9 / per_logit)))
        if dtype == "fp32":
            most = int(max(1, min(most, 1.0e8 / per_logit)))
        return dict(base, B=_log_int(rng, 1, most), n=n, T=T, mix=mix)
    if kind == "fork":
        pairs = _log_int(rng, 1, 16)
        n = _log_int(rng, 1, 12000)
        n = min(n, int(2.0e8 / (hkv * d * pairs)) + 1)
        return dict(base, S=pairs + rng.randint(1, 8), pairs=pairs, n=n,
                    extra=rng.choice([1, 5, 64, 200]))
    pages = _log_int(rng, 40, 9000)
    pages = min(pages, int(5.0e8 / (hkv * d * page)) + 4)
    return dict(base, S=rng.randint(2, 48), pages=pages, live=round(rng.uniform(0.2, 0.9), 2))


def _lengths(case):
    """(cached lengths, chunk lengths) of an extend case: the same for every seed."""
    r = random.Random("%d %d %d %s" % (case["B"], case["n"], case["T"], case["mix"]))
    n = [case["n"] - r.randint(0, case["n"] // 2) for _ in range(case["B"])]
    n[0] = case["n"]
    T = []
    for b in range(case["B"]):
        if case["mix"] in ("one", "even") or b == 0:
            T.append(case["T"])
        elif case["mix"] == "mixed":
            T.append(1)
        else:
            T.append(r.randint((case["T"] + 3) // 4, case["T"]))
    return n, T


def _pages(tokens, page):
    return -(-tokens // page)


def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    Hq, Hkv, d, page = case["Hq"], case["Hkv"], case["d"], case["page"]
    row = Hkv * d * e
    gate = 4 * Hq if case["fox"] else 0
    if case["op"] == "extend":
        byts = flops = 0
        for n, T in zip(*_lengths(case)):
            byts += n * (3 * row + 2 * gate)                     # keys in and out, values in, gates
            byts += T * (5 * row + 2 * Hq * d * e + 4 * Hkv + 2 * gate)
            flops += 4 * Hq * d * (T * n + T * (T + 1) // 2)     # logits and weighted values
            flops += 2 * Hkv * d * n * min(2 * T, d)             # the keys' transitions
            flops += 6 * Hkv * d * T * min(T, 64)                # the block factors
        return {"bytes": byts, "flops": flops}
    if case["op"] == "fork":
        tokens = sum(_fork_lens(case)[:case["pairs"]])
        part = sum(n % page for n in _fork_lens(case)[:case["pairs"]])
        return {"bytes": 2 * tokens * (row + gate) + 2 * part * row + 4 * sum(_fork_pool(case)),
                "flops": 0}
    live = _live(case)
    nlive = sum(live)
    moved = sum(live[nlive:])
    per = page * (2 * row + gate)
    return {"bytes": 2 * moved * per + 8 * case["pages"] + 8 * nlive, "flops": 0}


def _fork_lens(case):
    r = random.Random("fork %d %d" % (case["n"], case["S"]))
    n = [case["n"] - r.randint(0, case["n"] // 2) for _ in range(case["S"])]
    n[0] = case["n"]
    return n


def _fork_pool(case):
    """(key pages, value pages) of a fork case's pool: the live sequences', the children's, and
    a tenth to spare."""
    page, pairs = case["page"], case["pairs"]
    lens = _fork_lens(case)
    sources = [_pages(n, page) for n in lens[:case["S"] - pairs]]
    kids = [_pages(lens[i % len(sources)] + case["extra"], page) for i in range(pairs)]
    before = [_pages(lens[len(sources) + i], page) for i in range(pairs)]
    room = sum(sources) + max(sum(kids), sum(before)) + sum(before) + 8
    return room + room // 10, room + room // 10


def _live(case):
    r = random.Random("live %d %g" % (case["pages"], case["live"]))
    return [r.random() < case["live"] for _ in range(case["pages"])]


# ---------------------------------------------------------------- inputs

def _gate_sums(g, n, H):
    """Gate sums (H, n) that log f = logsigmoid(N(2, 1)) leaves behind: entry j sums the gates
    of the tokens after j."""
    lf = torch.nn.functional.logsigmoid(torch.randn((H, n), generator=g, device="cuda") + 2.0)
    tail = lf.double().flip(-1).cumsum(-1).flip(-1)
    return torch.cat([tail[:, 1:], tail.new_zeros((H, min(n, 1)))], -1).float()


def _pool(case, g, pages):
    dt = _DT[case["dtype"]]
    shape = (pages, case["Hkv"], case["page"], case["d"])
    k = torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)
    v = torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)
    return k, v


def _prepare_extend(case, g):
    B, Hq, Hkv, d, page = (case[x] for x in ("B", "Hq", "Hkv", "d", "page"))
    dt = _DT[case["dtype"]]
    n, T = _lengths(case)
    need = [_pages(a + b, page) for a, b in zip(n, T)]
    total = sum(need) + 3
    k_pages, v_pages = _pool(case, g, total)
    width = max(need) + 1
    k_table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    v_table = k_table.clone()
    # pages in the order in which a pool that has been in use for a while hands them out: any
    ids = [torch.randperm(total, generator=g, device="cuda").int() for _ in range(2)]
    at = 0
    for b in range(B):
        k_table[b, :need[b]] = ids[0][at:at + need[b]]
        v_table[b, :need[b]] = ids[1][at:at + need[b]]
        at += need[b]
    N = sum(T)
    x = {"q": torch.randn((N, Hq, d), generator=g, device="cuda").to(dt)}
    for name in ("k", "v"):
        x[name] = torch.randn((N, Hkv, d), generator=g, device="cuda").to(dt)
    w = torch.randn((N, Hkv, d), generator=g, device="cuda")
    x["w"] = (w / w.norm(dim=-1, keepdim=True)).to(dt)
    x["beta"] = (2 * torch.randn((N, Hkv), generator=g, device="cuda").sigmoid()).clamp(max=1.99)
    s = dict(x, k_pages=k_pages, v_pages=v_pages, g_pages=None, log_f=None, k_table=k_table,
             v_table=v_table, lens=torch.tensor(n, dtype=torch.int32, device="cuda"),
             cu=torch.tensor([sum(T[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda"),
             page=page, n_max=max(n), t_max=max(T), case=case)
    if case["fox"]:
        s["log_f"] = torch.nn.functional.logsigmoid(
            torch.randn((N, Hq), generator=g, device="cuda") + 2.0)
        s["g_pages"] = torch.zeros((total, Hq, page), device="cuda")
        for b in range(B):
            m = _pages(n[b], page)
            if m:
                row = torch.zeros((Hq, m * page), device="cuda")
                row[:, :n[b]] = _gate_sums(g, n[b], Hq)
                s["g_pages"][k_table[b, :m].long()] = row.view(Hq, m, page).transpose(0, 1)
    return s


def _prepare_fork(case, g):
    S, page, pairs = case["S"], case["page"], case["pairs"]
    lens = _fork_lens(case)
    pk, pv = _fork_pool(case)
    k_pages, v_pages = _pool(case, g, pk)
    need = [_pages(n, page) for n in lens]
    width = _pages(case["n"] + case["extra"], page) + 1
    tables, refs = [], []
    for total in (pk, pv):
        ids = torch.randperm(total, generator=g, device="cuda").int()
        t = torch.full((S, width), -1, dtype=torch.int32, device="cuda")
        ref = torch.zeros(total, dtype=torch.int32, device="cuda")
        at = 0
        for s in range(S):
            t[s, :need[s]] = ids[at:at + need[s]]
            at += need[s]
        ref[ids[:at].long()] = 1
        tables.append(t)
        refs.append(ref)
    kept = S - pairs
    extra = [0] * kept + [case["extra"]] * pairs
    s = dict(k_pages=k_pages, v_pages=v_pages, g_pages=None, k_table=tables[0], v_table=tables[1],
             k_ref=refs[0], v_ref=refs[1], lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             src=[i % kept for i in range(pairs)], dst=[kept + i for i in range(pairs)],
             extra=torch.tensor(extra, dtype=torch.int32, device="cuda"), page=page, case=case)
    if case["fox"]:
        s["g_pages"] = -torch.rand((pk, case["Hq"], page), generator=g, device="cuda") * 50
    return s


def _prepare_compact(case, g):
    P, S, page = case["pages"], case["S"], case["page"]
    k_pages, v_pages = _pool(case, g, P)
    ids = [i for i, x in enumerate(_live(case)) if x]
    ref = torch.zeros(P, dtype=torch.int32, device="cuda")
    ref[ids] = 1
    width = _pages(len(ids), S) + 1
    t = torch.full((2, S * width), -1, dtype=torch.int32, device="cuda")
    live = torch.tensor(ids, dtype=torch.int32, device="cuda")
    for r in t:
        order = torch.randperm(len(ids), generator=g, device="cuda")
        slots = torch.arange(len(ids), device="cuda")
        r[(slots % S) * width + slots // S] = live[order]
    t = t.view(2, S, width)
    lens = (t[0] >= 0).sum(-1).int() * page
    s = dict(k_pages=k_pages, v_pages=v_pages, g_pages=None, page=page, case=case, lens=lens,
             before=(t[0].clone(), t[1].clone(), ref.clone(), ref.clone()),
             k_table=t[0].clone(), v_table=t[1].clone(), k_ref=ref.clone(), v_ref=ref.clone())
    if case["fox"]:
        s["g_pages"] = -torch.rand((P, case["Hq"], page), generator=g, device="cuda") * 50
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    return {"extend": _prepare_extend, "fork": _prepare_fork,
            "compact": _prepare_compact}[case["op"]](case, g)


# ---------------------------------------------------------------- plain forms

def _gather(pages, table, n_max, page):
    """(B, H, n_max', d) fp32 of the first n_max positions of every sequence."""
    m = _pages(n_max, page)
    x = pages[table[:, :m].clamp(min=0).long()]                   # B, m, H, page[, d]
    x = x.transpose(1, 2).flatten(2, 3)
    return x[:, :, :n_max].float()


def _places(table, start, count, page, most):
    """(page ids, offsets, mask) of positions start .. start + count - 1 of every sequence."""
    t = torch.arange(most, device="cuda")
    pos = start[:, None] + t
    mask = t < count[:, None]
    slot = (pos // page).clamp(max=table.shape[1] - 1)
    return table.gather(1, slot.long()).long(), pos % page, mask


def _put(pages, where, values):
    """values (B, H, most[, d]) into their pages."""
    ids, off, mask = where
    pages[ids[mask], :, off[mask]] = values.transpose(1, 2)[mask].to(pages.dtype)


def _plain_extend(s):
    q, k, v, w = (s[x].float() for x in ("q", "k", "v", "w"))
    n, cu = s["lens"].long(), s["cu"].long()
    T = cu[1:] - cu[:-1]
    N, page, n_max, t_max = q.shape[0], s["page"], s["n_max"], s["t_max"]
    Hq, Hkv, d = q.shape[1], k.shape[1], q.shape[2]
    G = Hq // Hkv
    t = torch.arange(t_max, device="cuda")
    real = t < T[:, None]                                         # B, t_max
    at = (cu[:-1, None] + t).clamp(max=N - 1)
    pad = lambda x: (x[at] * real[:, :, None, None]).transpose(1, 2)  # noqa: E731
    qp, kp, vp, wp = pad(q), pad(k), pad(v), pad(w)               # B, H, t_max, d
    beta = (s["beta"][at] * real[:, :, None]).transpose(1, 2)
    heads = lambda x: x.repeat_interleave(G, 1)  # noqa: E731
    scale = d ** -0.5
    # A = (I + D strictly-lower(W W^T))^-1 D over the whole chunk, u = A w
    E = (wp @ wp.transpose(-1, -2)).tril(-1) * beta[..., None]
    E = E + torch.eye(t_max, device="cuda")
    A = torch.linalg.solve_triangular(E, torch.diag_embed(beta), upper=False, unitriangular=True)
    Lq = (qp @ heads(wp).transpose(-1, -2)).tril()                # s <= i
    R = (kp @ wp.transpose(-1, -2)).triu(1)                       # t > j
    LA = Lq @ heads(A)
    qt = qp - LA @ heads(wp)
    Snew = (qp @ heads(kp).transpose(-1, -2) - LA @ heads(R).transpose(-1, -2)) * scale
    K, V = (_gather(s[x], s[y], n_max, page) for x, y in (("k_pages", "k_table"), ("v_pages", "v_table")))
    Sold = (qt @ heads(K).transpose(-1, -2)) * scale
    have = torch.arange(n_max, device="cuda") < n[:, None]
    if s["log_f"] is not None:
        lf = (s["log_f"][at] * real[:, :, None]).transpose(1, 2).double()
        c = lf.cumsum(-1)                                         # B, Hq, t_max
        G_old = _gather(s["g_pages"], s["k_table"], n_max, page)
        Sold = Sold + (G_old.double()[:, :, None] + c[..., None]).float()
        Snew = Snew + (c[..., None] - c[:, :, None]).float()
    Sold = Sold.masked_fill(~have[:, None, None], -math.inf)
    Snew = Snew.masked_fill(t[None, :] > t[:, None], -math.inf)
    m = Snew.amax(-1, keepdim=True)
    if n_max:
        m = torch.maximum(m, Sold.amax(-1, keepdim=True))
    Pold, Pnew = (Sold - m).exp(), (Snew - m).exp()
    del Sold, Snew
    V = V.masked_fill(~have[:, None, :, None], 0)
    o = (Pold @ heads(V) + Pnew @ heads(vp)) / (Pold.sum(-1, keepdim=True) + Pnew.sum(-1, keepdim=True))
    out = o.transpose(1, 2)[real].to(s["q"].dtype)
    # the cache after the step
    U = A @ wp
    K2 = K - (K @ U.transpose(-1, -2)) @ wp
    k2 = kp - (R @ A.transpose(-1, -2)) @ wp
    old = _places(s["k_table"], torch.zeros_like(n), n, page, n_max)
    new = _places(s["k_table"], n, T, page, t_max)
    _put(s["k_pages"], old, K2)
    _put(s["k_pages"], new, k2)
    _put(s["v_pages"], _places(s["v_table"], n, T, page, t_max), vp)
    if s["log_f"] is not None:
        end = c[..., -1:]
        _put(s["g_pages"], old, G_old.double() + end)
        _put(s["g_pages"], new, end - c)
    return out


def _plain_free(s, rows):
    for table, ref in (("k_table", "k_ref"), ("v_table", "v_ref")):
        ids = s[table][rows]
        ids = ids[ids >= 0].long()
        s[ref].index_add_(0, ids, torch.full_like(ids, -1, dtype=torch.int32))
        s[table][rows] = -1
    s["lens"][rows] = 0


def _copy_rows(pages, new, old, rows):
    """Of every page `old`, its first `rows` token rows into page `new`."""
    page = pages.shape[2]
    mask = torch.arange(page, device="cuda") < rows[:, None]
    mask = mask[:, None, :, None] if pages.dim() == 4 else mask[:, None]
    pages[new] = torch.where(mask, pages[old], pages[new])


def _plain_fork(s, src, dst):
    n, page = s["lens"][src].long(), s["page"]
    slots = torch.arange(s["k_table"].shape[1], device="cuda")
    used = slots < (-(-n // page))[:, None]
    full = slots < (n // page)[:, None]
    rows = (n[:, None] - slots * page).clamp(0, page)
    # keys: every page anew
    new = (s["k_ref"] == 0).nonzero()[:, 0][:int(used.sum())]
    old = s["k_table"][src][used].long()
    row = torch.full_like(s["k_table"][src], -1)
    row[used] = new.int()
    s["k_table"][dst] = row
    s["k_ref"][new] = 1
    _copy_rows(s["k_pages"], new, old, rows[used])
    if s["g_pages"] is not None:
        _copy_rows(s["g_pages"], new, old, rows[used])
    # values: full pages are shared, a last page that still fills is copied
    part = used & ~full
    new = (s["v_ref"] == 0).nonzero()[:, 0][:int(part.sum())]
    row = torch.where(full, s["v_table"][src], -1)
    old = s["v_table"][src][part].long()
    row[part] = new.int()
    s["v_table"][dst] = row
    both = s["v_table"][src][full].long()
    s["v_ref"].index_add_(0, both, torch.ones_like(both, dtype=torch.int32))
    s["v_ref"][new] = 1
    _copy_rows(s["v_pages"], new, old, rows[part])
    s["lens"][dst] = n.int()


def _plain_reserve(s, extra):
    page = s["page"]
    upto = -(-(s["lens"] + extra).long() // page)
    for table, ref in (("k_table", "k_ref"), ("v_table", "v_ref")):
        slots = torch.arange(s[table].shape[1], device="cuda")
        want = (slots < upto[:, None]) & (s[table] < 0)
        new = (s[ref] == 0).nonzero()[:, 0][:int(want.sum())]
        s[table][want] = new.int()
        s[ref][new] = 1


def _plain_compact(s):
    for table, ref, pools in (("k_table", "k_ref", ("k_pages", "g_pages")),
                              ("v_table", "v_ref", ("v_pages",))):
        live = s[ref] > 0
        nlive = int(live.sum())
        hole = (~live[:nlive]).nonzero()[:, 0]
        move = live[nlive:].nonzero()[:, 0] + nlive
        to = torch.arange(live.numel(), device="cuda", dtype=torch.int32)
        to[move] = hole.int()
        for p in pools:
            if s[p] is not None:
                s[p][hole] = s[p][move]
        s[ref][hole] = s[ref][move]
        s[ref][move] = 0
        t = s[table]
        s[table].copy_(torch.where(t >= 0, to[t.clamp(min=0).long()], t))


# ---------------------------------------------------------------- one pass

_STATE = ("k_pages", "v_pages", "g_pages", "k_table", "v_table", "k_ref", "v_ref", "lens")


def _cache(s, pa):
    return pa.PathPagedCache(**{x: s.get(x) for x in _STATE})


def _answer(s, out=None):
    names = ("k_pages", "v_pages", "g_pages") if out is not None else _STATE
    r = {x: s[x] for x in names if s[x] is not None}
    if out is not None:
        r["out"] = out
    return r


def run(s):
    if own:
        import dependent_position_encoded_gb300 as pa
    if s["case"]["op"] == "extend":
        if own:
            cache = _cache(s, pa)
            if "ws" not in s:  # a serving loop keeps its workspace
                s["ws"] = pa.new_paged_workspace(cache, s["q"].shape[0], s["t_max"],
                                                   Hq=s["q"].shape[1])
            args = (s["q"], s["k"], s["v"], s["w"], s["beta"])
            if s["log_f"] is None:
                out = pa.path_paged_extend(*args, s["cu"], cache, s["t_max"], workspace=s["ws"])
            else:
                out = pa.path_fox_paged_extend(*args, s["log_f"], s["cu"], cache, s["t_max"],
                                               workspace=s["ws"])
        else:
            out = _plain_extend(s)
        return _answer(s, out)
    if s["case"]["op"] == "fork":
        # the rows that lost give up their pages and take over from their sources, with room
        # for what comes next
        if own:
            cache = _cache(s, pa)
            if "ws" not in s:
                s["ws"] = pa.new_paged_workspace(cache)
            pa.path_paged_free(s["dst"], cache, workspace=s["ws"])
            pa.path_paged_fork(s["src"], s["dst"], cache, workspace=s["ws"])
            pa.path_paged_reserve(s["extra"], cache, workspace=s["ws"])
        else:
            _plain_free(s, s["dst"])
            _plain_fork(s, s["src"], s["dst"])
            _plain_reserve(s, s["extra"])
        return _answer(s)
    # a pass begins from the scattered pool: its tables and counts are put back, and the pages
    # that a pass moves away from still hold what they held
    for x, y in zip(("k_table", "v_table", "k_ref", "v_ref"), s["before"]):
        s[x].copy_(y)
    if own:
        cache = _cache(s, pa)
        if "ws" not in s:
            s["ws"] = pa.new_paged_workspace(cache)
        pa.path_paged_compact(cache, workspace=s["ws"])
    else:
        _plain_compact(s)
    return _answer(s)


# ---------------------------------------------------------------- from the definition, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] != "extend":
        return None  # pages are moved, not computed
    n, T = _lengths(case)
    N, Hq, d = s["q"].shape
    Hkv, page = case["Hkv"], case["page"]
    G = Hq // Hkv
    f = torch.float64
    out = torch.zeros((N, Hq, d), dtype=f, device="cuda")
    kpg, vpg = s["k_pages"].to(f), s["v_pages"].to(f)
    gpg = None if s["g_pages"] is None else s["g_pages"].to(f)
    first = 0
    for b in range(case["B"]):
        total = n[b] + T[b]
        m = _pages(total, page)
        kid, vid = s["k_table"][b, :m].long(), s["v_table"][b, :m].long()
        K = kpg[kid].transpose(0, 1).reshape(Hkv, m * page, d)[:, :total].clone()
        V = vpg[vid].transpose(0, 1).reshape(Hkv, m * page, d)[:, :total].clone()
        if gpg is not None:
            g = gpg[kid].transpose(0, 1).reshape(Hq, m * page)[:, :total].clone()
        for t in range(T[b]):
            i, e = first + t, n[b] + t
            w, beta = s["w"][i].to(f), s["beta"][i].to(f)
            # every key so far takes the token's transition, then the token joins
            c = torch.einsum("hjd,hd->hj", K[:, :e], w) * beta[:, None]
            K[:, :e] -= c[..., None] * w[:, None]
            K[:, e], V[:, e] = s["k"][i].to(f), s["v"][i].to(f)
            x = torch.einsum("hgd,hjd->hgj", s["q"][i].to(f).view(Hkv, G, d), K[:, :e + 1])
            x = x.reshape(Hq, e + 1) / math.sqrt(d)
            if gpg is not None:
                g[:, :e] += s["log_f"][i].to(f)[:, None]
                g[:, e] = 0
                x = x + g[:, :e + 1]
            p = torch.softmax(x, -1).view(Hkv, G, e + 1)
            out[i] = torch.einsum("hgj,hjd->hgd", p, V[:, :e + 1]).reshape(Hq, d)
        put = torch.zeros((Hkv, m * page), dtype=torch.bool, device="cuda")
        put[:, :total] = True
        put = put.view(Hkv, m, page).transpose(0, 1)

        def back(pages, ids, X, H, put):
            full = pages[ids]
            new = torch.zeros((H, m * page) + X.shape[2:], dtype=f, device="cuda")
            new[:, :total] = X
            new = new.view((H, m, page) + X.shape[2:]).transpose(0, 1)
            pages[ids] = torch.where(put[..., None] if X.dim() == 3 else put, new, full)

        back(kpg, kid, K, Hkv, put)
        back(vpg, vid, V, Hkv, put)
        if gpg is not None:
            back(gpg, kid, g, Hq, put[:, :1].expand(-1, Hq, -1))
        first += T[b]
    r = {"k_pages": kpg, "v_pages": vpg, "out": out}
    if gpg is not None:
        r["g_pages"] = gpg
    return r
