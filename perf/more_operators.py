"""Shared prefixes and sliding windows over a paged cache as measurable cases.

Each case is one call that a serving program makes of these operators:
  prefix  path_paged_prefix_extend / path_fox_paged_prefix_extend: new tokens of sequences that
          continue a prefix which lies in the cache once and stays as it is
  window  path_paged_window_extend / path_fox_paged_window_extend: new tokens that see the last
          `window` tokens and the first `sinks` ones
  trim    path_paged_trim: the pages that no window reaches any more go back to the pools
With `own` false the same results are formed with elementary torch operations in 32 bits.

With H_s = I - beta_s w_s w_s^T, a sequence's n cached tokens and T new ones:
    logit of new token i with a cached key   scale * k_j . (H_1 ... H_i q_i) (+ g_j + sum_{s<=i} log f_s)
    with a new key j <= i                    scale * k_j . (H_{j+1} ... H_i q_i) (+ sum_{j<s<=i} log f_s)
    with a key of its prefix                 scale * k_j . (C H_1 ... H_i q_i) (+ g_j + c + sum_{s<=i} log f_s)
    keys after the step                      (H_1 ... H_T)^T k_j, (H_{j+1} ... H_T)^T k_j for a new one,
                                             unchanged for a key of the prefix, whose sequences'
                                             carries advance instead: C <- C H_1 ... H_T, c <- c + sum log f
    window: token i at position n + i sees position j where j > n + i - window or j < sinks; cached
    keys that no new token sees stay as they are.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- the cases

def listed():
    p, w, t = {"op": "prefix"}, {"op": "window"}, {"op": "trim"}
    return [
        # a few answers to one short prompt, one token each: what a step costs at the least
        dict(p, name="few samples", P=1, M=4, Hq=8, Hkv=8, d=64, page=16, n=500, tail=20, T=1,
             mix="even", fox=False, dtype="bf16"),
        # many samples of one long prompt, one token each
        dict(p, name="samples decode", P=1, M=32, Hq=16, Hkv=16, d=64, page=64, n=8192, tail=512,
             T=1, mix="even", fox=False, dtype="bf16"),
        # users of a few system prompts, with gates and four query heads to a key head
        dict(p, name="prompts gates", P=4, M=16, Hq=32, Hkv=8, d=128, page=64, n=16384, tail=256,
             T=1, mix="even", fox=True, dtype="bf16"),
        # branches of one text that bring a few tokens each: drafts to be checked
        dict(p, name="drafts", P=1, M=16, Hq=16, Hkv=4, d=64, page=32, n=6000, tail=40, T=7,
             mix="ragged", fox=False, dtype="bf16"),
        # questions to one long document: the first chunk behind the prefix
        dict(p, name="questions", P=1, M=8, Hq=32, Hkv=8, d=128, page=128, n=16384, tail=0, T=512,
             mix="ragged", fox=False, dtype="bf16"),
        # a reference run in full precision
        dict(p, name="fp32 samples", P=2, M=3, Hq=4, Hkv=2, d=64, page=32, n=1000, tail=70, T=33,
             mix="ragged", fox=True, dtype="fp32"),
        # one stream with a short window
        dict(w, name="window one token", B=1, Hq=8, Hkv=8, d=64, page=16, n=900, window=256,
             sinks=4, T=1, mix="even", fox=False, dtype="bf16"),
        # a batch of streams that are trimmed as they go
        dict(w, name="window decode", B=64, Hq=16, Hkv=16, d=64, page=64, n=4160, window=4096,
             sinks=4, T=1, mix="even", fox=False, dtype="bf16"),
        # long caches that keep all their pages, seen through a window, with gates
        dict(w, name="window gates", B=16, Hq=32, Hkv=8, d=128, page=64, n=16384, window=2048,
             sinks=16, T=1, mix="even", fox=True, dtype="bf16"),
        # a prompt's chunk behind a long one
        dict(w, name="window chunk", B=2, Hq=32, Hkv=8, d=128, page=128, n=16384, window=4096,
             sinks=4, T=1024, mix="ragged", fox=False, dtype="bf16"),
        # a few streams whose window has just left a page
        dict(t, name="trim few", S=6, page=16, n=300, window=256, sinks=4, Hkv=2, d=64),
        # many prompts that have just been read
        dict(t, name="trim prompts", S=256, page=16, n=32768, window=4096, sinks=16, Hkv=1, d=64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["prefix", "prefix", "prefix", "window", "window", "window", "trim"])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    if kind == "trim":
        n = _log_int(rng, 40, 32768)
        return dict(op=kind, S=_log_int(rng, 1, 256), page=rng.choice([16, 32, 64]), n=n,
                    window=_log_int(rng, 1, 2 * n), sinks=rng.choice([0, 1, 4, 16, 100]), Hkv=1, d=64)
    hkv = rng.choice([1, 2, 4, 8, 16])
    hq = hkv * rng.choice([1, 1, 2, 4, 8] if hkv <= 4 else [1, 2, 4] if hkv == 8 else [1, 2])
    dtype = "fp32" if rng.random() < 0.2 else "bf16"
    base = dict(op=kind, Hq=hq, Hkv=hkv, d=d, page=page, fox=rng.random() < 0.5, dtype=dtype)
    full = dtype == "fp32"
    mix = rng.choice(["one", "ragged", "ragged", "even"])
    T = 1 if mix == "one" else _log_int(rng, 2, 150 if full else 600)
    mix = "even" if mix == "one" else mix
    n = _log_int(rng, 1, 2000 if full else 20000)
    if kind == "prefix":
        tail = 0 if rng.random() < 0.2 else _log_int(rng, 1, 600)
        P = rng.choice([1, 1, 2, 4])
        # members: bounded by the logits of the step, by the tails and by the carries
        most = min(48, 1.0e9 / (P * hq * T * (n + tail + T)), 5.0e7 / (P * (tail + T) * hkv * d),
                   6.0e7 / (P * hkv * d * d), 2.0e7 / (P * T * hq * d))
        if full:
            most = min(most, 1.0e8 / (P * hq * T * (n + tail + T)))
        if n * P * hkv * d > 1.2e8:
            P = 1
        return dict(base, P=P, M=_log_int(rng, 1, max(1, int(most))), n=n, tail=tail, T=T, mix=mix)
    window = max(T, _log_int(rng, 1, 1.5 * n + 1))
    most = min(48, 1.0e8 / ((n + T) * hkv * d), 1.0e9 / (hq * T * (n + T)))
    if full:
        most = min(most, 1.0e8 / (hq * T * (n + T)))
    return dict(base, B=_log_int(rng, 1, max(1, int(most))), n=n, T=T, mix=mix, window=window,
                sinks=rng.choice([0, 1, 4, 16, 100]))


def _ragged(r, most, count):
    """`count` lengths of at most `most`, the first as long as that."""
    x = [most - r.randint(0, most // 2) for _ in range(count)]
    x[0] = most
    return x


def _chunks(case, r, count):
    T = case["T"]
    if case["mix"] == "even":
        return [T] * count
    return [T] + [r.randint((T + 3) // 4, T) for _ in range(count - 1)]


def _lengths(case):
    """(cached lengths, new tokens, prefix of each row) of a case: the same for every seed. Of a
    prefix case the rows stand in any order, as a program hands them out."""
    r = random.Random("%(op)s %(n)d" % case)
    if case["op"] == "window":
        return _ragged(r, case["n"], case["B"]), _chunks(case, r, case["B"]), None
    if case["op"] == "trim":
        return _ragged(r, case["n"], case["S"]), None, None
    P, M = case["P"], case["M"]
    n = _ragged(r, case["n"], P) + _ragged(r, case["tail"], P * M)
    T = [0] * P + _chunks(case, r, P * M)
    of = [-1] * P + [i // M for i in range(P * M)]
    order = list(range(P * (M + 1)))
    r.shuffle(order)                                   # row i is what was order[i]
    at = {x: i for i, x in enumerate(order)}
    return ([n[x] for x in order], [T[x] for x in order],
            [-1 if of[x] < 0 else at[of[x]] for x in order])


def _pages(tokens, page):
    return -(-tokens // page)


def _gone(n, case):
    """(first slot, slots) of the pages that no window reaches."""
    first = _pages(case["sinks"], case["page"])
    return first, max(0, max(0, n + 1 - case["window"]) // case["page"] - first)


def work(case):
    if case["op"] == "trim":
        n, _, _ = _lengths(case)
        moved = gone = 0
        for x in n:
            first, k = _gone(x, case)
            gone += k
            moved += max(0, _pages(x, case["page"]) - first - k) if k else 0
        # two tables: entries read and moved; counts read and written; lengths
        return {"bytes": 2 * (8 * moved + 12 * gone) + 8 * case["S"], "flops": 0}
    e = 4 if case["dtype"] == "fp32" else 2
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    row = Hkv * d * e
    gate = 4 * Hq if case["fox"] else 0
    byts = flops = 0
    n, T, of = _lengths(case)
    for b in range(len(n)):
        if T[b] == 0:
            continue
        see = n[b]
        if case["op"] == "window":
            lo = max(0, n[b] + 1 - case["window"])
            see = n[b] - lo + min(lo, case["sinks"])
        byts += see * (3 * row + 2 * gate)               # keys in and out, values in, gates
        byts += T[b] * (5 * row + 2 * Hq * d * e + 4 * Hkv + 2 * gate)
        pairs = T[b] * n[b]
        if case["op"] == "window":
            pairs = sum(min(n[b], case["window"] - 1 - t) +
                        max(0, min(case["sinks"], n[b] + t + 1 - case["window"]))
                        if n[b] + t + 1 > case["window"] else n[b] for t in range(T[b]))
        else:
            pairs += T[b] * n[of[b]]
            byts += 8 * Hkv * d * d + (2 * gate)         # the carry in and out
            flops += 2 * Hkv * d * d * min(2 * T[b], d) + 2 * T[b] * Hq * d * d
        flops += 4 * Hq * d * (pairs + T[b] * (T[b] + 1) // 2)
        flops += 2 * Hkv * d * see * min(2 * T[b], d)    # the keys' transitions
        flops += 6 * Hkv * d * T[b] * min(T[b], 64)      # the block factors
    if case["op"] == "prefix":
        for p in {x for x in of if x >= 0}:
            byts += n[p] * (2 * row + gate)              # once for all that continue it
    return {"bytes": byts, "flops": flops}


# ---------------------------------------------------------------- inputs

def _gate_sums(g, n, H):
    """Gate sums (H, n) that log f = logsigmoid(N(2, 1)) leaves behind: entry j sums the gates
    of the tokens after j."""
    lf = torch.nn.functional.logsigmoid(torch.randn((H, n), generator=g, device="cuda") + 2.0)
    tail = lf.double().flip(-1).cumsum(-1).flip(-1)
    return torch.cat([tail[:, 1:], tail.new_zeros((H, min(n, 1)))], -1).float()


def _prepare_step(case, g):
    Hq, Hkv, d, page = (case[x] for x in ("Hq", "Hkv", "d", "page"))
    dt = _DT[case["dtype"]]
    n, T, of = _lengths(case)
    S = len(n)
    need = [_pages(a + b, page) for a, b in zip(n, T)]
    total = sum(need) + 3
    shape = (total, Hkv, page, d)
    s = {x + "_pages": torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g) for x in "kv"}
    width = max(need) + 1
    # pages in the order in which a pool that has been in use for a while hands them out: any
    for x in "kv":
        ids = torch.randperm(total, generator=g, device="cuda").int()
        t = torch.full((S, width), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b in range(S):
            t[b, :need[b]] = ids[at:at + need[b]]
            at += need[b]
        s[x + "_table"] = t
    N = sum(T)
    s["q"] = torch.randn((N, Hq, d), generator=g, device="cuda").to(dt)
    for x in ("k", "v"):
        s[x] = torch.randn((N, Hkv, d), generator=g, device="cuda").to(dt)
    w = torch.randn((N, Hkv, d), generator=g, device="cuda")
    s["w"] = (w / w.norm(dim=-1, keepdim=True)).to(dt)
    s["beta"] = (2 * torch.randn((N, Hkv), generator=g, device="cuda").sigmoid()).clamp(max=1.99)
    s.update(g_pages=None, log_f=None, lens=torch.tensor(n, dtype=torch.int32, device="cuda"),
             cu=torch.tensor([sum(T[:b]) for b in range(S + 1)], dtype=torch.int32, device="cuda"),
             n_max=max(n), t_max=max(T), case=case)
    if case["fox"]:
        s["log_f"] = torch.nn.functional.logsigmoid(
            torch.randn((N, Hq), generator=g, device="cuda") + 2.0)
        s["g_pages"] = torch.zeros((total, Hq, page), device="cuda")
        for b in range(S):
            m = _pages(n[b], page)
            if m:
                row = torch.zeros((Hq, m * page), device="cuda")
                row[:, :n[b]] = _gate_sums(g, n[b], Hq)
                s["g_pages"][s["k_table"][b, :m].long()] = row.view(Hq, m, page).transpose(0, 1)
    if case["op"] == "prefix":
        # the carries that the tails have left behind: products of their transitions (a few of
        # them, reflections and shrinkings of random directions, stand for all)
        C = torch.eye(d, device="cuda").expand(S, Hkv, d, d).contiguous()
        for _ in range(12):
            u = torch.randn((S, Hkv, d), generator=g, device="cuda")
            u = u / u.norm(dim=-1, keepdim=True)
            b = 2 * torch.randn((S, Hkv), generator=g, device="cuda").sigmoid()
            C = C - b[..., None, None] * (C @ u[..., None]) * u[..., None, :]
        s["carry"] = C.contiguous()
        s["gate_carry"] = None
        if case["fox"]:
            tails = s["lens"].float()[:, None] * torch.rand((S, Hq), generator=g, device="cuda")
            s["gate_carry"] = -0.17 * tails
        s["prefix_of"] = torch.tensor(of, dtype=torch.int32, device="cuda")
        s["p_max"] = max(n[p] for p in of if p >= 0)
        s["tail_max"] = max(x for x, p in zip(n, of) if p >= 0)
    return s


def _prepare_trim(case, g):
    S, page = case["S"], case["page"]
    n, _, _ = _lengths(case)
    need = [_pages(x, page) for x in n]
    total = sum(need) + 5
    width = max(need) + 2
    shape = (total, case["Hkv"], page, case["d"])
    s = {x + "_pages": torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for x in "kv"}
    r = torch.Generator().manual_seed(int(torch.randint(1 << 30, (1,), generator=g, device="cuda")))
    slots = torch.arange(width)
    used = slots < torch.tensor(need)[:, None]
    for x in "kv":
        t = torch.full((S, width), -1, dtype=torch.int32)
        t[used] = torch.randperm(total, generator=r).int()[:sum(need)]
        ref = torch.zeros(total, dtype=torch.int32)
        ref[t[used].long()] = 1
        if x == "v":
            # some value pages are shared with sequences that were forked off
            ref += (torch.rand(total, generator=r) < 0.2).int() * (ref > 0)
        s[x + "_table"], s[x + "_ref"] = t.cuda(), ref.cuda()
    s.update(lens=torch.tensor(n, dtype=torch.int32, device="cuda"), g_pages=None, case=case)
    s["before"] = {x: s[x].clone() for x in _TABLES}
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    return _prepare_trim(case, g) if case["op"] == "trim" else _prepare_step(case, g)


# ---------------------------------------------------------------- plain forms

def _gather(pages, table, n_max, page):
    """(B, H, n_max[, d]) fp32 of the first n_max positions of every given row."""
    m = _pages(n_max, page)
    x = pages[table[:, :m].clamp(min=0).long()]                   # B, m, H, page[, d]
    x = x.transpose(1, 2).flatten(2, 3)
    return x[:, :, :n_max].float()


def _places(table, start, count, page, most):
    """(page ids, offsets, mask) of positions start .. start + count - 1 of every row."""
    t = torch.arange(most, device="cuda")
    pos = start[:, None] + t
    mask = t < count[:, None]
    slot = (pos // page).clamp(max=table.shape[1] - 1)
    return table.gather(1, slot.long()).long(), pos % page, mask


def _put(pages, where, values):
    """values (B, H, most[, d]) into their pages."""
    ids, off, mask = where
    pages[ids[mask], :, off[mask]] = values.transpose(1, 2)[mask].to(pages.dtype)


def _plain_step(s):
    """A step of the rows that bring tokens, in the order of their prefixes."""
    case, page = s["case"], s["case"]["page"]
    prefix = case["op"] == "prefix"
    cu, t_max = s["cu"].long(), s["t_max"]
    if prefix:
        P, M = case["P"], case["M"]
        rows = s["prefix_of"].argsort(stable=True)[P:]            # P groups of M rows
        k_table, v_table = s["k_table"][rows], s["v_table"][rows]
        n, n_max = s["lens"][rows].long(), s["tail_max"]
        start, T = cu[rows], cu[rows + 1] - cu[rows]
    else:
        k_table, v_table = s["k_table"], s["v_table"]
        n, n_max = s["lens"].long(), s["n_max"]
        start, T = cu[:-1], cu[1:] - cu[:-1]
    q, k, v, w = (s[x].float() for x in ("q", "k", "v", "w"))
    N, Hq, d = q.shape
    G = Hq // k.shape[1]
    t = torch.arange(t_max, device="cuda")
    real = t < T[:, None]                                         # B, t_max
    at = (start[:, None] + t).clamp(max=N - 1)
    pad = lambda x: (x[at] * real[:, :, None, None]).transpose(1, 2)  # noqa: E731
    qp, kp, vp, wp = pad(q), pad(k), pad(v), pad(w)               # B, H, t_max, d
    beta = (s["beta"][at] * real[:, :, None]).transpose(1, 2)
    heads = lambda x: x.repeat_interleave(G, 1)  # noqa: E731
    scale = d ** -0.5
    # A = (I + D strictly-lower(W W^T))^-1 D over the whole chunk, u = A w
    E = (wp @ wp.transpose(-1, -2)).tril(-1) * beta[..., None]
    E = E + torch.eye(t_max, device="cuda")
    A = torch.linalg.solve_triangular(E, torch.diag_embed(beta), upper=False, unitriangular=True)
    U = A @ wp
    LA = (qp @ heads(wp).transpose(-1, -2)).tril() @ heads(A)     # s <= i
    R = (kp @ wp.transpose(-1, -2)).triu(1)                       # t > j
    qt = qp - LA @ heads(wp)
    Snew = (qp @ heads(kp).transpose(-1, -2) - LA @ heads(R).transpose(-1, -2)) * scale
    Snew = Snew.masked_fill(t[None, :] > t[:, None], -math.inf)
    K, V = _gather(s["k_pages"], k_table, n_max, page), _gather(s["v_pages"], v_table, n_max, page)
    Sold = (qt @ heads(K).transpose(-1, -2)) * scale
    j = torch.arange(n_max, device="cuda")
    see = (j < n[:, None])[:, None].expand(-1, t_max, -1)         # B, t_max, n_max
    if not prefix:
        see = see & ((j > n[:, None, None] + t[:, None] - case["window"]) | (j < case["sinks"]))
    if s["log_f"] is not None:
        c = (s["log_f"][at] * real[:, :, None]).transpose(1, 2).double().cumsum(-1)
        G_old = _gather(s["g_pages"], k_table, n_max, page)
        Sold = Sold + (G_old.double()[:, :, None] + c[..., None]).float()
        Snew = Snew + (c[..., None] - c[:, :, None]).float()
    Sold = Sold.masked_fill_(~see[:, None], -math.inf)
    V = V.masked_fill((j >= n[:, None])[:, None, :, None], 0)
    m = Snew.amax(-1, keepdim=True)
    if n_max:
        m = torch.maximum(m, Sold.amax(-1, keepdim=True))
    if prefix:
        # the rows of a group against its prefix, which is gathered once
        heads_of = s["prefix_of"][rows].view(P, M)[:, 0].long()
        pn, p_max = s["lens"][heads_of].long(), s["p_max"]
        C = s["carry"][rows]
        qc = qt @ heads(C).transpose(-1, -2)                      # B, Hq, t_max, d
        x = qc.view(P, M, Hq // G, G, t_max, d).transpose(1, 2).reshape(P, Hq // G, -1, d)
        Kp = _gather(s["k_pages"], s["k_table"][heads_of], p_max, page)
        Sp = (x @ Kp.transpose(-1, -2)).mul_(scale).view(P, Hq // G, M, G, t_max, p_max)
        if s["log_f"] is not None:
            Gp = _gather(s["g_pages"], s["k_table"][heads_of], p_max, page)
            own_gates = (s["gate_carry"][rows].double()[..., None] + c).view(P, M, Hq // G, G, t_max)
            Sp += (Gp.view(P, Hq // G, 1, G, 1, p_max).double() +
                   own_gates.transpose(1, 2)[..., None]).float()
        dead = torch.arange(p_max, device="cuda") >= pn[:, None]
        Sp = Sp.masked_fill_(dead[:, None, None, None, None], -math.inf)
        back = lambda y: y.transpose(1, 2).reshape(P * M, Hq, t_max, -1)  # noqa: E731
        m = torch.maximum(m, back(Sp.amax(-1, keepdim=True)))
        Sp = (Sp - m.view(P, M, Hq // G, G, t_max, 1).transpose(1, 2)).exp_()
    Pold, Pnew = Sold.sub_(m).exp_(), Snew.sub_(m).exp_()
    o = Pold @ heads(V) + Pnew @ heads(vp)
    total = Pold.sum(-1, keepdim=True) + Pnew.sum(-1, keepdim=True)
    if prefix:
        Vp = _gather(s["v_pages"], s["v_table"][heads_of], p_max, page)
        Vp = Vp.masked_fill(dead[:, None, :, None], 0)
        total = total + back(Sp.sum(-1, keepdim=True))
        o = o + back((Sp.flatten(2, 4) @ Vp).view(P, Hq // G, M, G, t_max, d))
        s["carry"][rows] = C - (C @ U.transpose(-1, -2)) @ wp
        if s["log_f"] is not None:
            s["gate_carry"][rows] = (s["gate_carry"][rows].double() + c[..., -1]).float()
    o = (o / total).transpose(1, 2)[real].to(s["q"].dtype)
    out = torch.empty_like(s["q"])
    out[at[real]] = o
    # the cache after the step
    K2 = K - (K @ U.transpose(-1, -2)) @ wp
    k2 = kp - (R @ A.transpose(-1, -2)) @ wp
    ids, off, mask = _places(k_table, torch.zeros_like(n), n, page, n_max)
    old = ids, off, mask & see[:, 0]                              # what the first new token sees
    new = _places(k_table, n, T, page, t_max)
    _put(s["k_pages"], old, K2)
    _put(s["k_pages"], new, k2)
    _put(s["v_pages"], _places(v_table, n, T, page, t_max), vp)
    if s["log_f"] is not None:
        end = c[..., -1:]
        _put(s["g_pages"], old, G_old.double() + end)
        _put(s["g_pages"], new, end - c)
    return out


def _plain_trim(s):
    case, page = s["case"], s["case"]["page"]
    first = _pages(case["sinks"], page)
    gone = (((s["lens"] + 1 - case["window"]).clamp(min=0) // page) - first).clamp(min=0)
    slots = torch.arange(s["k_table"].shape[1], device="cuda")
    dead = (slots >= first) & (slots < first + gone[:, None])
    src = slots + gone[:, None] * (slots >= first)
    _free_slots(s["k_table"], s["k_ref"], dead, src)
    _free_slots(s["v_table"], s["v_ref"], dead, src)
    s["lens"] -= (gone * page).int()


def _free_slots(table, ref, dead, src):
    ids = table[dead].long()
    ref.index_add_(0, ids, torch.full_like(ids, -1, dtype=torch.int32))
    inside = src < table.shape[1]
    moved = table.gather(1, src.clamp(max=table.shape[1] - 1))
    table.copy_(torch.where(inside, moved, -1))


# ---------------------------------------------------------------- one pass

_TABLES = ("k_table", "v_table", "k_ref", "v_ref", "lens")
_STATE = ("k_pages", "v_pages", "g_pages") + _TABLES


def _own_step(s):
    import dependent_position_encoded_gb300 as pa
    case, fox = s["case"], s["log_f"] is not None
    cache = pa.PathPagedCache(**{x: s.get(x) for x in _STATE})
    prefix = case["op"] == "prefix"
    if "ws" not in s:  # a serving loop keeps its workspace
        s["ws"] = pa.new_paged_workspace(cache, s["q"].shape[0], s["t_max"], Hq=s["q"].shape[1],
                                         prefix=prefix)
    args = [s["q"], s["k"], s["v"], s["w"], s["beta"]] + ([s["log_f"]] if fox else [])
    args += [s["cu"], cache]
    if prefix:
        call = pa.path_fox_paged_prefix_extend if fox else pa.path_paged_prefix_extend
        more = (s["prefix_of"], s["carry"]) + ((s["gate_carry"],) if fox else ())
        return call(*args, *more, s["t_max"], workspace=s["ws"])
    call = pa.path_fox_paged_window_extend if fox else pa.path_paged_window_extend
    return call(*args, s["t_max"], case["window"], case["sinks"], workspace=s["ws"])


def _own_trim(s):
    import dependent_position_encoded_gb300 as pa
    cache = pa.PathPagedCache(**{x: s.get(x) for x in _STATE})
    if "ws" not in s:
        s["ws"] = pa.new_paged_workspace(cache)
    pa.path_paged_trim(cache, s["case"]["window"], s["case"]["sinks"], workspace=s["ws"])


def run(s):
    if s["case"]["op"] == "trim":
        # a pass begins from the tables as they were
        for x, y in s["before"].items():
            s[x].copy_(y)
        if own:
            _own_trim(s)
        else:
            _plain_trim(s)
        return {x: s[x] for x in _TABLES}
    out = _own_step(s) if own else _plain_step(s)
    names = ("k_pages", "v_pages", "g_pages", "carry", "gate_carry")
    return dict({x: s[x] for x in names if s.get(x) is not None}, out=out)


# ---------------------------------------------------------------- from the definition, 64 bits

def exact(case, seed):
    """One token after the other: every key in sight takes the token's transition, then the token
    joins and asks; a prefix's keys are asked with C q, C the product of the transitions since."""
    if case["op"] == "trim":
        return None  # pages are counted, not computed
    s = prepare(case, seed)
    n, T, of = _lengths(case)
    N, Hq, d = s["q"].shape
    Hkv, page = case["Hkv"], case["page"]
    G = Hq // Hkv
    f = torch.float64
    out = torch.zeros((N, Hq, d), dtype=f, device="cuda")
    kpg, vpg = s["k_pages"].to(f), s["v_pages"].to(f)
    gpg = None if s["g_pages"] is None else s["g_pages"].to(f)
    carry = s["carry"].to(f) if of else None
    gcarry = s["gate_carry"].to(f) if of and gpg is not None else None

    def lines(pages, table, b, m):
        x = pages[table[b, :m].long()].transpose(0, 1)
        return x.reshape((x.shape[0], m * page) + tuple(x.shape[3:]))

    first = 0
    for b in range(len(n)):
        if T[b] == 0:
            continue
        total = n[b] + T[b]
        m = _pages(total, page)
        K, V = lines(kpg, s["k_table"], b, m), lines(vpg, s["v_table"], b, m)
        g = None if gpg is None else lines(gpg, s["k_table"], b, m)
        low = max(0, n[b] + 1 - case["window"]) if of is None else 0  # what moves: sinks, then from here
        ends = min(case["sinks"], low) if of is None else 0
        queries, scores = [], []
        for t in range(T[b]):
            i, e = first + t, n[b] + t
            w, beta = s["w"][i].to(f), s["beta"][i].to(f)
            for part in ((0, ends), (low, e)) if ends else ((low, e),):
                x = K[:, part[0]:part[1]]
                x -= (torch.einsum("hjd,hd->hj", x, w) * beta[:, None])[..., None] * w[:, None]
                if g is not None:
                    g[:, part[0]:part[1]] += s["log_f"][i].to(f)[:, None]
            K[:, e], V[:, e] = s["k"][i].to(f), s["v"][i].to(f)
            if g is not None:
                g[:, e] = 0
            q = s["q"][i].to(f).view(Hkv, G, d)
            x = torch.einsum("hgd,hjd->hgj", q, K[:, :e + 1]).reshape(Hq, e + 1) / math.sqrt(d)
            if g is not None:
                x = x + g[:, :e + 1]
            if of is None:
                hidden = slice(case["sinks"], max(case["sinks"], e + 1 - case["window"]))
                x[:, hidden] = -math.inf
                p = torch.softmax(x, -1).view(Hkv, G, e + 1)
                out[i] = torch.einsum("hgj,hjd->hgd", p, V[:, :e + 1]).reshape(Hq, d)
                continue
            # the same with the prefix: its keys see the query through the carry
            C = carry[b]
            C -= beta[:, None, None] * torch.einsum("hid,hd->hi", C, w)[..., None] * w[:, None]
            queries.append(torch.einsum("hid,hgd->hgi", C, q))
            if gcarry is not None:
                gcarry[b] += s["log_f"][i].to(f)
            lse = torch.logsumexp(x, -1)
            o = torch.einsum("hgj,hjd->hgd", torch.softmax(x, -1).view(Hkv, G, e + 1), V[:, :e + 1])
            scores.append((lse, o.reshape(Hq, d), None if gcarry is None else gcarry[b].clone()))
        if of is not None:
            p = of[b]
            pm = _pages(n[p], page)
            Kp, Vp = (lines(a, tb, p, pm)[:, :n[p]] for a, tb in ((kpg, s["k_table"]), (vpg, s["v_table"])))
            x = torch.einsum("thgi,hji->thgj", torch.stack(queries), Kp).reshape(T[b], Hq, n[p]) / math.sqrt(d)
            if gcarry is not None:
                x += lines(gpg, s["k_table"], p, pm)[:, :n[p]] + torch.stack([z[2] for z in scores])[..., None]
            lse, o = torch.stack([z[0] for z in scores]), torch.stack([z[1] for z in scores])
            both = torch.logaddexp(lse, torch.logsumexp(x, -1))
            x = (x - both[..., None]).exp_().view(T[b], Hkv, G, n[p])
            out[first:first + T[b]] = (o * (lse - both).exp()[..., None] +
                                       torch.einsum("thgj,hjd->thgd", x, Vp).reshape(T[b], Hq, d))

        def back(pages, table, X):
            new = X.reshape((X.shape[0], m, page) + tuple(X.shape[2:])).transpose(0, 1)
            pages[table[b, :m].long()] = new

        back(kpg, s["k_table"], K)
        back(vpg, s["v_table"], V)
        if g is not None:
            back(gpg, s["k_table"], g)
        first += T[b]
    r = {"k_pages": kpg, "v_pages": vpg, "out": out}
    for name, x in (("g_pages", gpg), ("carry", carry), ("gate_carry", gcarry)):
        if x is not None:
            r[name] = x
    return r
