"""Inputs of the paged-cache tests and a plain fp64 reference of the step, written from the
definition (one token at a time, one sequence at a time)."""
import math

import torch


def pages(tokens, page):
    return -(-tokens // page)


def make(lens, chunks, Hq, Hkv, d, page, dtype, fox, seed=0, head_major=False, spare=3, tail=0,
         width=None, device="cuda"):
    """A cache holding `lens` tokens per sequence, and a step of `chunks` new ones; `tail` token
    rows lie behind the last sequence's. Pages are scattered over the pools, unused rows and
    pages hold NaN. head_major: tensors stored (heads, tokens, d) and viewed as (tokens, heads,
    d)."""
    g = torch.Generator(device=device).manual_seed(seed)
    S = len(lens)
    need = [pages(a + b, page) for a, b in zip(lens, chunks)]
    total = sum(need) + spare
    x = {"page": page, "d": d, "Hq": Hq, "Hkv": Hkv, "chunks": list(chunks), "n": list(lens)}
    nan = float("nan")
    x["k_pages"] = torch.full((total, Hkv, page, d), nan, dtype=dtype, device=device)
    x["v_pages"] = torch.full((total + 2, Hkv, page, d), nan, dtype=dtype, device=device)
    x["g_pages"] = torch.full((total, Hq, page), nan, device=device) if fox else None
    width = max(need + [1]) if width is None else width
    for name, pool in (("k", total), ("v", total + 2)):
        ids = torch.randperm(pool, generator=g, device=device).int()
        t = torch.full((S, width), -1, dtype=torch.int32, device=device)
        ref = torch.zeros(pool, dtype=torch.int32, device=device)
        at = 0
        for s in range(S):
            t[s, :need[s]] = ids[at:at + need[s]]
            at += need[s]
        ref[ids[:at].long()] = 1
        x[name + "_table"], x[name + "_ref"] = t, ref
        for s in range(S):
            rows = torch.randn((lens[s], Hkv, d), generator=g, device=device).to(dtype)
            put(x[name + "_pages"], t[s], 0, rows)
    if fox:
        for s in range(S):
            u = torch.randn((lens[s], Hq), generator=g, device=device) + 2.0
            lf = torch.nn.functional.logsigmoid(u).double()
            sums = lf.flip(0).cumsum(0).flip(0) - lf  # the gates behind each token
            put(x["g_pages"], x["k_table"][s], 0, sums.float())
    x["lens"] = torch.tensor(lens, dtype=torch.int32, device=device)
    cu = [0]
    for c in chunks:
        cu.append(cu[-1] + c)
    x["cu"] = torch.tensor(cu, dtype=torch.int32, device=device)
    N = cu[-1] + tail

    def rand(*shape):
        return torch.randn(shape, generator=g, device=device)

    def lay(t):
        return t.transpose(0, 1).contiguous().transpose(0, 1) if head_major else t

    x["q"] = lay(rand(N, Hq, d).to(dtype))
    x["k"], x["v"] = lay(rand(N, Hkv, d).to(dtype)), lay(rand(N, Hkv, d).to(dtype))
    w = rand(N, Hkv, d)
    x["w"] = lay((w / w.norm(dim=-1, keepdim=True)).to(dtype))
    x["beta"] = lay((2 * rand(N, Hkv).sigmoid()).clamp(max=1.99))
    x["log_f"] = lay(torch.nn.functional.logsigmoid(rand(N, Hq) + 2.0)) if fox else None
    return x


def put(pool, table, start, rows):
    """rows (tokens, H[, d]) at positions start .. of the sequence with this table row."""
    page = pool.shape[2]
    p = torch.arange(start, start + rows.shape[0], device=pool.device)
    pool[table[(p // page).long()].long(), :, p % page] = rows


def rows_of(pool, table, n):
    """(n, H[, d]) fp64 of a sequence's first n positions."""
    page = pool.shape[2]
    m = pages(n, page)
    t = pool[table[:m].long()].double().transpose(1, 2)
    return t.reshape((m * page,) + tuple(t.shape[2:]))[:n]


def reference(x, scale=None, step_dtype=None):
    """(out, [K rows], [V rows], [gate rows]) of the step in fp64; per sequence the rows of all
    its n + T positions. Rows of `out` behind the last sequence are zero."""
    scale = x["d"] ** -0.5 if scale is None else scale
    out = torch.zeros(x["q"].shape, dtype=torch.float64, device=x["q"].device)
    G = x["Hq"] // x["Hkv"]
    Ks, Vs, Gs = [], [], []
    first = 0
    for s, (n, T) in enumerate(zip(x["n"], x["chunks"])):
        K, V = (rows_of(x[a + "_pages"], x[a + "_table"][s], n).transpose(0, 1) for a in "kv")
        g = rows_of(x["g_pages"], x["k_table"][s], n).transpose(0, 1) if x["log_f"] is not None else None
        for i in range(first, first + T):
            w, b = x["w"][i].double(), x["beta"][i].double()
            K = K - b[:, None, None] * torch.einsum("hjd,hd->hj", K, w)[..., None] * w[:, None]
            K = torch.cat([K, x["k"][i].double()[:, None]], 1)
            V = torch.cat([V, x["v"][i].double()[:, None]], 1)
            z = torch.einsum("hgd,hjd->hgj", x["q"][i].double().view(x["Hkv"], G, -1), K) * scale
            if g is not None:
                g = torch.cat([g + x["log_f"][i].double()[:, None], torch.zeros_like(g[:, :1])
                               if g.shape[1] else g.new_zeros((x["Hq"], 1))], 1)
                z = z + g.view(x["Hkv"], G, -1)
            out[i] = torch.einsum("hgj,hjd->hgd", z.softmax(-1), V).reshape(x["Hq"], -1)
        first += T
        Ks.append(K.transpose(0, 1))
        Vs.append(V.transpose(0, 1))
        Gs.append(g.transpose(0, 1) if g is not None else None)
    return out, Ks, Vs, Gs


def cache_of(lib, x):
    return lib.PathPagedCache(**{n: x[n] for n in ("k_pages", "v_pages", "g_pages", "k_table",
                                                   "v_table", "k_ref", "v_ref", "lens")})


def step(lib, x, cache=None, **kw):
    """One call of the entry point on these inputs."""
    cache = cache_of(lib, x) if cache is None else cache
    most = max(max(x["chunks"]), 1)
    if x["log_f"] is not None:
        return lib.path_fox_paged_extend(x["q"], x["k"], x["v"], x["w"], x["beta"], x["log_f"],
                                         x["cu"], cache, most, **kw)
    return lib.path_paged_extend(x["q"], x["k"], x["v"], x["w"], x["beta"], x["cu"], cache, most,
                                 **kw)


def close(got, ref, dtype, what):
    """The error bounds of a step's outputs.

    fp32: 1e-5 of the reference's norm (sums of up to a few thousand terms of unit size lose a
    few 2^-24 each; the framework's own bar is 1e-4).
    bf16 out: four independent roundings of relative size at most 2^-8, uniform in that range
    (root mean square 2^-8 / sqrt 3 = 2.3e-3 at most), enter an output: the carried query (as a
    logit error of that relative size, whose logits are of unit size here), the weights, the
    values' product sums and the output itself; added as independent errors 4.5e-3. The bar is 5e-3
    of the norm, and 2e-2 on every element, the framework's bf16 bar.
    bf16 keys: one rounding, 2^-8 of the value, plus 2^-11 of a unit key entry for the products of
    the transitions, which carry 16 bits."""
    got, ref = got.double(), ref.double()
    assert got.shape == ref.shape
    if not ref.numel():
        return
    assert torch.isfinite(got).all(), what
    err = (got - ref).abs()
    norm = float(err.norm() / ref.norm().clamp(min=1e-30))
    if dtype == torch.float32:
        assert norm <= 1e-5, (what, norm)
    elif what == "keys":
        over = err - ref.abs() * 2.0 ** -8 - 2.0 ** -11
        assert float(over.max()) <= 0, (what, float(over.max()))
    else:
        assert norm <= 5e-3, (what, norm)
        assert float(err.max()) <= 2e-2, (what, float(err.max()))


def check(x, before, out, scale=None):
    """The step's outputs and the whole cache against the reference; `before`: clones of the
    pools as they were. Every row that the step does not own must be as it was, bit for bit."""
    y = dict(x, **before)
    ref, Ks, Vs, Gs = reference(y, scale)
    N = sum(x["chunks"])
    close(out[:N], ref[:N], x["q"].dtype, "out")
    for name in ("k_pages", "v_pages", "g_pages"):
        if x[name] is None:
            continue
        table = x["v_table"] if name == "v_pages" else x["k_table"]
        same = torch.ones(x[name].shape[0], x["page"], dtype=torch.bool, device=x["q"].device)
        for s, (n, T) in enumerate(zip(x["n"], x["chunks"])):
            got = rows_of(x[name], table[s], n + T)
            if name == "v_pages":
                assert torch.equal(got, Vs[s])
            elif T:
                if name == "k_pages":
                    close(got, Ks[s], x["q"].dtype, "keys")
                else:
                    # sums of n + T gates kept in fp32 relative to the last token
                    err = (got - Gs[s]).abs() - Gs[s].abs() * 2.0 ** -22
                    assert float(err.max()) <= 1e-6
            lo = n if name == "v_pages" else (0 if T else n)
            p = torch.arange(lo, n + T, device=same.device)
            same[table[s][p // x["page"]].long(), p % x["page"]] = False
        keep = same[:, None].expand(x[name].shape[:3]) if x[name].dim() == 4 else \
            same[:, None].expand(x[name].shape)
        a, b = x[name][keep], before[name][keep]
        assert torch.equal(a.view(torch.int16 if a.dtype == torch.bfloat16 else torch.int32),
                           b.view(torch.int16 if b.dtype == torch.bfloat16 else torch.int32)), name


def snapshot(x):
    return {n: (x[n].clone() if x[n] is not None else None) for n in ("k_pages", "v_pages", "g_pages")}


def close_scale(x):
    return 1.0 / math.sqrt(x["d"])
