"""Inputs of steps behind shared prefixes and a plain fp64 reference, written from the definition (one
token at a time, one sequence at a time)."""
import torch

from tests import paged_cases as pc


def make(lens, chunks, of, Hq, Hkv, d, page, dtype, fox, seed=0, device="cuda", **kw):
    """paged_cases.make with prefix_of, a carry (a product of 20 random transitions) and gate sums."""
    x = pc.make(lens, chunks, Hq, Hkv, d, page, dtype, fox, seed=seed, device=device, **kw)
    g = torch.Generator(device=device).manual_seed(seed + 1000)
    S = len(lens)
    x["of"] = list(of)
    x["prefix_of"] = torch.tensor(of, dtype=torch.int32, device=device)
    C = torch.eye(d, device=device, dtype=torch.float64).repeat(S, Hkv, 1, 1)
    for _ in range(20):
        w = torch.randn((S, Hkv, d), generator=g, device=device).double()
        w = w / w.norm(dim=-1, keepdim=True)
        b = 2 * torch.randn((S, Hkv), generator=g, device=device).double().sigmoid()
        C = C - b[..., None, None] * torch.einsum("shij,shj->shi", C, w)[..., None] * w[..., None, :]
    x["carry"] = C.float().contiguous()
    x["gate_carry"] = -torch.rand((S, Hq), generator=g, device=device) * 2 if fox else None
    return x


def snapshot(x):
    return dict(pc.snapshot(x), carry=x["carry"].clone(),
                gate_carry=None if x["gate_carry"] is None else x["gate_carry"].clone())


def step(lib, x, cache=None, **kw):
    cache = pc.cache_of(lib, x) if cache is None else cache
    most = max(max(x["chunks"]), 1)
    args = (x["q"], x["k"], x["v"], x["w"], x["beta"])
    if x["log_f"] is not None:
        return lib.path_fox_paged_prefix_extend(*args, x["log_f"], x["cu"], cache, x["prefix_of"], x["carry"],
                                                x["gate_carry"], most, **kw)
    return lib.path_paged_prefix_extend(*args, x["cu"], cache, x["prefix_of"], x["carry"], most, **kw)


def reference(x):
    """(out, [K], [V], [gates], carry, gate_carry) in fp64."""
    out, Ks, Vs, Gs = pc.reference(x)  # (the cache's part of it holds for every sequence)
    carry = x["carry"].double().clone()
    gates = None if x["gate_carry"] is None else x["gate_carry"].double().clone()
    G, Hkv, first = x["Hq"] // x["Hkv"], x["Hkv"], 0
    for s, (n, T) in enumerate(zip(x["n"], x["chunks"])):
        p = x["of"][s]
        if T == 0 or p < 0:
            first += T
            continue
        m = x["n"][p]
        Kp, Vp = (pc.rows_of(x[a + "_pages"], x[a + "_table"][p], m).transpose(0, 1) for a in "kv")
        gp = None if gates is None else pc.rows_of(x["g_pages"], x["k_table"][p], m).transpose(0, 1)
        K, V = (pc.rows_of(x[a + "_pages"], x[a + "_table"][s], n).transpose(0, 1) for a in "kv")
        g = None if gates is None else pc.rows_of(x["g_pages"], x["k_table"][s], n).transpose(0, 1)
        for i in range(first, first + T):
            w, b, q = x["w"][i].double(), x["beta"][i].double(), x["q"][i].double().view(Hkv, G, -1)
            K = K - b[:, None, None] * torch.einsum("hjd,hd->hj", K, w)[..., None] * w[:, None]
            K = torch.cat([K, x["k"][i].double()[:, None]], 1)
            V = torch.cat([V, x["v"][i].double()[:, None]], 1)
            carry[s] -= b[:, None, None] * torch.einsum("hij,hj->hi", carry[s], w)[..., None] * w[:, None]
            qc = torch.einsum("hij,hgj->hgi", carry[s], q)
            z = torch.cat([torch.einsum("hgd,hjd->hgj", qc, Kp), torch.einsum("hgd,hjd->hgj", q, K)], -1)
            z = z * x["d"] ** -0.5
            if gates is not None:
                f = x["log_f"][i].double()
                g = torch.cat([g + f[:, None], g.new_zeros((x["Hq"], 1))], 1)
                gates[s] += f
                z = z + torch.cat([gp + gates[s][:, None], g], 1).view(Hkv, G, -1)
            out[i] = torch.einsum("hgj,hjd->hgd", z.softmax(-1), torch.cat([Vp, V], 1)).reshape(x["Hq"], -1)
        first += T
    return out, Ks, Vs, Gs, carry, gates


def check(x, before, out, ref=None):
    """Outputs, carries and the whole cache against the reference. A prefix's row has no tokens, so
    paged_cases.check holds it, as everything that is not the step's, to its bits."""
    y = dict(x, **before)
    ref = reference(y) if ref is None else ref
    N = sum(x["chunks"])
    pc.close(out[:N], ref[0][:N], x["q"].dtype, "out")
    pc.check(x, {n: before[n] for n in ("k_pages", "v_pages", "g_pages")}, _plain(y, out))
    for s, T in enumerate(x["chunks"]):
        if T == 0 or x["of"][s] < 0:
            assert torch.equal(x["carry"][s], before["carry"][s])
            assert x["gate_carry"] is None or torch.equal(x["gate_carry"][s], before["gate_carry"][s])
            continue
        # a chunk of T transitions in fp32: each rounds a sum of d products and its own entries, a few 2^-24
        # of a row's norm, which no transition lets grow; independent, so sqrt(T) of them
        err = (x["carry"][s].double() - ref[4][s]).norm(dim=-1) / before["carry"][s].double().norm(dim=-1).clamp(min=1e-3)
        assert float(err.max()) <= 8 * 2.0 ** -24 * T ** 0.5 + 2.0 ** -22, float(err.max())
        if x["gate_carry"] is not None:
            err = (x["gate_carry"][s].double() - ref[5][s]).abs() - ref[5][s].abs() * 2.0 ** -22
            assert float(err.max()) <= 1e-6


def _plain(y, out):
    """`out` with what its rows have of their own sequence alone in place of the rows behind a prefix, so
    that paged_cases.check, which knows no prefix, holds the cache."""
    own = out.clone()
    ref, first = pc.reference(y)[0], 0
    for T, p in zip(y["chunks"], y["of"]):
        if p >= 0:
            own[first:first + T] = ref[first:first + T].to(out.dtype)
        first += T
    return own
