"""A plain fp64 reference of a window step over a paged cache, written from the definition, and what
a trimmed sequence's table must be."""
import torch

from tests.paged_cases import close, pages, rows_of, snapshot

NAN = float("nan")


def advanced(n, window, sinks, device):
    """The cached positions that the first new token sees."""
    j = torch.arange(n, device=device)
    return (j > n - window) | (j < sinks)


def hide(x, window, sinks):
    """NaN in every cached position that no new token sees; pages that hold only such ones are
    unmapped."""
    for s, (n, T) in enumerate(zip(x["n"], x["chunks"])):
        if T == 0:
            continue
        dead = (~advanced(n, window, sinks, x["q"].device)).nonzero()[:, 0]
        for name in ("k_pages", "v_pages", "g_pages"):
            if x[name] is not None:
                table = x["v_table" if name == "v_pages" else "k_table"][s]
                x[name][table[dead // x["page"]].long(), :, dead % x["page"]] = NAN
        for slot in range(pages(n, x["page"])):
            lo, hi = slot * x["page"], (slot + 1) * x["page"]
            if hi <= n + 1 - window and lo >= sinks:
                x["k_table"][s, slot] = x["v_table"][s, slot] = -1


def window_reference(x, window, sinks, scale=None):
    """(out, [K rows], [V rows], [gate rows]) in fp64, as paged_cases.reference."""
    scale = x["d"] ** -0.5 if scale is None else scale
    out = torch.zeros(x["q"].shape, dtype=torch.float64, device=x["q"].device)
    G = x["Hq"] // x["Hkv"]
    Ks, Vs, Gs, first = [], [], [], 0
    for s, (n, T) in enumerate(zip(x["n"], x["chunks"])):
        K, V = (rows_of(x[a + "_pages"], x[a + "_table"][s], n).transpose(0, 1) for a in "kv")
        g = rows_of(x["g_pages"], x["k_table"][s], n).transpose(0, 1) if x["log_f"] is not None else None
        moves = advanced(n, window, sinks, K.device)
        for i in range(first, first + T):
            w, b = x["w"][i].double(), x["beta"][i].double()
            K2 = K - b[:, None, None] * torch.einsum("hjd,hd->hj", K, w)[..., None] * w[:, None]
            K = torch.cat([torch.where(moves[:, None], K2, K), x["k"][i].double()[:, None]], 1)
            V = torch.cat([V, x["v"][i].double()[:, None]], 1)
            if g is not None:
                g = torch.where(moves, g + x["log_f"][i].double()[:, None], g)
                g = torch.cat([g, g.new_zeros((x["Hq"], 1))], 1)
            moves = torch.cat([moves, moves.new_ones(1)])
            here = K.shape[1] - 1
            j = torch.arange(here + 1, device=K.device)
            sees = ((j > here - window) | (j < sinks)).nonzero()[:, 0]
            z = torch.einsum("hgd,hjd->hgj", x["q"][i].double().view(x["Hkv"], G, -1), K[:, sees]) * scale
            if g is not None:
                z = z + g[:, sees].view(x["Hkv"], G, -1)
            out[i] = torch.einsum("hgj,hjd->hgd", z.softmax(-1), V[:, sees]).reshape(x["Hq"], -1)
        first += T
        Ks.append(K.transpose(0, 1))
        Vs.append(V.transpose(0, 1))
        Gs.append(g.transpose(0, 1) if g is not None else None)
    return out, Ks, Vs, Gs


def window_step(lib, x, cache, window, sinks, **kw):
    most = max(max(x["chunks"]), 1)
    if x["log_f"] is not None:
        return lib.path_fox_paged_window_extend(x["q"], x["k"], x["v"], x["w"], x["beta"], x["log_f"],
                                                x["cu"], cache, most, window, sinks, **kw)
    return lib.path_paged_window_extend(x["q"], x["k"], x["v"], x["w"], x["beta"], x["cu"], cache,
                                        most, window, sinks, **kw)


def same_bits(a, b):
    it = torch.int16 if a.dtype == torch.bfloat16 else torch.int32
    return torch.equal(a.contiguous().view(it), b.contiguous().view(it))


def check_window(x, before, out, window, sinks, ref=None):
    """Outputs and the whole cache; what the step does not own is as it was, bit for bit."""
    dev = x["q"].device
    ref, Ks, Vs, Gs = window_reference(dict(x, **before), window, sinks) if ref is None else ref
    N = sum(x["chunks"])
    close(out[:N], ref[:N], x["q"].dtype, "out")
    for name in ("k_pages", "v_pages", "g_pages"):
        if x[name] is None:
            continue
        table = x["v_table"] if name == "v_pages" else x["k_table"]
        mine = torch.zeros(x[name].shape[0], x["page"], dtype=torch.bool, device=dev)
        for s, (n, T) in enumerate(zip(x["n"], x["chunks"])):
            if T == 0:
                continue
            if name == "v_pages":
                p = torch.arange(n, n + T, device=dev)
                got, want = _at(x[name], table[s], p), Vs[s][n:]
                assert torch.equal(got, want)
            else:
                moves = advanced(n, window, sinks, dev)
                p = torch.cat([moves.nonzero()[:, 0], torch.arange(n, n + T, device=dev)])
                got, want = _at(x[name], table[s], p), (Ks if name == "k_pages" else Gs)[s][p]
                if name == "k_pages":
                    close(got, want, x["q"].dtype, "keys")
                else:
                    # sums of n + T gates kept in fp32 relative to the last token
                    err = (got - want).abs() - want.abs() * 2.0 ** -22
                    assert float(err.max()) <= 1e-6
            mine[table[s][p // x["page"]].long(), p % x["page"]] = True
        keep = ~mine[:, None].expand(x[name].shape[:3])
        assert same_bits(x[name][keep], before[name][keep]), name


def _at(pool, table, p):
    page = pool.shape[2]
    return pool[table[p // page].long(), :, p % page].double()


def trimmed(table, lens, window, sinks, page):
    """(tables after trimming, lengths, entries that left, in lists) of host lists."""
    rows, out_lens, left = [], [], []
    for row, n in zip(table, lens):
        lo, keep, gone = n + 1 - window, [], []
        for slot, e in enumerate(row):
            dead = slot * page >= sinks and (slot + 1) * page <= lo
            (gone if dead else keep).append(e)
        rows.append(keep + [-1] * len(gone))
        out_lens.append(n - len(gone) * page)
        left += [e for e in gone if e >= 0]
    return rows, out_lens, left


__all__ = ["NAN", "advanced", "hide", "window_reference", "window_step", "same_bits", "check_window",
           "trimmed", "snapshot"]
