"""Steps over a paged cache whose forget gates reach the ends of fp32: a gate that closes for good
(a document's border, log f = -1e30 or the type's lowest value) among ordinary ones. The reference
adds one gate at a time and so never loses the gates behind a closing one."""
import pytest
import torch

from tests import paged_cases as pc

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
LOWEST = torch.finfo(torch.float32).min


def check(x, before, out):
    """Outputs and keys as everywhere; gate sums within fp32's range as everywhere (n + T gates
    kept in fp32: 2^-22 of the sum and 1e-6), below it -inf, as the same gates added one by one
    in fp32 give."""
    ref, Ks, _, Gs = pc.reference(dict(x, **before))
    N = sum(x["chunks"])
    pc.close(out[:N], ref[:N], x["q"].dtype, "out")
    for s, (n, T) in enumerate(zip(x["n"], x["chunks"])):
        pc.close(pc.rows_of(x["k_pages"], x["k_table"][s], n + T), Ks[s], x["q"].dtype, "keys")
        got = pc.rows_of(x["g_pages"], x["k_table"][s], n + T)
        below = Gs[s] < LOWEST
        assert (got[below] < LOWEST * 0.999).all()
        err = (got - Gs[s]).abs() - Gs[s].abs() * 2.0 ** -22
        assert float(err[~below].max()) <= 1e-6


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,Hq,Hkv", [(64, 4, 2), (128, 3, 1)])
@pytest.mark.parametrize("gate", [-1e5, -3e7, -1e30, LOWEST])
@pytest.mark.parametrize("chunks,at", [
    ([40, 1], [5]),                 # one in a block
    ([40, 9], [0, 20, 43]),         # a first token, two in a block, another sequence's
    ([64, 2], [31, 32, 63]),        # neighbours, a block's last token
    ([150, 70], [10, 64, 70, 215]),  # several blocks, with and without
])
def test_gates_behind_a_closing_one(lib, dtype, d, Hq, Hkv, gate, chunks, at):
    x = pc.make([90, 33], chunks, Hq, Hkv, d, 16, dtype, True, seed=31)
    x["log_f"][at] = gate
    if len(at) > 1:  # not for every head
        x["log_f"][at[-1], 1:] = -0.25
    before = pc.snapshot(x)
    out = pc.step(lib, x)
    check(x, before, out)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("chunks", [[1, 1], [6, 66]])
def test_a_step_on_closed_keys(lib, dtype, chunks):
    """Keys whose sums have passed fp32's range take further gates and stay without weight."""
    x = pc.make([90, 33], chunks, 4, 2, 64, 16, dtype, True, seed=32)
    for s, n in enumerate([50, 33]):
        pc.put(x["g_pages"], x["k_table"][s], 0, torch.full((n, 4), -float("inf"), device="cuda"))
    x["log_f"][0] = LOWEST
    before = pc.snapshot(x)
    out = pc.step(lib, x)
    check(x, before, out)


def test_one_call_equals_single_steps_across_a_border(lib):
    x = pc.make([20], [60], 2, 2, 64, 16, F32, True, seed=33)
    x["log_f"][[7, 30]] = -1e30
    y = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}
    out = pc.step(lib, x)
    cache = pc.cache_of(lib, y)
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    outs = torch.empty_like(out)
    for t in range(60):
        r = {n: y[n][t:t + 1] for n in ("q", "k", "v", "w", "beta", "log_f")}
        outs[t:t + 1] = lib.path_fox_paged_extend(*r.values(), cu, cache, 1)
        cache.lens += 1
    assert float((out - outs).norm() / out.norm()) < 2e-5
    a, b = (pc.rows_of(z["g_pages"], z["k_table"][0], 80) for z in (x, y))
    # sixty fp32 additions, each off by 2^-24 of the sum
    assert float(((a - b).abs() - a.abs() * 60 * 2.0 ** -24).max()) <= 0
