"""What the calls behind a shared prefix refuse, on the CPU: all before any launch."""
import pytest
import torch

import dependent_position_encoded_gb300 as pa
from tests.test_paged_checks import D, FAKE, HKV, HQ, N, S, _c, _cache, _step, no_gpu


def _more(**kw):
    a = dict(prefix_of=torch.full((S,), -1, dtype=torch.int32), carry=torch.zeros(S, HKV, D, D),
             gate_carry=torch.zeros(S, HQ))
    a.update(kw)
    return a.values()


@pytest.mark.parametrize("kw,exc", [
    (dict(prefix_of=None), TypeError),
    (dict(prefix_of=torch.zeros(S, dtype=torch.int64)), TypeError),
    (dict(prefix_of=torch.zeros(S + 1, dtype=torch.int32)), ValueError),
    (dict(prefix_of=torch.zeros(2 * S, dtype=torch.int32)[::2]), ValueError),
    (dict(carry=torch.zeros(S, HKV, D, D, dtype=torch.bfloat16)), TypeError),
    (dict(carry=torch.zeros(S, HQ, D, D)), ValueError),
    (dict(carry=torch.zeros(S, HKV, D, D).transpose(2, 3)), ValueError),
    (dict(gate_carry=None), TypeError),
    (dict(gate_carry=torch.zeros(S, HKV)), ValueError),
])
def test_prefix_errors_raise_before_any_call(kw, exc):
    with pytest.raises(exc):
        pa.path_fox_paged_prefix_extend(*_step().values(), _cache(), *_more(**kw), 2)


@pytest.mark.parametrize("kw,exc", [
    (dict(q=torch.zeros(N, HQ, 64)), TypeError),
    (dict(q=torch.zeros(N, HQ * 64, dtype=torch.bfloat16)), ValueError),
    (dict(q=None), TypeError),
    (dict(log_f=None), TypeError),
    (dict(cu_tokens=torch.zeros(S, dtype=torch.int32)), ValueError),
])
def test_step_errors_raise_before_any_call(kw, exc):
    with pytest.raises(exc):
        pa.path_fox_paged_prefix_extend(*_step(**kw).values(), _cache(), *_more(), 2)


def test_host_tensors_need_a_gpu():
    with pytest.raises(TypeError, match="CUDA"):
        pa.path_fox_paged_prefix_extend(*_step().values(), _cache(), *_more(), 2)
    with pytest.raises(TypeError):
        pa.path_fox_paged_prefix_extend(*_step().values(), None, *_more(), 2)


@pytest.fixture(scope="module")
def so():
    pa.ensure_built()
    return pa._load()


def _prefix(so, cache, fox, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, w=FAKE, beta=FAKE, log_f=FAKE, cu=FAKE, N=N, chunk=2, of=FAKE, carry=FAKE,
             gates=FAKE, scale=0.125, out=FAKE, st=None, ws=FAKE, bytes=1 << 30, stream=None)
    a.update(kw)
    args = [a[n] for n in ("q", "k", "v", "w", "beta")] + ([a["log_f"]] if fox else [])
    more = [a["of"], a["carry"]] + ([a["gates"]] if fox else [])
    fn = so.path_fox_paged_prefix_extend if fox else so.path_paged_prefix_extend
    return fn(cache, *args, a["cu"], a["N"], a["chunk"], *more, a["scale"], a["out"], a["st"], a["ws"], a["bytes"],
              a["stream"])


@no_gpu
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(of=None), pa.ERR_NULL),
    (dict(carry=None), pa.ERR_NULL),
    (dict(of=FAKE + 2), pa.ERR_ALIGN),
    (dict(carry=FAKE + 4), pa.ERR_ALIGN),
    (dict(q=None), pa.ERR_NULL),
    (dict(chunk=0), pa.ERR_SHAPE),
    (dict(scale=float("inf")), pa.ERR_ARG),
    (dict(ws=None), pa.ERR_NULL),
    (dict(bytes=256), pa.ERR_WORKSPACE),
    (dict(N=0, chunk=0, of=None), pa.OK),
])
def test_prefix_arguments(so, fox, kw, code):
    assert _prefix(so, _c(), fox, **kw) == code


@no_gpu
def test_gate_carry(so):
    assert _prefix(so, _c(), True, gates=None) == pa.ERR_NULL
    assert _prefix(so, _c(), True, gates=FAKE + 2) == pa.ERR_ALIGN


@no_gpu
@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("Hq,Hkv,seqs", [(4, 2, 3), (8, 1, 70), (16, 16, 600)])
def test_a_workspace_serves_smaller_steps(so, dtype, Hq, Hkv, seqs):
    c = _c(dtype=dtype, Hq=Hq, Hkv=Hkv, seqs=seqs, max_pages=64, num_k_pages=500, num_v_pages=500)
    assert so.path_paged_prefix_workspace_bytes(c, 0, 0) == so.path_paged_workspace_bytes(c, 0, 0)
    sizes, chunks = (1, 2, 63, 64, 65, 127, 129, 1000, 5000), (1, 2, 64, 65, 512, 513, 1000, 5000)
    need = {(n, k): so.path_paged_prefix_workspace_bytes(c, n, k) for n in sizes for k in chunks if k <= n}
    for (n, k), size in need.items():
        assert size > so.path_paged_workspace_bytes(c, n, k)
        assert all(size <= other for (n2, k2), other in need.items() if n <= n2 and k <= k2)
    assert so.path_paged_prefix_workspace_bytes(c, 5, 6) == 0
