"""The paged cache's argument checks, on the CPU: the binding's (tensor shapes, dtypes,
devices) and the C ABI's (sizes, lists of rows, alignment), all before any launch."""
import ctypes

import pytest
import torch

import dependent_position_encoded_gb300 as pa

S, MP, P, HQ, HKV, PAGE, D, N = 3, 4, 9, 4, 2, 16, 64, 6
BF = torch.bfloat16


def _cache(**kw):
    a = dict(k_pages=torch.zeros(P, HKV, PAGE, D, dtype=BF), v_pages=torch.zeros(P, HKV, PAGE, D, dtype=BF),
             k_table=torch.zeros(S, MP, dtype=torch.int32), v_table=torch.zeros(S, MP, dtype=torch.int32),
             lens=torch.zeros(S, dtype=torch.int32), g_pages=torch.zeros(P, HQ, PAGE),
             k_ref=torch.zeros(P, dtype=torch.int32), v_ref=torch.zeros(P, dtype=torch.int32))
    a.update(kw)
    return pa.PathPagedCache(**a)


def _step(**kw):
    a = dict(q=torch.zeros(N, HQ, D, dtype=BF), k=torch.zeros(N, HKV, D, dtype=BF),
             v=torch.zeros(N, HKV, D, dtype=BF), w=torch.zeros(N, HKV, D, dtype=BF),
             beta=torch.zeros(N, HKV), log_f=torch.zeros(N, HQ),
             cu_tokens=torch.zeros(S + 1, dtype=torch.int32))
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,exc", [
    (dict(k_pages=torch.zeros(P, HKV, PAGE, dtype=BF)), ValueError),
    (dict(v_pages=torch.zeros(P, HKV, PAGE * 2, D, dtype=BF)), ValueError),
    (dict(v_pages=torch.zeros(P, HKV, PAGE, D)), TypeError),
    (dict(k_table=torch.zeros(S, MP, dtype=torch.int64)), TypeError),
    (dict(v_table=torch.zeros(S, MP + 1, dtype=torch.int32)), ValueError),
    (dict(lens=torch.zeros(S + 1, dtype=torch.int32)), ValueError),
    (dict(lens=None), TypeError),
    (dict(g_pages=torch.zeros(P, HQ + 1, PAGE)), ValueError),
    (dict(g_pages=torch.zeros(P, HQ, PAGE, dtype=BF)), TypeError),
    (dict(g_pages=None), TypeError),
    (dict(k_ref=torch.zeros(P - 1, dtype=torch.int32)), ValueError),
    (dict(v_ref=None), TypeError),
])
def test_cache_errors_raise_before_any_call(kw, exc):
    c, a = _cache(**kw), _step()
    with pytest.raises(exc):
        pa.path_fox_paged_extend(*a.values(), c, 2)


@pytest.mark.parametrize("kw,exc", [
    (dict(q=torch.zeros(N, HQ, D)), TypeError),
    (dict(q=torch.zeros(N, HQ * D, dtype=BF)), ValueError),
    (dict(k=torch.zeros(N, HQ, D, dtype=BF)), ValueError),
    (dict(v=torch.zeros(N - 1, HKV, D, dtype=BF)), ValueError),
    (dict(w=torch.zeros(N, HKV, D // 2, dtype=BF)), ValueError),
    (dict(beta=torch.zeros(N, HQ)), ValueError),
    (dict(beta=torch.zeros(N, HKV, dtype=BF)), TypeError),
    (dict(log_f=torch.zeros(N, HKV)), ValueError),
    (dict(log_f=None), TypeError),
    (dict(cu_tokens=torch.zeros(S, dtype=torch.int32)), ValueError),
    (dict(cu_tokens=torch.zeros(S + 1, dtype=torch.int64)), TypeError),
    (dict(q=torch.zeros(N, D, HQ, dtype=BF).transpose(1, 2)), ValueError),
])
def test_step_errors_raise_before_any_call(kw, exc):
    a = _step(**kw)
    with pytest.raises(exc):
        pa.path_fox_paged_extend(*a.values(), _cache(), 2)


def test_out_is_checked():
    a = _step()
    for out, exc in ((torch.zeros(N, HQ, D), TypeError), (torch.zeros(N, HKV, D, dtype=BF), ValueError),
                     (torch.zeros(1, HQ, D, dtype=BF).expand(N, HQ, D), ValueError)):
        with pytest.raises(exc):
            pa.path_fox_paged_extend(*a.values(), _cache(), 2, out=out)


def test_host_tensors_need_a_gpu():
    with pytest.raises(TypeError, match="CUDA"):
        pa.path_fox_paged_extend(*_step().values(), _cache(), 2)
    with pytest.raises(TypeError, match="CUDA"):
        pa.path_paged_compact(_cache())
    with pytest.raises(TypeError):
        pa.path_paged_reserve(torch.zeros(S), _cache())
    with pytest.raises(TypeError):
        pa.path_paged_extend(*list(_step().values())[:5], torch.zeros(S + 1, dtype=torch.int32), None, 2)
    with pytest.raises(ValueError):
        pa.path_paged_fork([0], [1, 2], _cache())


# ---------------------------------------------------------------- the C ABI, fake pointers

FAKE = 0x7F0000000000  # 256-byte aligned, never dereferenced


def _gpu():
    return torch.cuda.is_available()


no_gpu = pytest.mark.skipif(_gpu(), reason="fake device pointers: run only where no GPU is reachable")


def _c(**kw):
    a = dict(k_pages=FAKE, v_pages=FAKE, g_pages=FAKE, k_table=FAKE, v_table=FAKE, k_ref=FAKE,
             v_ref=FAKE, lens=FAKE, seqs=S, max_pages=MP, page=PAGE, num_k_pages=P, num_v_pages=P,
             Hq=HQ, Hkv=HKV, d=D, dtype=1)
    a.update(kw)
    return ctypes.byref(pa._CPagedCache(*a.values()))


def _extend(so, cache, fox=True, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, w=FAKE, beta=FAKE, log_f=FAKE, cu=FAKE, N=N, chunk=2,
             scale=0.125, out=FAKE, st=None, ws=FAKE, bytes=1 << 30, stream=None)
    a.update(kw)
    args = [a[n] for n in ("q", "k", "v", "w", "beta")] + ([a["log_f"]] if fox else [])
    fn = so.path_fox_paged_extend if fox else so.path_paged_extend
    return fn(cache, *args, a["cu"], a["N"], a["chunk"], a["scale"], a["out"], a["st"], a["ws"],
              a["bytes"], a["stream"])


def _strides(**kw):
    a = {n: (64, 64) for n in ("q", "k", "v", "w", "beta", "log_f", "out")}
    a.update(kw)
    return (ctypes.c_int64 * 14)(*[x for n in a for x in a[n]])


@no_gpu
@pytest.mark.parametrize("cache,kw,code", [
    (dict(k_pages=None), {}, pa.ERR_NULL), (dict(v_table=None), {}, pa.ERR_NULL),
    (dict(lens=None), {}, pa.ERR_NULL), (dict(g_pages=None), {}, pa.ERR_NULL),
    (dict(k_pages=FAKE + 8), {}, pa.ERR_ALIGN), (dict(k_table=FAKE + 2), {}, pa.ERR_ALIGN),
    (dict(d=96), {}, pa.ERR_SHAPE), (dict(page=24), {}, pa.ERR_SHAPE), (dict(page=8), {}, pa.ERR_SHAPE),
    (dict(page=512), {}, pa.ERR_SHAPE), (dict(Hkv=3), {}, pa.ERR_SHAPE), (dict(Hkv=0), {}, pa.ERR_SHAPE),
    (dict(seqs=-1), {}, pa.ERR_SHAPE), (dict(max_pages=1 << 20), {}, pa.ERR_SHAPE),
    (dict(dtype=2), {}, pa.ERR_DTYPE),
    ({}, dict(q=None), pa.ERR_NULL), ({}, dict(log_f=None), pa.ERR_NULL), ({}, dict(cu=None), pa.ERR_NULL),
    ({}, dict(ws=None), pa.ERR_NULL), ({}, dict(out=FAKE + 8), pa.ERR_ALIGN),
    ({}, dict(ws=FAKE + 16), pa.ERR_ALIGN), ({}, dict(beta=FAKE + 2), pa.ERR_ALIGN),
    ({}, dict(N=-1), pa.ERR_SHAPE), ({}, dict(chunk=0), pa.ERR_SHAPE), ({}, dict(chunk=N + 1), pa.ERR_SHAPE),
    ({}, dict(scale=float("nan")), pa.ERR_ARG), ({}, dict(bytes=100), pa.ERR_WORKSPACE),
    ({}, dict(st="odd"), pa.ERR_ALIGN), ({}, dict(st="neg"), pa.ERR_ALIGN),
])
def test_extend_rejects_bad_arguments_before_launch(lib, cache, kw, code):
    if "st" in kw:
        kw = dict(kw, st=_strides(k=(64, 4)) if kw["st"] == "odd" else _strides(out=(-64, 64)))
    assert _extend(lib._load(), _c(**cache), **kw) == code


@no_gpu
def test_empty_calls_launch_nothing(lib):
    so = lib._load()
    assert _extend(so, _c(), N=0, chunk=0, q=None, ws=None) == pa.OK
    assert _extend(so, _c(seqs=0), q=None, ws=None) == pa.OK
    assert so.path_paged_fork(_c(), None, None, 0, None, 0, None) == pa.OK
    assert so.path_paged_free(_c(), None, 0, None, 0, None) == pa.OK
    assert so.path_paged_reserve(_c(seqs=0), None, None, 0, None) == pa.OK
    assert so.path_paged_compact(_c(num_k_pages=0, num_v_pages=0), None, 0, None) == pa.OK


@no_gpu
@pytest.mark.parametrize("src,dst,code", [
    ([0], [0], pa.ERR_ARG), ([0, 1], [2, 2], pa.ERR_ARG), ([0, 1], [1, 2], pa.ERR_ARG),
    ([3], [0], pa.ERR_ARG), ([0], [-1], pa.ERR_ARG), ([0] * 1025, [1] * 1025, pa.ERR_SHAPE),
])
def test_fork_rejects_bad_rows(lib, src, dst, code):
    a, b = ((ctypes.c_int * len(x))(*x) for x in (src, dst))
    assert lib._load().path_paged_fork(_c(), a, b, len(src), FAKE, 1 << 30, None) == code


@no_gpu
def test_page_calls_reject_bad_arguments(lib):
    so = lib._load()
    row = (ctypes.c_int * 2)(1, 1)
    assert so.path_paged_free(_c(), row, 2, FAKE, 1 << 30, None) == pa.ERR_ARG
    assert so.path_paged_free(_c(), None, 1, FAKE, 1 << 30, None) == pa.ERR_NULL
    assert so.path_paged_free(_c(k_ref=None), row, 1, FAKE, 1 << 30, None) == pa.ERR_NULL
    assert so.path_paged_free(_c(v_ref=FAKE + 4), row, 1, FAKE, 1 << 30, None) == pa.ERR_ALIGN
    assert so.path_paged_free(_c(), row, 1, FAKE, 64, None) == pa.ERR_WORKSPACE
    assert so.path_paged_reserve(_c(), None, FAKE, 1 << 30, None) == pa.ERR_NULL
    assert so.path_paged_reserve(_c(), FAKE + 1, FAKE, 1 << 30, None) == pa.ERR_ALIGN
    assert so.path_paged_compact(_c(), None, 1 << 30, None) == pa.ERR_NULL
    assert so.path_paged_compact(None, FAKE, 1 << 30, None) == pa.ERR_NULL


def test_workspace_sizes(lib):
    so = lib._load()
    assert so.path_paged_workspace_bytes(_c(), 0, 0) > 256
    assert so.path_paged_workspace_bytes(_c(d=96), 0, 0) == 0
    assert so.path_paged_workspace_bytes(_c(), 5, 6) == 0
    assert so.path_paged_workspace_bytes(None, 1, 1) == 0
    # a workspace never shrinks as the step grows
    for dtype in (0, 1):
        for hq, hkv in ((1, 1), (8, 2), (48, 16)):
            c = dict(dtype=dtype, Hq=hq, Hkv=hkv, seqs=5, max_pages=2048)
            last = 0
            for n in (1, 2, 63, 64, 65, 200, 640, 1000, 5000, 20000):
                for chunk in (1, 2, 64, 65, n):
                    if chunk > n:
                        continue
                    now = so.path_paged_workspace_bytes(_c(**c), n, chunk)
                    assert now >= last
                    last = max(last, so.path_paged_workspace_bytes(_c(**c), n, 1))
