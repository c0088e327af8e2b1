"""GB300 (sm_103a) PaTH attention.

A thin Python binding over ``libpath_attn.so``, whose C ABI is declared in
``include/path_attn.h``. Every step of the computation runs in the library's
CUDA kernels; this module only checks tensor arguments, allocates outputs and
workspaces with PyTorch (device memory and streams are PyTorch's job here) and
passes raw pointers. There is no CPU fallback: without the built library or a
CUDA device every call raises.

Entry points keep the C names: ``path_attn_fwd``, ``path_fox_fwd``,
``path_fwd_prepare``, ``path_fwd_scan``, ``path_decode_step``, ``path_fox_decode_step``,
``path_wbeta_produce``, ``path_paged_extend``, ``path_fox_paged_extend``,
``path_paged_window_extend``, ``path_fox_paged_window_extend``, ``path_paged_prefix_extend``,
``path_fox_paged_prefix_extend``, ``path_paged_reserve``,
``path_paged_fork``, ``path_paged_free``, ``path_paged_trim``, ``path_paged_compact`` (on a
``PathPagedCache``), ``path_workspace_bytes``, ``path_check_workspace``, ``path_status_string``.
"""
import ctypes
import dataclasses
import functools
import math
import os

from . import build as _build

# status codes and enums, mirroring include/path_attn.h
OK, ERR_NULL, ERR_SHAPE, ERR_DTYPE, ERR_ALIGN, ERR_WORKSPACE, ERR_CAPACITY, ERR_TIMEOUT, \
    ERR_CUDA, ERR_ARG, ERR_CACHE = range(11)
F32, BF16 = 0, 1
OP_FWD, OP_FOX_FWD, OP_DECODE, OP_FOX_DECODE, OP_BWD, OP_FOX_BWD = 0, 1, 2, 3, 4, 5
HEAD_DIM = 64

EXPORTED = ("path_workspace_bytes", "path_attn_fwd", "path_fox_fwd", "path_fwd_prepare",
            "path_fwd_scan", "path_decode_step", "path_check_workspace", "path_status_string",
            "path_decode_step_noalloc", "path_fox_first_blocks", "path_fox_decode_step",
            "path_wbeta_workspace_bytes", "path_wbeta_produce", "path_attn_bwd",
            "path_fox_bwd", "path_paged_workspace_bytes", "path_paged_extend",
            "path_fox_paged_extend", "path_paged_reserve", "path_paged_fork", "path_paged_free",
            "path_paged_compact", "path_paged_window_extend", "path_fox_paged_window_extend",
            "path_paged_trim", "path_paged_trim_rows", "path_paged_prefix_workspace_bytes",
            "path_paged_prefix_extend", "path_fox_paged_prefix_extend")

_lib = None


class _CPagedCache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_pages", "v_pages", "g_pages", "k_table",
                                               "v_table", "k_ref", "v_ref", "lens")] + \
               [(n, ctypes.c_int) for n in ("seqs", "max_pages", "page", "num_k_pages",
                                            "num_v_pages", "Hq", "Hkv", "d", "dtype")]


# path_paged_strides: {token, head} strides of q, k, v, w, beta, log_f, out
_C14 = ctypes.c_int64 * 14


class PathError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__("%s: %s" % (where, path_status_string(code)))


def library_path():
    return _build.LIB


def ensure_built():
    """Builds libpath_attn.so if it is missing or older than its sources."""
    if not _build.up_to_date():
        _build.build()
    return _build.LIB


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_build.LIB):
        raise RuntimeError("libpath_attn.so is not built; run dependent_position_encoded_gb300."
                           "build.build() (or __graft_entry__.build())")
    lib = ctypes.CDLL(_build.LIB)
    P, I, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.path_workspace_bytes.argtypes = [I, I, I, I, I, I]
    lib.path_workspace_bytes.restype = S
    lib.path_attn_fwd.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, F, P, S, P]
    lib.path_attn_fwd.restype = I
    lib.path_fox_fwd.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, F, P, S, P]
    lib.path_fox_fwd.restype = I
    lib.path_fwd_prepare.argtypes = [P, P, P, P, P, I, I, I, I, I, F, P, S, P]
    lib.path_fwd_prepare.restype = I
    lib.path_fwd_scan.argtypes = [P, P, P, I, I, I, I, I, I, F, P, S, P]
    lib.path_fwd_scan.restype = I
    lib.path_decode_step.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, F, P, P, S, P]
    lib.path_decode_step.restype = I
    lib.path_fox_decode_step.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, P, P, S,
                                         P]
    lib.path_fox_decode_step.restype = I
    lib.path_wbeta_workspace_bytes.argtypes = [I, I, I, I, I, I, I]
    lib.path_wbeta_workspace_bytes.restype = S
    lib.path_wbeta_produce.argtypes = [P, P, P, P, P, P, F, P, P, I, I, I, I, I, I, I, P, S, P]
    lib.path_wbeta_produce.restype = I
    lib.path_attn_bwd.argtypes = [P] * 8 + [I] * 5 + [F] + [P] * 6 + [S, P]
    lib.path_attn_bwd.restype = I
    lib.path_fox_bwd.argtypes = [P] * 9 + [I] * 5 + [F] + [P] * 7 + [S, P]
    lib.path_fox_bwd.restype = I
    lib.path_decode_step_noalloc.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, F, P, P]
    lib.path_decode_step_noalloc.restype = I
    lib.path_fox_first_blocks.argtypes = [P, S, I, I, I, I, I, P, P]
    lib.path_fox_first_blocks.restype = I
    C = ctypes.POINTER(_CPagedCache)
    T = ctypes.POINTER(ctypes.c_int64)
    lib.path_paged_workspace_bytes.argtypes = [C, I, I]
    lib.path_paged_workspace_bytes.restype = S
    lib.path_paged_extend.argtypes = [C, P, P, P, P, P, P, I, I, F, P, T, P, S, P]
    lib.path_paged_extend.restype = I
    lib.path_fox_paged_extend.argtypes = [C, P, P, P, P, P, P, P, I, I, F, P, T, P, S, P]
    lib.path_fox_paged_extend.restype = I
    lib.path_paged_window_extend.argtypes = [C, P, P, P, P, P, P, I, I, I, I, F, P, T, P, S, P]
    lib.path_paged_window_extend.restype = I
    lib.path_fox_paged_window_extend.argtypes = [C, P, P, P, P, P, P, P, I, I, I, I, F, P, T, P, S, P]
    lib.path_fox_paged_window_extend.restype = I
    lib.path_paged_prefix_workspace_bytes.argtypes = [C, I, I]
    lib.path_paged_prefix_workspace_bytes.restype = S
    lib.path_paged_prefix_extend.argtypes = [C, P, P, P, P, P, P, I, I, P, P, F, P, T, P, S, P]
    lib.path_paged_prefix_extend.restype = I
    lib.path_fox_paged_prefix_extend.argtypes = [C, P, P, P, P, P, P, P, I, I, P, P, P, F, P, T, P, S, P]
    lib.path_fox_paged_prefix_extend.restype = I
    lib.path_paged_trim.argtypes = [C, I, I, P, S, P]
    lib.path_paged_trim.restype = I
    lib.path_paged_trim_rows.argtypes = [C, P, I, I, I, P, S, P]
    lib.path_paged_trim_rows.restype = I
    lib.path_paged_reserve.argtypes = [C, P, P, S, P]
    lib.path_paged_reserve.restype = I
    lib.path_paged_fork.argtypes = [C, P, P, I, P, S, P]
    lib.path_paged_fork.restype = I
    lib.path_paged_free.argtypes = [C, P, I, P, S, P]
    lib.path_paged_free.restype = I
    lib.path_paged_compact.argtypes = [C, P, S, P]
    lib.path_paged_compact.restype = I
    lib.path_check_workspace.argtypes = [P, P]
    lib.path_check_workspace.restype = I
    lib.path_status_string.argtypes = [I]
    lib.path_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def path_status_string(code):
    return _load().path_status_string(int(code)).decode()


def _check(code, where):
    if code != OK:
        raise PathError(code, where)


# ---------------------------------------------------------------- marshalling helpers

def _torch():
    import torch
    return torch


def _dtype_code_of(dtype):
    torch = _torch()
    if dtype == torch.bfloat16:
        return BF16
    if dtype == torch.float32:
        return F32
    raise TypeError("unsupported dtype %s (bfloat16 or float32)" % dtype)


def _dtype_code(t):
    return _dtype_code_of(t.dtype)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _cuda_tensor(t, name, dtype=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    return t


def _stream(stream, device):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _ws(workspace, device):
    """A workspace's address and size: a contiguous tensor on the call's device."""
    _cuda_tensor(workspace, "workspace")
    if workspace.device != device:
        raise ValueError("workspace must be on %s" % device)
    return _ptr(workspace), workspace.numel()


def _scale(scale, d):
    return 1.0 / math.sqrt(d) if scale is None else float(scale)


def path_workspace_bytes(op, B, H, L, d=HEAD_DIM, dtype=BF16):
    return int(_load().path_workspace_bytes(int(op), int(B), int(H), int(L), int(d), int(dtype)))


def new_workspace(op, B, H, L, dtype, device, d=HEAD_DIM):
    """A device workspace sized by path_workspace_bytes (256-byte aligned by PyTorch)."""
    torch = _torch()
    n = path_workspace_bytes(op, B, H, L, d, dtype)
    if n == 0:
        raise PathError(ERR_SHAPE, "path_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _fwd_args(q, k, v, w, beta):
    torch = _torch()
    _cuda_tensor(q, "q")
    dt = q.dtype
    for t, n in ((k, "k"), (v, "v"), (w, "w")):
        _cuda_tensor(t, n, dt)
        if t.shape != q.shape:
            raise ValueError("%s has shape %s, expected %s" % (n, tuple(t.shape), tuple(q.shape)))
    if q.dim() != 4:
        raise ValueError("q must be (B, H, L, d)")
    B, H, L, d = q.shape
    _cuda_tensor(beta, "beta", torch.float32)
    if beta.shape != (B, H, L):
        raise ValueError("beta must be (B, H, L) float32")
    return B, H, L, d, _dtype_code(q)


def _outputs(q, out, lse, B, H, L):
    torch = _torch()
    if out is None:
        out = torch.empty_like(q)
    else:
        _cuda_tensor(out, "out", q.dtype)
    if lse is True:
        lse = torch.empty((B, H, L), dtype=torch.float32, device=q.device)
    elif lse is not None and lse is not False:
        _cuda_tensor(lse, "lse", torch.float32)
    else:
        lse = None
    return out, lse


def path_attn_fwd(q, k, v, w, beta, out=None, lse=True, scale=None, workspace=None, stream=None):
    """PaTH forward; returns (out, lse or None). lse=True allocates it, None skips it."""
    B, H, L, d, dt = _fwd_args(q, k, v, w, beta)
    out, lse = _outputs(q, out, lse, B, H, L)
    if workspace is None:
        workspace = new_workspace(OP_FWD, B, H, L, dt, q.device, d=d)
    _check(_load().path_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(w), _ptr(beta), _ptr(out),
                                 _ptr(lse), B, H, L, d, dt, _scale(scale, d),
                                 *_ws(workspace, q.device), _stream(stream, q.device)),
           "path_attn_fwd")
    return out, lse


def _bwd_grads(q, grads, B, H, L, d, fox):
    torch = _torch()
    g = dict(grads or {})
    for n in ("dq", "dk", "dv", "dw"):
        if n not in g:
            g[n] = torch.empty((B, H, L, d), dtype=torch.float32, device=q.device)
        _cuda_tensor(g[n], n, torch.float32)
    names = ("dbeta", "dlog_f") if fox else ("dbeta",)
    for n in names:
        if n not in g:
            g[n] = torch.empty((B, H, L), dtype=torch.float32, device=q.device)
        _cuda_tensor(g[n], n, torch.float32)
    return g


def _bwd_checks(q, out, lse, d_out, B, H, L):
    torch = _torch()
    _cuda_tensor(out, "out", q.dtype)
    _cuda_tensor(d_out, "d_out", q.dtype)
    _cuda_tensor(lse, "lse", torch.float32)
    if out.shape != q.shape or d_out.shape != q.shape or lse.shape != (B, H, L):
        raise ValueError("out, d_out must be (B, H, L, d) and lse (B, H, L)")


def path_attn_bwd(q, k, v, w, beta, out, lse, d_out, scale=None, grads=None, workspace=None,
                  stream=None):
    """PaTH backward; returns a dict of fp32 gradients dq, dk, dv, dw (B, H, L, d) and
    dbeta (B, H, L). `out` and `lse` are the forward's outputs for the same inputs and scale;
    `grads` may hold preallocated fp32 buffers under those names."""
    B, H, L, d, dt = _fwd_args(q, k, v, w, beta)
    _bwd_checks(q, out, lse, d_out, B, H, L)
    g = _bwd_grads(q, grads, B, H, L, d, False)
    if workspace is None:
        workspace = new_workspace(OP_BWD, B, H, L, dt, q.device, d=d)
    _check(_load().path_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(w), _ptr(beta), _ptr(out),
                                 _ptr(lse), _ptr(d_out), B, H, L, d, dt, _scale(scale, d),
                                 _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]), _ptr(g["dw"]),
                                 _ptr(g["dbeta"]), *_ws(workspace, q.device),
                                 _stream(stream, q.device)), "path_attn_bwd")
    return g


def path_fox_bwd(q, k, v, w, beta, log_f, out, lse, d_out, scale=None, grads=None,
                 workspace=None, stream=None):
    """PaTH-FoX backward; as path_attn_bwd plus dlog_f (B, H, L) fp32. `out` and `lse` are
    path_fox_fwd's outputs."""
    torch = _torch()
    B, H, L, d, dt = _fwd_args(q, k, v, w, beta)
    _cuda_tensor(log_f, "log_f", torch.float32)
    if log_f.shape != (B, H, L):
        raise ValueError("log_f must be (B, H, L) float32")
    _bwd_checks(q, out, lse, d_out, B, H, L)
    g = _bwd_grads(q, grads, B, H, L, d, True)
    if workspace is None:
        workspace = new_workspace(OP_FOX_BWD, B, H, L, dt, q.device, d=d)
    _check(_load().path_fox_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(w), _ptr(beta), _ptr(log_f),
                                _ptr(out), _ptr(lse), _ptr(d_out), B, H, L, d, dt,
                                _scale(scale, d), _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]),
                                _ptr(g["dw"]), _ptr(g["dbeta"]), _ptr(g["dlog_f"]),
                                *_ws(workspace, q.device), _stream(stream, q.device)),
           "path_fox_bwd")
    return g


def path_fox_fwd(q, k, v, w, beta, log_f, out=None, lse=True, scale=None, workspace=None,
                 stream=None):
    """PaTH-FoX forward; returns (out, lse or None)."""
    torch = _torch()
    B, H, L, d, dt = _fwd_args(q, k, v, w, beta)
    _cuda_tensor(log_f, "log_f", torch.float32)
    if log_f.shape != (B, H, L):
        raise ValueError("log_f must be (B, H, L) float32")
    out, lse = _outputs(q, out, lse, B, H, L)
    if workspace is None:
        workspace = new_workspace(OP_FOX_FWD, B, H, L, dt, q.device, d=d)
    _check(_load().path_fox_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(w), _ptr(beta), _ptr(log_f),
                                _ptr(out), _ptr(lse), B, H, L, d, dt, _scale(scale, d),
                                *_ws(workspace, q.device), _stream(stream, q.device)),
           "path_fox_fwd")
    return out, lse


def path_fwd_prepare(q, k, w, beta, workspace, log_f=None, scale=None, stream=None):
    """First stage (UT preprocessing) into `workspace`."""
    torch = _torch()
    B, H, L, d, dt = _fwd_args(q, k, q, w, beta)
    if log_f is not None:
        _cuda_tensor(log_f, "log_f", torch.float32)
    _check(_load().path_fwd_prepare(_ptr(q), _ptr(k), _ptr(w), _ptr(beta), _ptr(log_f), B, H, L,
                                    d, dt, _scale(scale, d), *_ws(workspace, q.device),
                                    _stream(stream, q.device)), "path_fwd_prepare")


def path_fwd_scan(v, workspace, out=None, lse=True, fox=False, scale=None, stream=None):
    """Second stage (block scan) from `workspace`; returns (out, lse or None)."""
    _cuda_tensor(v, "v")
    B, H, L, d = v.shape
    dt = _dtype_code(v)
    out, lse = _outputs(v, out, lse, B, H, L)
    _check(_load().path_fwd_scan(_ptr(v), _ptr(out), _ptr(lse), int(bool(fox)), B, H, L, d, dt,
                                 _scale(scale, d), *_ws(workspace, v.device),
                                 _stream(stream, v.device)), "path_fwd_scan")
    return out, lse


def path_fox_first_blocks(workspace, B, H, L, dtype, stream=None, d=HEAD_DIM):
    """PaTH-FoX early-exit extents left in `workspace` by path_fwd_prepare(..., log_f):
    an int32 tensor (B, H, ceil(L / 64)) of the lowest key block each query block needs.
    Head size 64 only: the head-size-128 scan decides its exit as it runs (d = 128 raises
    PathError with ERR_SHAPE)."""
    torch = _torch()
    nq = (L + 63) // 64
    first = torch.empty((B, H, nq), dtype=torch.int32, device=workspace.device)
    _check(_load().path_fox_first_blocks(*_ws(workspace, workspace.device), B, H, L, int(d),
                                         _dtype_code_of(dtype), _ptr(first),
                                         _stream(stream, workspace.device)),
           "path_fox_first_blocks")
    return first


def _decode_args(q, k, v, w, beta, k_cache, v_cache, out):
    """Checks the decode arguments and returns (inputs, out, (B, H, cap, d)). Shapes and
    dtypes are checked before devices, so every size error is raised before any call."""
    torch = _torch()
    named = [(k_cache, "k_cache"), (v_cache, "v_cache"), (q, "q"), (k, "k"), (v, "v"),
             (w, "w"), (beta, "beta")] + ([(out, "out")] if out is not None else [])
    for t, n in named:
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s must be a tensor" % n)
    if k_cache.dim() != 4:
        raise ValueError("k_cache must have shape (B, H, cap, d)")
    dt_t = k_cache.dtype
    B, H, cap, d = k_cache.shape
    if tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("v_cache must match k_cache")
    for t, n, dt, count in ((v_cache, "v_cache", dt_t, None), (q, "q", dt_t, B * H * d),
                            (k, "k", dt_t, B * H * d), (v, "v", dt_t, B * H * d),
                            (w, "w", dt_t, B * H * d), (beta, "beta", torch.float32, B * H),
                            (out, "out", dt_t, B * H * d)):
        if t is None:
            continue
        if t.dtype != dt:
            raise TypeError("%s must be %s, got %s" % (n, dt, t.dtype))
        if count is not None and t.numel() != count:
            raise ValueError("%s must hold %d values, got %d" % (n, count, t.numel()))
    for t, n in named:
        _cuda_tensor(t, n)
        if t.device != k_cache.device:
            raise ValueError("%s must be on %s" % (n, k_cache.device))
    if out is None:
        out = torch.empty((B, H, d), dtype=dt_t, device=k_cache.device)
    return [q, k, v, w], out, (B, H, cap, d)


def path_decode_step(q, k, v, w, beta, k_cache, v_cache, cache_len, scale=None, out=None,
                     workspace=None, stream=None):
    """One decode step: updates k_cache in place, appends (k, v) at cache_len and returns
    the attention output (B, H, d). q, k, v, w: (B, H, d) (a trailing length-1 axis is
    accepted); beta: (B, H); caches: (B, H, cap, d)."""
    ins, out, (B, H, cap, d) = _decode_args(q, k, v, w, beta, k_cache, v_cache, out)
    if workspace is None:
        workspace = new_workspace(OP_DECODE, B, H, cap, _dtype_code(k_cache), k_cache.device, d)
    _check(_load().path_decode_step(_ptr(ins[0]), _ptr(ins[1]), _ptr(ins[2]), _ptr(ins[3]),
                                    _ptr(beta), _ptr(k_cache), _ptr(v_cache), B, H,
                                    int(cache_len), cap, d, _dtype_code(k_cache),
                                    _scale(scale, d), _ptr(out),
                                    *_ws(workspace, k_cache.device),
                                    _stream(stream, k_cache.device)),
           "path_decode_step")
    return out


def path_fox_decode_step(q, k, v, w, beta, log_f, k_cache, v_cache, g_cache, cache_len,
                         scale=None, out=None, workspace=None, stream=None):
    """One PaTH-FoX decode step: as path_decode_step, plus the per-key gate sums g_cache
    (B, H, cap) fp32, updated in place (g_j += log_f for j < cache_len, g = 0 appended), and
    the bias g_j on every logit. log_f: (B, H) fp32, the new token's log forget gate."""
    torch = _torch()
    ins, out, (B, H, cap, d) = _decode_args(q, k, v, w, beta, k_cache, v_cache, out)
    _cuda_tensor(log_f, "log_f", torch.float32)
    if log_f.numel() != B * H:
        raise ValueError("log_f must hold (B, H) values")
    _cuda_tensor(g_cache, "g_cache", torch.float32)
    if tuple(g_cache.shape) != (B, H, cap):
        raise ValueError("g_cache must have shape (B, H, cap)")
    if workspace is None:
        workspace = new_workspace(OP_FOX_DECODE, B, H, cap, _dtype_code(k_cache), k_cache.device,
                                  d)
    _check(_load().path_fox_decode_step(_ptr(ins[0]), _ptr(ins[1]), _ptr(ins[2]), _ptr(ins[3]),
                                        _ptr(beta), _ptr(log_f), _ptr(k_cache), _ptr(v_cache),
                                        _ptr(g_cache), B, H, int(cache_len), cap, d,
                                        _dtype_code(k_cache), _scale(scale, d), _ptr(out),
                                        *_ws(workspace, k_cache.device),
                                        _stream(stream, k_cache.device)),
           "path_fox_decode_step")
    return out


def path_check_workspace(workspace, stream=None):
    """Synchronises the stream and returns the status code left by kernels in `workspace`."""
    return int(_load().path_check_workspace(_ptr(workspace), _stream(stream, workspace.device)))


def path_decode_step_noalloc(q, k, v, w, beta, k_cache, v_cache, cache_len, scale=None, out=None,
                             stream=None):
    """path_decode_step without a workspace, for callers that may not allocate device memory
    for the library on the call path. The split partials live in a fixed 16 MiB array inside
    the library; calls that overlap on one GPU share it and must be serialised. Raises
    PathError(ERR_WORKSPACE) when B * H * ceil(cache_len / 1024) partials do not fit."""
    ins, out, (B, H, cap, d) = _decode_args(q, k, v, w, beta, k_cache, v_cache, out)
    _check(_load().path_decode_step_noalloc(_ptr(ins[0]), _ptr(ins[1]), _ptr(ins[2]),
                                            _ptr(ins[3]), _ptr(beta), _ptr(k_cache),
                                            _ptr(v_cache), B, H, int(cache_len), cap, d,
                                            _dtype_code(k_cache), _scale(scale, d), _ptr(out),
                                            _stream(stream, k_cache.device)),
           "path_decode_step_noalloc")
    return out


def path_wbeta_workspace_bytes(B, L, D, R, H, d=HEAD_DIM, dtype=BF16):
    return int(_load().path_wbeta_workspace_bytes(int(B), int(L), int(D), int(R), int(H), int(d),
                                                  int(dtype)))


def path_wbeta_produce(x, w_down, w_up, conv, u, bias, beta_max=2.0, w_out=None, beta_out=None,
                       workspace=None, stream=None):
    """The w / beta producer: x (B, L, D) bf16; w_down (R, D), w_up (H*d, R), u (H, D) bf16;
    conv (H*d, 3) and bias (H,) fp32. Returns (w (B, H, L, d) bf16, beta (B, H, L) fp32),
    the layouts path_attn_fwd takes."""
    torch = _torch()
    _cuda_tensor(x, "x", torch.bfloat16)
    B, L, D = x.shape
    _cuda_tensor(w_down, "w_down", torch.bfloat16)
    _cuda_tensor(w_up, "w_up", torch.bfloat16)
    _cuda_tensor(u, "u", torch.bfloat16)
    _cuda_tensor(conv, "conv", torch.float32)
    _cuda_tensor(bias, "bias", torch.float32)
    R, H = w_down.shape[0], u.shape[0]
    d = w_up.shape[0] // H
    if (tuple(w_down.shape) != (R, D) or tuple(w_up.shape) != (H * d, R)
            or tuple(u.shape) != (H, D) or tuple(conv.shape) != (H * d, 3)
            or tuple(bias.shape) != (H,)):
        raise ValueError("inconsistent producer shapes")
    if w_out is None:
        w_out = torch.empty((B, H, L, d), dtype=torch.bfloat16, device=x.device)
    if beta_out is None:
        beta_out = torch.empty((B, H, L), dtype=torch.float32, device=x.device)
    if workspace is None:
        n = path_wbeta_workspace_bytes(B, L, D, R, H, d, BF16)
        if n == 0:
            raise PathError(ERR_SHAPE, "path_wbeta_workspace_bytes")
        workspace = torch.empty(n, dtype=torch.uint8, device=x.device)
    _check(_load().path_wbeta_produce(_ptr(x), _ptr(w_down), _ptr(w_up), _ptr(conv), _ptr(u),
                                      _ptr(bias), float(beta_max), _ptr(w_out), _ptr(beta_out), B,
                                      L, D, R, H, d, BF16, *_ws(workspace, x.device),
                                      _stream(stream, x.device)),
           "path_wbeta_produce")
    return w_out, beta_out


# ---------------------------------------------------------------- paged cache

@dataclasses.dataclass
class PathPagedCache:
    """The tensors of a paged cache (see path_paged_cache in include/path_attn.h): k_pages
    (pages, Hkv, page, d) and v_pages of the same form, bfloat16 or float32; k_table, v_table
    (seqs, max_pages) and lens (seqs) int32; k_ref, v_ref (pages) int32, which only the page
    calls need; g_pages (K pages, Hq, page) float32 for PaTH-FoX. The object holds no state of
    its own: calls read and update the tensors, and the caller advances ``lens``."""
    k_pages: object
    v_pages: object
    k_table: object
    v_table: object
    lens: object
    g_pages: object = None
    k_ref: object = None
    v_ref: object = None


def new_paged_cache(seqs, max_pages, num_k_pages, num_v_pages=None, Hq=1, Hkv=None, d=HEAD_DIM,
                    page=64, dtype=None, fox=False, device="cuda"):
    """An empty PathPagedCache: all pages free, no slot mapped, all lengths 0. Keys and values
    are not initialised (nothing reads a position before it is written)."""
    torch = _torch()
    Hkv = Hq if Hkv is None else Hkv
    nv = num_k_pages if num_v_pages is None else num_v_pages
    dtype = torch.bfloat16 if dtype is None else dtype
    i32 = dict(dtype=torch.int32, device=device)
    return PathPagedCache(
        k_pages=torch.empty((num_k_pages, Hkv, page, d), dtype=dtype, device=device),
        v_pages=torch.empty((nv, Hkv, page, d), dtype=dtype, device=device),
        k_table=torch.full((seqs, max_pages), -1, **i32),
        v_table=torch.full((seqs, max_pages), -1, **i32),
        lens=torch.zeros(seqs, **i32),
        g_pages=torch.empty((num_k_pages, Hq, page), dtype=torch.float32, device=device)
        if fox else None,
        k_ref=torch.zeros(num_k_pages, **i32), v_ref=torch.zeros(nv, **i32))


_I32_FIELDS = ("k_table", "v_table", "lens", "k_ref", "v_ref")


def _paged_cache(cache, counts=False, Hq=None, on_gpu=True):
    """Checks the cache's tensors and returns its C form. Shapes and dtypes are checked before
    devices (on_gpu=False: the caller checks those with _paged_devices), so that every size
    error is raised before any call. What is usual is tested in one expression (a step's host
    time is a few microseconds); what fails it goes through _paged_cache_errors."""
    torch = _torch()
    i32 = torch.int32
    try:
        kp, vp, gp, kt, vt = cache.k_pages, cache.v_pages, cache.g_pages, cache.k_table, cache.v_table
        ln, kr, vr = cache.lens, cache.k_ref, cache.v_ref
        ks, vs, ts, dtype = kp.shape, vp.shape, kt.shape, kp.dtype
        nk, Hkv, page, d = ks
        seqs, max_pages = ts
        refs = counts or kr is not None or vr is not None
        fine = (ks[1:] == vs[1:] and vp.dtype == dtype and kt.dtype == i32 and vt.dtype == i32
                and ln.dtype == i32 and vt.shape == ts and ln.shape == (seqs,) and kp.is_contiguous()
                and vp.is_contiguous() and kt.is_contiguous() and vt.is_contiguous()
                and ln.is_contiguous())
        if fine and refs:
            fine = (kr.dtype == i32 and vr.dtype == i32 and kr.shape == (nk,)
                    and vr.shape == (vs[0],) and kr.is_contiguous() and vr.is_contiguous())
        if fine and gp is not None:
            if Hq is None:
                Hq = gp.shape[1]
            fine = (gp.dtype == torch.float32 and gp.shape == (nk, Hq, page)
                    and gp.is_contiguous())
    except (AttributeError, TypeError, ValueError, IndexError):
        fine = False
    if not fine or type(cache) is not PathPagedCache:
        _paged_cache_errors(cache, counts, Hq)
    code = _dtype_code_of(dtype)
    if on_gpu:
        _paged_devices(cache)
    return _CPagedCache(kp.data_ptr(), vp.data_ptr(), None if gp is None else gp.data_ptr(),
                        kt.data_ptr(), vt.data_ptr(), kr.data_ptr() if refs else None,
                        vr.data_ptr() if refs else None, ln.data_ptr(), seqs, max_pages, page, nk,
                        vs[0], Hkv if Hq is None else Hq, Hkv, d, code)


def _paged_cache_errors(cache, counts, Hq):
    """Raises what is wrong with the cache."""
    torch = _torch()
    if type(cache) is not PathPagedCache:
        raise TypeError("cache must be a PathPagedCache")
    kp, vp, gp = cache.k_pages, cache.v_pages, cache.g_pages
    named = [("k_table", cache.k_table), ("v_table", cache.v_table), ("lens", cache.lens)]
    if counts or cache.k_ref is not None or cache.v_ref is not None:
        named += [("k_ref", cache.k_ref), ("v_ref", cache.v_ref)]
    for n, t in [("k_pages", kp), ("v_pages", vp)] + named + ([("g_pages", gp)] if gp is not None else []):
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s must be a tensor" % n)
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % n)
    for n, t in named:
        if t.dtype != torch.int32:
            raise TypeError("%s must be %s, got %s" % (n, torch.int32, t.dtype))
    if kp.dim() != 4 or vp.dim() != 4 or kp.shape[1:] != vp.shape[1:]:
        raise ValueError("k_pages and v_pages must be (pages, Hkv, page, d) of equal pages")
    if vp.dtype != kp.dtype:
        raise TypeError("v_pages must be %s, got %s" % (kp.dtype, vp.dtype))
    if cache.k_table.dim() != 2 or cache.v_table.shape != cache.k_table.shape:
        raise ValueError("k_table and v_table must be (seqs, max_pages) of equal shape")
    if cache.lens.shape != (cache.k_table.shape[0],):
        raise ValueError("lens must be (seqs,)")
    if gp is not None:
        if gp.dtype != torch.float32:
            raise TypeError("g_pages must be %s, got %s" % (torch.float32, gp.dtype))
        raise ValueError("g_pages must be (K pages, Hq, page), k_ref and v_ref one count per page")
    raise ValueError("k_ref and v_ref must hold one count per page")


def _paged_devices(cache, *more):
    """Every tensor on the GPU that holds k_pages; `more`: tensors or None."""
    dev = cache.k_pages.get_device()
    all_of = [t for t in (cache.k_pages, cache.v_pages, cache.g_pages, cache.k_table, cache.v_table,
                          cache.lens, cache.k_ref, cache.v_ref, *more) if t is not None]
    if dev < 0 or not cache.k_pages.is_cuda or [t.get_device() for t in all_of].count(dev) != len(all_of):
        if not all(t.is_cuda for t in all_of):
            raise TypeError("the cache and the step's tensors must be CUDA tensors")
        raise ValueError("the cache and the step's tensors must be on one device")
    return dev


def _paged_workspace(ws):
    """Refuses what is no workspace (`ws`: a tensor or None); its device is checked with the cache's."""
    torch = _torch()
    if ws is None or (isinstance(ws, torch.Tensor) and ws.dtype == torch.uint8 and ws.is_cuda
                      and ws.is_contiguous()):
        return
    if not isinstance(ws, torch.Tensor) or ws.dtype != torch.uint8:
        raise TypeError("workspace must be a uint8 tensor (new_paged_workspace)")
    if not ws.is_contiguous():
        raise ValueError("workspace must be contiguous")
    raise TypeError("workspace must be a CUDA tensor")


def _paged_found(name, ws, on_stream):
    """Of a workspace that the caller does not hold: waits for the call and raises what its kernels
    found wrong (in a capture there is nothing to wait for)."""
    if not _torch().cuda.is_current_stream_capturing():
        _check(_load().path_check_workspace(ws.data_ptr(), on_stream), name)


class _on:
    """The device (its index) and, where one is given, the stream of a call, as torch's current
    ones: what is allocated inside belongs to the stream that the call runs on, whose handle it
    gives."""
    __slots__ = ("guards", "dev")

    def __init__(self, dev, stream):
        cuda = _torch().cuda
        self.dev = dev
        self.guards = [] if dev == cuda.current_device() else [cuda.device(dev)]
        if stream is not None:
            if stream.device.index != dev:
                raise ValueError("stream must be on the cache's device")
            self.guards.append(cuda.stream(stream))

    def __enter__(self):
        for g in self.guards:
            g.__enter__()
        return _torch()._C._cuda_getCurrentRawStream(self.dev)

    def __exit__(self, *e):
        for g in reversed(self.guards):
            g.__exit__(*e)


def _ints(names, *values):
    """The values as C ints, which would take the low bits of larger numbers."""
    values = tuple(int(x) for x in values)
    if not all(-2**31 <= x < 2**31 for x in values):
        raise ValueError("%s must be 32-bit ints" % names)
    return values


def _window(window, sinks):
    return _ints("window and sinks", window, sinks)


def path_paged_workspace_bytes(cache, num_tokens=0, max_chunk=0, Hq=None, prefix=False):
    """Workspace bytes of every call on `cache` with up to num_tokens new tokens in all and
    max_chunk per sequence (0: the page calls alone); of those behind a prefix only with
    prefix=True. Hq: query heads, where the cache has no g_pages to tell (default: the key heads)."""
    c = _paged_cache(cache, Hq=Hq)
    call = _load().path_paged_prefix_workspace_bytes if prefix else _load().path_paged_workspace_bytes
    return int(call(ctypes.byref(c), *_ints("num_tokens and max_chunk", num_tokens, max_chunk)))


def new_paged_workspace(cache, num_tokens=0, max_chunk=0, Hq=None, prefix=False):
    """A workspace of path_paged_workspace_bytes, its status word cleared."""
    torch = _torch()
    n = path_paged_workspace_bytes(cache, num_tokens, max_chunk, Hq, prefix)
    if n == 0:
        raise PathError(ERR_SHAPE, "path_paged_workspace_bytes")
    ws = torch.empty(n, dtype=torch.uint8, device=cache.k_pages.device)
    ws[:256].zero_()
    return ws


def _paged_extend(name, q, k, v, w, beta, log_f, cu_tokens, cache, max_chunk, scale, out,
                  workspace, stream, more=(), tensors=()):
    torch = _torch()
    f32 = torch.float32
    try:
        kp = cache.k_pages
        dt, Hkv = kp.dtype, kp.shape[1]
        qs = q.shape
        N, Hq, d = qs
        rows, heads = (N, Hkv, d), (N, Hkv)
        q0, k0, v0, w0 = q.stride(), k.stride(), v.stride(), w.stride()
        b0 = beta.stride()
        f0 = (0, 0) if log_f is None else log_f.stride()
        o0 = q0 if out is None else out.stride()
        fine = (q.dtype == dt and k.dtype == dt and v.dtype == dt and w.dtype == dt
                and beta.dtype == f32 and cu_tokens.dtype == torch.int32 and k.shape == rows
                and v.shape == rows and w.shape == rows and beta.shape == heads
                and cu_tokens.dim() == 1 and cu_tokens.is_contiguous()
                and q0[2] == 1 and k0[2] == 1 and v0[2] == 1 and w0[2] == 1 and o0[2] == 1
                and (log_f is None or (log_f.dtype == f32 and log_f.shape == qs[:2]))
                and (out is None or (out.dtype == dt and out.shape == qs)))
    except (AttributeError, TypeError, ValueError, IndexError):
        fine = False
    if not fine:
        _paged_extend_errors(q, k, v, w, beta, log_f, cu_tokens, cache, out)
    c = _paged_cache(cache, Hq=Hq, on_gpu=False)
    if cu_tokens.shape[0] != c.seqs + 1:
        raise ValueError("cu_tokens must be (seqs + 1,)")
    if d != c.d:
        raise ValueError("q has head size %d, the cache %d" % (d, c.d))
    if out is not None and (N > 1 and o0[0] == 0 or Hq > 1 and o0[1] == 0):
        raise ValueError("out must not repeat its own memory")
    most = int(max_chunk)
    if not -2**31 <= most < 2**31:  # (as _ints, on the way of every step)
        raise ValueError("max_chunk must be a 32-bit int")
    _paged_workspace(workspace)
    dev = _paged_devices(cache, q, k, v, w, beta, log_f, out, cu_tokens, workspace, *tensors)
    gate = () if log_f is None else (log_f.data_ptr(),)
    with _on(dev, stream) as on_stream:
        if out is None:
            out = torch.empty_like(q)
            o0 = out.stride()
        own = workspace is None and N > 0 and c.seqs > 0
        if own:
            workspace = new_paged_workspace(cache, N, max_chunk, Hq, prefix=len(tensors) > 0)
        _check(getattr(_load(), name)(
            ctypes.byref(c), q.data_ptr(), k.data_ptr(), v.data_ptr(), w.data_ptr(),
            beta.data_ptr(), *gate, cu_tokens.data_ptr(), N, most, *more,
            *(t.data_ptr() for t in tensors), _scale(scale, d),
            out.data_ptr(), _C14(q0[0], q0[1], k0[0], k0[1], v0[0], v0[1], w0[0], w0[1], b0[0], b0[1],
                                 f0[0], f0[1], o0[0], o0[1]), None if workspace is None else workspace.data_ptr(),
            0 if workspace is None else workspace.numel(), on_stream), name)
        if own:
            _paged_found(name, workspace, on_stream)
    return out


def _paged_extend_errors(q, k, v, w, beta, log_f, cu_tokens, cache, out):
    """Raises what is wrong with a step's tensors (or with the cache)."""
    torch = _torch()
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a tensor")
    if q.dim() != 3:
        raise ValueError("q must be (tokens, Hq, d)")
    N, Hq, d = q.shape
    _paged_cache(cache, Hq=Hq, on_gpu=False)
    Hkv, dt = cache.k_pages.shape[1], cache.k_pages.dtype
    for t, n, shape, want in ((q, "q", (N, Hq, d), dt), (k, "k", (N, Hkv, d), dt),
                              (v, "v", (N, Hkv, d), dt), (w, "w", (N, Hkv, d), dt),
                              (beta, "beta", (N, Hkv), torch.float32),
                              (log_f, "log_f", (N, Hq), torch.float32), (out, "out", (N, Hq, d), dt)):
        if t is None and n in ("log_f", "out"):
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s must be a tensor" % n)
        if t.dtype != want:
            raise TypeError("%s must be %s, got %s" % (n, want, t.dtype))
        if tuple(t.shape) != shape:
            raise ValueError("%s must have shape %s, got %s" % (n, shape, tuple(t.shape)))
        if len(shape) == 3 and t.stride()[2] != 1:
            raise ValueError("the last axis of %s must be contiguous" % n)
    if not isinstance(cu_tokens, torch.Tensor) or cu_tokens.dtype != torch.int32:
        raise TypeError("cu_tokens must be an int32 tensor")
    raise ValueError("cu_tokens must be (seqs + 1,), contiguous")


def path_paged_extend(q, k, v, w, beta, cu_tokens, cache, max_chunk, scale=None, out=None,
                      workspace=None, stream=None):
    """Attention of every sequence's new tokens over its paged cache, the cached keys' update
    and the new tokens' entry into the cache; returns out (tokens, Hq, d). q: (tokens, Hq, d);
    k, v, w: (tokens, Hkv, d); beta: (tokens, Hkv); any strides with a contiguous last axis.
    cu_tokens: (seqs + 1) int32, where each sequence's tokens begin; max_chunk: the most of one
    sequence. The pages must be mapped (path_paged_reserve); the caller advances cache.lens.

    What the kernels find wrong (lengths that do not fit, pages that are not mapped) is in the
    status word of `workspace`, for path_check_workspace. Without a workspace the call makes one,
    waits for its end and raises PathError (in a capture it cannot: give a workspace)."""
    return _paged_extend("path_paged_extend", q, k, v, w, beta, None, cu_tokens, cache, max_chunk,
                         scale, out, workspace, stream)


def path_fox_paged_extend(q, k, v, w, beta, log_f, cu_tokens, cache, max_chunk, scale=None,
                          out=None, workspace=None, stream=None):
    """path_paged_extend with the forget gates of PaTH-FoX: log_f (tokens, Hq) fp32, and
    cache.g_pages advanced like the keys."""
    _paged_gates(log_f, cache)
    return _paged_extend("path_fox_paged_extend", q, k, v, w, beta, log_f, cu_tokens, cache,
                         max_chunk, scale, out, workspace, stream)


def path_paged_window_extend(q, k, v, w, beta, cu_tokens, cache, max_chunk, window, sinks=0,
                             scale=None, out=None, workspace=None, stream=None):
    """path_paged_extend through a sliding window: every new token sees the last `window`
    positions of its sequence, its own among them, and the first `sinks` ones. max_chunk must not
    be larger than the window. Cached keys that no new token sees are neither read nor advanced;
    path_paged_trim gives their pages back."""
    return _paged_extend("path_paged_window_extend", q, k, v, w, beta, None, cu_tokens, cache,
                         max_chunk, scale, out, workspace, stream, _window(window, sinks))


def path_fox_paged_window_extend(q, k, v, w, beta, log_f, cu_tokens, cache, max_chunk, window,
                                 sinks=0, scale=None, out=None, workspace=None, stream=None):
    """path_paged_window_extend with the forget gates of path_fox_paged_extend."""
    _paged_gates(log_f, cache)
    return _paged_extend("path_fox_paged_window_extend", q, k, v, w, beta, log_f, cu_tokens, cache,
                         max_chunk, scale, out, workspace, stream, _window(window, sinks))


def _prefix_tensors(q, cache, prefix_of, carry, gates=None, fox=False):
    """Checks prefix_of, carry and (PaTH-FoX) gate_carry against the cache."""
    torch = _torch()
    tensors = (prefix_of, carry, gates) if fox else (prefix_of, carry)
    try:
        (seqs,), (_, Hkv, _, d), (_, Hq, _) = cache.lens.shape, cache.k_pages.shape, q.shape
        if (prefix_of.dtype == torch.int32 and carry.dtype == torch.float32 and prefix_of.shape == (seqs,)
                and carry.shape == (seqs, Hkv, d, d) and prefix_of.is_contiguous() and carry.is_contiguous()
                and (not fox or (gates.dtype == torch.float32 and gates.shape == (seqs, Hq)
                                 and gates.is_contiguous()))):
            return tensors
    except (AttributeError, TypeError, ValueError):
        pass
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise (ValueError if isinstance(q, torch.Tensor) else TypeError)("q must be a (tokens, Hq, d) tensor")
    _paged_cache(cache, Hq=q.shape[1], on_gpu=False)
    seqs, (_, Hkv, _, d) = cache.lens.shape[0], cache.k_pages.shape
    named = [(prefix_of, "prefix_of", torch.int32, (seqs,)), (carry, "carry", torch.float32, (seqs, Hkv, d, d))]
    if fox:
        named.append((gates, "gate_carry", torch.float32, (seqs, q.shape[1])))
    for t, n, dt, shape in named:
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s must be a tensor" % n)
        if t.dtype != dt:
            raise TypeError("%s must be %s, got %s" % (n, dt, t.dtype))
        if tuple(t.shape) != shape:
            raise ValueError("%s must have shape %s, got %s" % (n, shape, tuple(t.shape)))
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % n)
    return tensors


def path_paged_prefix_extend(q, k, v, w, beta, cu_tokens, cache, prefix_of, carry, max_chunk,
                             scale=None, out=None, workspace=None, stream=None):
    """path_paged_extend for sequences that continue a prefix. prefix_of (seqs) int32: the row of the
    cache that a sequence continues, -1 for none; that row brings no tokens and stays as it is, however
    many sequences continue it. carry (seqs, Hkv, d, d) fp32: the product of the transitions of a
    sequence's own cached tokens (the identity where it has none, see new_paged_carry), advanced in
    place. Workspaces: new_paged_workspace(..., prefix=True), or none as in path_paged_extend."""
    return _paged_extend("path_paged_prefix_extend", q, k, v, w, beta, None, cu_tokens, cache, max_chunk,
                         scale, out, workspace, stream, (), _prefix_tensors(q, cache, prefix_of, carry))


def path_fox_paged_prefix_extend(q, k, v, w, beta, log_f, cu_tokens, cache, prefix_of, carry, gate_carry,
                                 max_chunk, scale=None, out=None, workspace=None, stream=None):
    """path_paged_prefix_extend with the forget gates of path_fox_paged_extend: gate_carry (seqs, Hq)
    fp32 is the sum of the gates of a sequence's own cached tokens, advanced in place."""
    _paged_gates(log_f, cache)
    return _paged_extend("path_fox_paged_prefix_extend", q, k, v, w, beta, log_f, cu_tokens, cache,
                         max_chunk, scale, out, workspace, stream, (),
                         _prefix_tensors(q, cache, prefix_of, carry, gate_carry, True))


def new_paged_carry(cache, Hq=None):
    """(carry, gate_carry) of sequences without tokens of their own: identities and zeros. To begin
    a row anew behind a prefix, set carry[row] to the identity and gate_carry[row] to 0."""
    torch = _torch()
    c = _paged_cache(cache, Hq=Hq)
    dev = cache.k_pages.device
    carry = torch.eye(c.d, dtype=torch.float32, device=dev).repeat(c.seqs, c.Hkv, 1, 1)
    return carry, torch.zeros((c.seqs, c.Hq), dtype=torch.float32, device=dev)


def _paged_gates(log_f, cache):
    if not isinstance(log_f, _torch().Tensor):
        raise TypeError("log_f must be a tensor")
    if isinstance(cache, PathPagedCache) and cache.g_pages is None:
        raise TypeError("cache.g_pages must be a tensor")


def _paged_call(name, cache, workspace, stream, *args):
    c = _paged_cache(cache, counts=True, on_gpu=False)
    _paged_workspace(workspace)
    with _on(_paged_devices(cache, workspace), stream) as on_stream:
        own = workspace is None
        if own:
            workspace = new_paged_workspace(cache)
        _check(getattr(_load(), name)(ctypes.byref(c), *args, workspace.data_ptr(),
                                      workspace.numel(), on_stream), name)
        if own:
            _paged_found(name, workspace, on_stream)
    return workspace


@functools.lru_cache(maxsize=64)
def _row_list(n):
    return ctypes.c_int * n


def _rows(rows):
    rows = [int(r) for r in rows]
    return _row_list(max(len(rows), 1))(*rows), len(rows)


def path_paged_reserve(extra, cache, workspace=None, stream=None):
    """Maps the lowest free pages so that every sequence can hold lens + extra tokens (extra:
    (seqs) int32 on the device). Nothing changes if the pages run out: the workspace's status
    word says so (path_check_workspace). Returns the workspace.

    As every page call: without a workspace it makes one, waits for its end and raises PathError
    if something was wrong; in a capture it does not wait, and the workspace that it returns has
    the status of the last replay."""
    torch = _torch()
    if not isinstance(extra, torch.Tensor):
        raise TypeError("extra must be a tensor")
    if extra.dtype != torch.int32:
        raise TypeError("extra must be torch.int32, got %s" % extra.dtype)
    if isinstance(cache, PathPagedCache) and extra.shape != cache.lens.shape:
        raise ValueError("extra must be (seqs,)")
    _cuda_tensor(extra, "extra")
    if isinstance(cache, PathPagedCache) and extra.get_device() != cache.k_pages.get_device():
        raise ValueError("extra must be on %s" % cache.k_pages.device)
    return _paged_call("path_paged_reserve", cache, workspace, stream, extra.data_ptr())


def path_paged_fork(src, dst, cache, workspace=None, stream=None):
    """Rows dst (empty) become copies of rows src (lists of ints): keys copied, full value
    pages shared, a value page that still fills copied. Workspaces as in path_paged_reserve."""
    (a, n), (b, m) = _rows(src), _rows(dst)
    if n != m:
        raise ValueError("src and dst must be equally long")
    return _paged_call("path_paged_fork", cache, workspace, stream, a, b, n)


def path_paged_free(rows, cache, workspace=None, stream=None):
    """Empties rows (a list of ints): their pages go back, their lengths become 0.
    Workspaces as in path_paged_reserve."""
    a, n = _rows(rows)
    return _paged_call("path_paged_free", cache, workspace, stream, a, n)


def path_paged_trim(cache, window, sinks=0, workspace=None, stream=None, rows=None):
    """Gives back the pages that no later step through this window reaches: the slots behind them
    move down and cache.lens falls by their tokens. rows (a list of ints): the sequences that are
    trimmed, by default every one of the cache. Rows that other steps read whole (prefixes, sequences
    behind them or of path_paged_extend) must not be among them. Workspaces as in path_paged_reserve."""
    if rows is None:
        return _paged_call("path_paged_trim", cache, workspace, stream, *_window(window, sinks))
    a, n = _rows(rows)
    return _paged_call("path_paged_trim_rows", cache, workspace, stream, a, n, *_window(window, sinks))


def path_paged_compact(cache, workspace=None, stream=None):
    """Moves the pages in use to the front of each pool; the tables follow. Workspaces as in
    path_paged_reserve."""
    return _paged_call("path_paged_compact", cache, workspace, stream)
