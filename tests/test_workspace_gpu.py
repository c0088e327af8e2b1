"""Workspaces of the host are refused by every call that takes one."""
import pytest
import torch

import path_inputs as pi

pytestmark = pytest.mark.gpu


def test_host_workspaces_are_refused(lib):
    B, H, L = 1, 2, 80
    x = pi.make_fwd_inputs(B, H, L, seed=3, fox=True, device="cuda")
    ws = torch.zeros(1 << 24, dtype=torch.uint8)
    args = [x[n] for n in ("q", "k", "v", "w", "beta")]
    out, lse = lib.path_attn_fwd(*args)
    kc = torch.zeros((B, H, 64, 64), dtype=torch.bfloat16, device="cuda")
    one = [t[:, :, 0].contiguous() for t in args]
    gate = x["log_f"][:, :, 0].contiguous()
    gc = torch.zeros((B, H, 64), device="cuda")
    calls = [
        lambda: lib.path_attn_fwd(*args, workspace=ws),
        lambda: lib.path_fox_fwd(*args, x["log_f"], workspace=ws),
        lambda: lib.path_attn_bwd(*args, out, lse, out, workspace=ws),
        lambda: lib.path_fox_bwd(*args, x["log_f"], out, lse, out, workspace=ws),
        lambda: lib.path_fwd_prepare(x["q"], x["k"], x["w"], x["beta"], ws),
        lambda: lib.path_fwd_scan(x["v"], ws),
        lambda: lib.path_fox_first_blocks(ws, B, H, L, torch.bfloat16),
        lambda: lib.path_decode_step(*one, kc, kc.clone(), 5, workspace=ws),
        lambda: lib.path_fox_decode_step(*one, gate, kc, kc.clone(), gc, 5, workspace=ws),
    ]
    for call in calls:
        with pytest.raises(TypeError, match="workspace"):
            call()
    with pytest.raises(ValueError, match="workspace"):
        lib.path_attn_fwd(*args, workspace=torch.zeros(1, dtype=torch.uint8, device="cuda").expand(1 << 24))
