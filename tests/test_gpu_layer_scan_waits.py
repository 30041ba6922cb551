"""The tensor-core scan's bounded waits.  The warp that loads a block's inputs
waits for what cannot come, and the other warps for the loads that it does not
make: the call ends all the same, the workspace says KDA_ERR_TIMEOUT, and the next call,
in the same workspace, gives the bits it gave before."""
import ctypes
import time

import pytest
import torch

import gated_delta_rule_121_b200 as kda
from gated_delta_rule_121_b200 import layer
from layer_inputs import offsets, randn, scan_inputs
from test_gpu_layer_scan import run

BF16, F32 = torch.bfloat16, torch.float32
NEVER = 2 ** 31 - 1


def hook(d, init, cu, out, fin, ws, wait_ns, stop_at):
    f = kda.lib().kda_testing_ssm_fwd
    f.restype = ctypes.c_int
    f.argtypes = layer._SIGNATURES["kda_ssm_fwd"] + [ctypes.c_uint64, ctypes.c_int]
    B, T, H, dv = d["x"].shape
    G, dk = d["b"].shape[-2:]
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    rows = [v for k in ("x", "b", "c") for v in (p(d[k]), d[k].stride(1))]
    return f(*rows, *(p(d[k]) for k in ("delta", "A_log", "D", "dt_bias")), p(init), p(out), p(fin),
             B if cu is None else cu.numel() - 1, T, H, G, dk, dv, p(cu),
             torch.cuda.current_stream().cuda_stream if d["x"].is_cuda else None,
             kda.KDA_BF16 if d["x"].dtype == BF16 else kda.KDA_F32, p(ws), ws.numel(), wait_ns, stop_at)


def test_only_the_tensor_core_path_has_the_hook():
    for dtype, dk in ((F32, 128), (BF16, 32)):
        d, g = scan_inputs(1, (1, 70), 2, 1, dk, 64, dtype, device="cpu")
        ws = torch.empty(1 << 20, dtype=torch.uint8)
        assert hook(d, None, None, d["x"], None, ws, 1000, 0) == kda.KDA_ERR_UNSUPPORTED


# Chunks that are loaded ahead: 5 (first pass over pieces: 6) of x, 3 (6) of b and c.
@pytest.mark.gpu
@pytest.mark.parametrize("dk,dv,H,B,T,lengths,stops", [
    (128, 64, 2, 1, 100, None, [-5, -4, -2]),                          # one piece, two chunks
    (128, 128, 2, 2, 1500, None, [-6, -5, -3, 0]),                     # pieces of four chunks, both passes
    (64, 64, 3, 1, 1500, [70, 0, 900, 1, 529], [-6, -5, 0]),
    (64, 128, 1, 1, None, [(7 * i * i + 3) % 183 for i in range(400)], [-5, 0, 1]),  # several items per block
])
def test_waits_run_out(dk, dv, H, B, T, lengths, stops):
    T = T or sum(lengths)
    d, g = scan_inputs(dk, (B, T), H, 1, dk, dv, BF16)
    cu = offsets(lengths) if lengths else None
    init = randn(g, len(lengths) if lengths else B, H, dk, dv)
    ws = torch.zeros(kda.kda_ssm_fwd_workspace_size(len(lengths) if lengths else B, T, H, 1, dk, dv, cu is not None),
                     dtype=torch.uint8, device="cuda")
    want, wfin = run(d, init, cu, workspace=ws)
    assert kda.kda_workspace_status(ws) == kda.KDA_OK
    for stop in stops:
        out, fin = torch.empty_like(want), torch.empty_like(wfin)
        t0 = time.perf_counter()
        assert hook(d, init, cu, out, fin, ws, 1_000_000, stop) == kda.KDA_OK
        assert kda.kda_workspace_status(ws) == kda.KDA_ERR_TIMEOUT, stop
        assert time.perf_counter() - t0 < 1.0  # waits of 1 ms, a few waves of blocks
        out, fin = run(d, init, cu, workspace=ws)
        assert kda.kda_workspace_status(ws) == kda.KDA_OK
        assert torch.equal(out, want) and torch.equal(fin, wfin)


@pytest.mark.gpu
def test_the_hook_alone_changes_nothing():
    d, g = scan_inputs(3, (2, 700), 2, 1, 128, 64, BF16)
    ws = torch.empty(kda.kda_ssm_fwd_workspace_size(2, 700, 2, 1, 128, 64), dtype=torch.uint8, device="cuda")
    want, wfin = run(d, None, None)
    out, fin = torch.empty_like(want), torch.empty_like(wfin)
    assert hook(d, None, None, out, fin, ws, 10 ** 12, NEVER) == kda.KDA_OK
    assert kda.kda_workspace_status(ws) == kda.KDA_OK
    assert torch.equal(out, want) and torch.equal(fin, wfin)
