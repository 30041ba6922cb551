"""The scan's workspace: its size never falls as a batch or its prompts grow, so
that one made for the largest call serves every other one."""
import pytest
import torch

import gated_delta_rule_121_b200 as kda
from layer_inputs import offsets, randn, scan_inputs
from test_gpu_layer_scan import run

BF16, F32 = torch.bfloat16, torch.float32
size = kda.kda_ssm_fwd_workspace_size
FORMS = [(96, 8, 128, 64, BF16), (16, 1, 128, 128, BF16), (2, 1, 64, 64, BF16), (1, 1, 128, 128, BF16), (5, 1, 128, 64, BF16),
         (4, 2, 16, 16, F32), (48, 1, 32, 64, BF16), (8, 8, 128, 128, F32)]


@pytest.mark.parametrize("H,G,dk,dv,dtype", FORMS)
@pytest.mark.parametrize("packed", [False, True])
def test_size_grows_with_the_batch(H, G, dk, dv, dtype, packed):
    for B in (1, 2, 7, 40, 300):
        last = 0
        for T in [*range(0, 9000, 61), *range(9000, 1 << 20, 4999), 1 << 24]:
            n = size(B, T, H, G, dk, dv, packed, dtype)
            assert n >= max(last, 256), (B, T)
            last = n
        # sixteen device-fulls of states of one block each, and the table
        assert last <= (170 << 20) + 64 * B
    for T in (100, 1000, 5000, 65536):
        last = 0
        for B in [*range(0, 200), *range(200, 3000, 97), 100000]:
            n = size(B, T, H, G, dk, dv, packed, dtype)
            assert n >= max(last, 256), (B, T)
            last = n


@pytest.mark.gpu
@pytest.mark.parametrize("H,G,dk,dv,dtype", [(2, 1, 128, 64, BF16), (1, 1, 64, 128, BF16), (2, 2, 32, 16, BF16), (2, 1, 16, 32, F32)])
def test_one_workspace_for_all(H, G, dk, dv, dtype):
    """Of exactly the largest call's size, filled with other calls' remains."""
    ws = torch.full((max(size(4, 3200, H, G, dk, dv, p, dtype) for p in (False, True)),), 0xff, dtype=torch.uint8, device="cuda")
    for B, T in ((4, 3200), (1, 3136), (4, 1088), (2, 1024), (3, 513), (1, 130), (4, 1), (2, 2500)):
        d, g = scan_inputs(T, (B, T), H, G, dk, dv, dtype, rate=0.1)
        init = randn(g, B, H, dk, dv)
        for a, b in zip(run(d, init, None, workspace=ws), run(d, init, None)):
            assert torch.equal(a, b), (B, T)
        if B == 1 and T > 700:
            cu = offsets([T - 700, 0, 600, 100])
            init = randn(g, 4, H, dk, dv)
            for a, b in zip(run(d, init, cu, workspace=ws), run(d, init, cu)):
                assert torch.equal(a, b), T
        assert kda.kda_workspace_status(ws) == kda.KDA_OK
