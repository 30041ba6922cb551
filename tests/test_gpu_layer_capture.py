"""Packed prompts captured into a graph: the offsets lie on the device, so a
replay takes whatever they hold then; and calls of several host threads."""
import threading

import pytest
import torch

import gated_delta_rule_121_b200 as kda
from layer_inputs import offsets, randn, scan_inputs
from test_gpu_layer_scan import run

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
BATCHES = [[1000, 0, 700, 1, 299], [0, 0, 2000, 0, 0], [400] * 5, [1, 2, 3, 4, 5], [0] * 5, [64, 65, 63, 1600, 208]]


@pytest.mark.parametrize("dtype,dk,dv", [(BF16, 128, 64), (BF16, 64, 128), (BF16, 32, 16), (F32, 16, 32)])
def test_offsets_that_change_between_replays(dtype, dk, dv):
    T, H = 2000, 2
    d, g = scan_inputs(91, (1, T), H, 1, dk, dv, dtype, rate=0.1)
    x, w = randn(g, 1, T, 72, dtype=dtype), randn(g, 72, 4)
    conv0, init = randn(g, 5, 3, 72, dtype=dtype), randn(g, 5, H, dk, dv)
    cu = offsets(BATCHES[0])
    out, u = torch.empty(1, T, H, dv, dtype=dtype, device="cuda"), torch.empty_like(x)
    state, conv_state = init.clone(), conv0.clone()

    def call():
        kda.kda_conv_fwd(x, w, None, conv_state, cu, out=u, final_state=conv_state)
        run(d, state, cu, out=out, final_state=state)

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lengths in BATCHES + BATCHES[:1]:
        now = offsets(lengths)
        want, wfin = run(d, init, now, out=torch.full_like(out, 3))
        wu, wconv = kda.kda_conv_fwd(x, w, None, conv0, now, out=torch.full_like(u, 3))
        cu.copy_(now)
        state.copy_(init)
        conv_state.copy_(conv0)
        out.fill_(3)
        u.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(state, wfin), lengths
        assert torch.equal(u, wu) and torch.equal(conv_state, wconv), lengths


def test_calls_of_several_threads():
    a = []
    for i in range(6):
        d, g = scan_inputs(200 + i, (1, 900 + 100 * i), 2, 1, 128 if i % 2 else 64, 64, BF16, rate=0.1)
        a.append((d, run(d, None, None)))
    torch.cuda.synchronize()
    bad = []

    def work(d, want):
        s = torch.cuda.Stream()
        for _ in range(20):
            with torch.cuda.stream(s):
                got = run(d, None, None)
            s.synchronize()
            if not all(torch.equal(x, y) for x, y in zip(got, want)):
                bad.append(d["x"].shape)

    threads = [threading.Thread(target=work, args=v) for v in a]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
