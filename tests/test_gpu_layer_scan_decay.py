"""The selective scan over prompts where the log decays of a chunk add up far:
every element within the bounds that ordinary decays are held to.  A score's
decay e^{G_t - G_s} must not lose what G_t and G_s have in common, and a step that
leaves nothing of the state must not blur the steps around it."""
import math

import pytest
import torch

import gated_delta_rule_121_b200 as kda
from layer_inputs import offsets, randn, scan_inputs
from oracle import layer as ref
from test_gpu_layer_scan import compare, run

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
SIZES = [(BF16, 128, 64), (BF16, 128, 128), (BF16, 64, 64), (F32, 32, 32)]


@pytest.mark.parametrize("dtype,dk,dv", SIZES)
@pytest.mark.parametrize("rate", [1e4, 1e5, 1e6])
def test_fast_rates(dtype, dk, dv, rate):
    """exp(A_log) up to 1e6 with ordinary steps: sums of 1e6 to 1e8 over a chunk."""
    d, g = scan_inputs(101, (1, 150), 4, 2, dk, dv, dtype, rate=rate)
    d["delta"][:, 40:60] = -60.0  # steps of zero: the state stands still
    init = randn(g, 1, 4, dk, dv)
    compare(*run(d, init, None), d, init, None)


@pytest.mark.parametrize("dtype,dk,dv", SIZES)
@pytest.mark.parametrize("step", [50.0, 1e3, 1e4])
def test_large_steps_throughout(dtype, dk, dv, step):
    d, g = scan_inputs(102, (2, 130), 4, 2, dk, dv, dtype, rate=16.0)
    d["dt_bias"] = None
    d["delta"] = (step * (1 + 0.1 * torch.tanh(d["delta"]))).contiguous()
    init = randn(g, 2, 4, dk, dv)
    compare(*run(d, init, None), d, init, None)


@pytest.mark.parametrize("dtype,dk,dv", SIZES)
@pytest.mark.parametrize("step", [1e2, 1e4, 1e6])
@pytest.mark.parametrize("at", [0, 1, 3, 14, 15, 16, 31, 33, 62, 63])
def test_one_large_step_ahead_of_small_ones(dtype, dk, dv, step, at):
    """A token that resets the state, at every place of interest in a chunk of 64
    (of its fours and sixteens), and slow decays around it: the rest of the chunk
    reads that token's values."""
    d, g = scan_inputs(103, (1, 140), 2, 1, dk, dv, dtype, rate=16.0)
    d["dt_bias"] = None
    d["delta"] = (0.002 * torch.rand(1, 140, 2, generator=g)).cuda()
    for chunk in (0, 64):
        d["delta"][:, chunk + at] = step
    init = randn(g, 1, 2, dk, dv)
    compare(*run(d, init, None), d, init, None)


@pytest.mark.parametrize("dtype,dk,dv", SIZES)
def test_many_resets_and_slow_decays(dtype, dk, dv):
    """Resets among slow decays, over sequences that are cut into pieces and packed ones."""
    for lengths, T in ((None, 1500), ([70, 0, 900, 1, 529], 1500)):
        d, g = scan_inputs(104, (1, T), 2, 1, dk, dv, dtype, rate=8.0)
        d["dt_bias"] = None
        delta = 0.003 * torch.rand(1, T, 2, generator=g)
        reset = torch.rand(1, T, 2, generator=g) < 0.08
        delta[reset] = torch.exp(torch.rand(int(reset.sum()), generator=g) * math.log(1e5)) * 0.5
        d["delta"] = delta.cuda()
        cu = offsets(lengths) if lengths else None
        init = randn(g, len(lengths) if lengths else 1, 2, dk, dv)
        compare(*run(d, init, cu), d, init, cu)


@pytest.mark.parametrize("dk,dv", [(128, 64), (64, 128)])
def test_steps_of_float32s_range(dk, dv):
    """Steps whose log decay is beyond fp32: nothing is left of the state, and no
    product of what is left and what is not comes out as NaN."""
    d, g = scan_inputs(105, (1, 100), 2, 1, dk, dv, BF16, rate=1e8)
    d["dt_bias"] = None
    d["delta"] = (0.001 * torch.rand(1, 100, 2, generator=g) * 1e-8).cuda()
    d["delta"][:, 20] = 1e33
    for k in ("x", "b", "c"):
        d[k][:, 20] *= 1e-5  # the state after it: of order 1e23
    out, fin = run(d, randn(g, 1, 2, dk, dv), None)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(fin).all())


@pytest.mark.parametrize("dtype,dk,dv", SIZES)
@pytest.mark.parametrize("A_log", [88.0, 89.5, 300.0])
def test_rates_beyond_float32(dtype, dk, dv, A_log):
    """exp(A_log) beyond fp32's range: a step of zero leaves the state, any other resets it."""
    d, g = scan_inputs(106, (1, 90), 2, 1, dk, dv, dtype)
    d["A_log"].fill_(A_log)
    d["delta"][:, 30:50] = -700.0
    init = randn(g, 1, 2, dk, dv)
    r = compare(*run(d, init, None), d, init, None)
    state = init.clone()
    for t in (0, 30, 31):  # a reset and two steps of zero, token by token
        a = [d[k][:, t].contiguous() for k in ("x", "b", "c", "delta")]
        out = kda.kda_ssm_step(*a, d["A_log"], state, d["D"], d["dt_bias"])
        assert bool(torch.isfinite(out).all())
        if t == 0:
            after = state.clone()
            ref.assert_within(out, r["out"][:, 0], r["err_out"][:, 0], "step")
    assert torch.equal(state, after)
