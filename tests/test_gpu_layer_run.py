"""The layer's operators together, as a layer calls them: convolution, scan and
gated norm over a prompt and then token by token; on another stream, several
calls in flight, and captured into a graph."""
import pytest
import torch

import gated_delta_rule_121_b200 as kda
from layer_inputs import gen, offsets, randn
from oracle import layer as ref
from parity import errors

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
H, G, DK, DV = 4, 1, 128, 64
C = H * DV + 2 * G * DK


def parameters(dtype, seed=1):
    g = gen(seed)
    p = dict(w=randn(g, C, 4, std=0.5), b=randn(g, C, std=0.1), A_log=randn(g, H) - 2, D=1 + randn(g, H, std=0.1),
             dt_bias=randn(g, H) - 2, norm=1 + randn(g, H * DV, std=0.1))
    return p, g


def layer(p, x, delta, z, conv_state, state, cu=None):
    """A prompt through the layer."""
    y, conv_state = kda.kda_conv_fwd(x, p["w"], p["b"], conv_state, cu)
    B, T = x.shape[:2]
    xs, b, c = y.split([H * DV, G * DK, G * DK], -1)
    o, state = kda.kda_ssm_fwd(xs.unflatten(-1, (H, DV)), b.unflatten(-1, (G, DK)), c.unflatten(-1, (G, DK)), delta,
                               p["A_log"], p["D"], p["dt_bias"], state, cu)
    return kda.kda_group_norm(o.view(B, T, H * DV), 1, p["norm"], None, z, activation=kda.KDA_ACT_SILU,
                              gate_first=True), conv_state, state


def layer_step(p, x, delta, z, conv_state, state, out=None):
    """One token through the layer, both states in place."""
    y = kda.kda_conv_step(x, p["w"], p["b"], conv_state)
    xs, b, c = y.split([H * DV, G * DK, G * DK], -1)
    o = kda.kda_ssm_step(xs.unflatten(-1, (H, DV)), b.unflatten(-1, (G, DK)), c.unflatten(-1, (G, DK)), delta, p["A_log"],
                         state, p["D"], p["dt_bias"])
    return kda.kda_group_norm(o.view(-1, H * DV), 1, p["norm"], None, z, activation=kda.KDA_ACT_SILU, gate_first=True,
                              out=out)


def reference(p, x, delta, z, cu=None):
    y, _, _ = ref.conv(x, p["w"], p["b"], None, cu, "silu")
    xs, b, c = y.split([H * DV, G * DK, G * DK], -1)
    r = ref.scan(xs.unflatten(-1, (H, DV)), b.unflatten(-1, (G, DK)), c.unflatten(-1, (G, DK)), delta, p["A_log"], p["D"],
                 p["dt_bias"], None, cu)
    o, _ = ref.norm(r["out"].flatten(-2), 1, p["norm"], None, z, 1e-5, False, "silu", True)
    return o, r["final"]


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompt_then_tokens(dtype):
    p, g = parameters(dtype)
    B, T, more = 2, 90, 5
    x, z = randn(g, B, T + more, C, dtype=dtype), randn(g, B, T + more, H * DV, dtype=dtype)
    delta = randn(g, B, T + more, H)
    o, f = reference(p, x, delta, z)
    cut = lambda v: v[:, :T].contiguous()  # noqa: E731
    out, conv_state, state = layer(p, cut(x), cut(delta), cut(z), None, None)
    outs = [out] + [layer_step(p, x[:, t], delta[:, t].contiguous(), z[:, t], conv_state, state)[:, None]
                    for t in range(T, T + more)]
    e = errors(torch.cat(outs, 1), o)
    # three roundings to the tensors' type in a row (convolution, scan, norm), each
    # within half a step of its values, and the scan's bf16 operands
    assert e["rel_fro"] <= (1e-2 if dtype == BF16 else 2e-6), e
    # the convolution's outputs reach the state rounded to their type, x and b both
    assert errors(state, f)["rel_fro"] <= (8e-3 if dtype == BF16 else 2e-6)


def test_packed_prompts_are_the_single_ones():
    p, g = parameters(BF16, 2)
    lens = [70, 0, 1, 129]
    x, z, delta = randn(g, 1, 200, C, dtype=BF16), randn(g, 1, 200, H * DV, dtype=BF16), randn(g, 1, 200, H)
    out, conv_state, state = layer(p, x, delta, z, None, None, offsets(lens))
    s = 0
    for i, n in enumerate(lens):
        if n:
            a = [v[:, s:s + n].contiguous() for v in (x, delta, z)]
            o1, c1, s1 = layer(p, *a, None, None)
            assert torch.equal(out[:, s:s + n], o1) and torch.equal(conv_state[i:i + 1], c1)
            assert torch.equal(state[i:i + 1], s1)
        s += n


def test_repeats_bit_for_bit_with_several_calls_in_flight():
    p, g = parameters(BF16, 3)
    a = [[randn(g, 2, 300, C, dtype=BF16), randn(g, 2, 300, H), randn(g, 2, 300, H * DV, dtype=BF16)] for _ in range(3)]
    want = [layer(p, *v, None, None) for v in a]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in a]
    got = []
    for v, s in zip(a, streams):
        with torch.cuda.stream(s):
            got.append(layer(p, *v, None, None))
    torch.cuda.synchronize()
    for x, y in zip(want, got):
        assert all(torch.equal(i, j) for i, j in zip(x, y))


def test_stream_argument():
    p, g = parameters(BF16, 4)
    x, delta = randn(g, 1, 100, C, dtype=BF16), randn(g, 1, 100, H)
    want, _ = kda.kda_conv_fwd(x, p["w"], p["b"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, _ = kda.kda_conv_fwd(x, p["w"], p["b"], stream=s)
    xs, b, c = out.split([H * DV, G * DK, G * DK], -1)
    args = (xs.unflatten(-1, (H, DV)), b.unflatten(-1, (G, DK)), c.unflatten(-1, (G, DK)), delta, p["A_log"], p["D"],
            p["dt_bias"])
    o, _ = kda.kda_ssm_fwd(*args, stream=s)
    n = kda.kda_group_norm(o, 1, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    assert torch.equal(o, kda.kda_ssm_fwd(*args)[0]) and torch.equal(n, kda.kda_group_norm(o, 1))


def test_captured_steps_and_prompts():
    """A graph of a token step (states advance with every replay), and two
    graphs of prompts that own their workspaces, replayed in turn."""
    p, g = parameters(BF16, 5)
    x, z, delta = randn(g, 3, C, dtype=BF16), randn(g, 3, H * DV, dtype=BF16), randn(g, 3, H)
    conv_state, state = randn(g, 3, 3, C, dtype=BF16), randn(g, 3, H, DK, DV)
    c0, s0 = conv_state.clone(), state.clone()
    want = [layer_step(p, x, delta, z, c0, s0) for _ in range(3)]
    out = torch.empty_like(z)
    layer_step(p, x, delta, z, conv_state.clone(), state.clone(), out)  # warm-up
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer_step(p, x, delta, z, conv_state, state, out)
    for w in want:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
    assert torch.equal(conv_state, c0) and torch.equal(state, s0)

    a = [[randn(g, 1, n, C, dtype=BF16), randn(g, 1, n, H), randn(g, 1, n, H * DV, dtype=BF16)] for n in (1500, 700)]
    want = [layer(p, *v, None, None) for v in a]
    graphs, got = [], []
    for v in a:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(layer(p, *v, None, None))
    for i in (0, 1, 0, 1, 1):
        for t in got[i]:
            t.fill_(3)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(want[i], got[i]))
