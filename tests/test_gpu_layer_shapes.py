"""The launch shapes that large calls of the layer operators take, at the least
data that reaches them: several runs of tokens per thread in the convolution,
several sequences per thread in its single-token form, four rows per team in
the norm, and the CUDA-core scan in pieces for bf16."""
import random

import pytest
import torch

import gated_delta_rule_121_b200 as kda
from layer_inputs import gen, offsets, randn, scan_inputs, sliced
from oracle import layer as ref
from test_gpu_layer_conv import check as check_conv
from test_gpu_layer_norm import check as check_norm
from test_gpu_layer_scan import compare, run

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32

# The convolution gives a thread 2, 4 or 8 runs (of 16 tokens, or 8 where it takes
# single channels) when 1184 blocks remain; a block of few channels has 8 threads
# along the tokens.  So 8 runs from 1184 * 8 * 8 runs of tokens on.
RUNS8 = 1184 * 8 * 8


def lengths_of(total, seed, longest):
    """Lengths around whole runs, empty and odd ones among them."""
    r, out = random.Random(seed), []
    while total > 0:
        n = min(r.choice([0, 1, 15, 16, 17, 32, 48, 64, 127, 128, 129, 256, r.randint(1, longest)]), total)
        out.append(n)
        total -= n
    return out


@pytest.mark.parametrize("C,K,dtype,runs", [(4, 4, BF16, 8), (4, 3, F32, 4), (3, 4, BF16, 8), (36, 2, BF16, 2), (5, 2, F32, 2)])
def test_convolution_with_several_runs_per_thread(C, K, dtype, runs):
    T = RUNS8 * (16 if C % 4 == 0 else 8) // 8 * runs + 5
    g = gen(C + K)
    x, w, b = sliced(g, (1, T), 0, (C,), 4, dtype), randn(g, C, K), randn(g, C)
    lens = lengths_of(T - 37, C, 3000)
    cu = offsets(lens) + 16  # rows of no sequence before and behind
    init = randn(g, len(lens), K - 1, C, dtype=dtype)
    out = torch.full((1, T, C), 7.0, dtype=dtype, device="cuda")
    check_conv(x, w, b, init, cu, "silu", out=out)
    assert bool((out[:, :16] == 7).all()) and bool((out[:, T - 21:] == 7).all())
    check_conv(x, w, None, None, None, "none")  # one sequence


@pytest.mark.parametrize("T", [16, 32, 64, 200])
def test_convolution_of_many_equal_lengths(T):
    """Every sequence's end at a run's end, or inside one; two runs per thread."""
    g = gen(T)
    B = RUNS8 * 16 // 4 // T + 1
    x, w, b = randn(g, B, T, 4, dtype=BF16), randn(g, 4, 4), randn(g, 4)
    check_conv(x, w, b, randn(g, B, 3, 4, dtype=BF16), None, "silu")


@pytest.mark.parametrize("C,K,dtype,more", [(4, 4, BF16, 3), (3, 3, F32, 0), (516, 2, BF16, 1), (4, 4, F32, 7)])
def test_steps_of_many_sequences(C, K, dtype, more):
    """Eight sequences per thread, the last thread with fewer."""
    g = gen(C + K)
    blocks = -(-C // (128 * (4 if C % 4 == 0 else 1)))
    N = 1184 * 16 // blocks + more
    x, w, b = randn(g, N, C, dtype=dtype), randn(g, C, K), randn(g, C)
    state = randn(g, N, K - 1, C, dtype=dtype)
    # the sequences side by side as channels of one token
    o, f, err = ref.conv(x.reshape(1, 1, N * C), w.repeat(N, 1), b.repeat(N), state.transpose(0, 1).reshape(1, K - 1, N * C),
                         None, "silu")
    out = kda.kda_conv_step(x, w, b, state)
    ref.assert_within(out, o.view(N, C), err.view(N, C), "conv step")
    assert torch.equal(state.cpu().double(), f.view(K - 1, N, C).transpose(0, 1))


# Four rows per team from 4736 blocks of 256 threads on, where a warp or less holds a
# group in one piece per thread.
@pytest.mark.parametrize("width,team,dtype", [(128, 16, BF16), (256, 32, BF16), (24, 4, BF16), (20, 32, F32), (15, 16, BF16)])
@pytest.mark.parametrize("tail", [0, 3])
def test_norm_with_four_rows_per_team(width, team, dtype, tail):
    groups = 12
    rows = (4736 * (256 // team) // groups + 4) // 4 * 4 + tail
    g = gen(width + tail)
    x, z = sliced(g, (rows,), 8, (groups * width,), 0, dtype), randn(g, rows, groups * width, dtype=dtype)
    w, b = 1 + randn(g, groups * width, std=0.2), randn(g, width)
    check_norm(x, groups, w, None, z, "sigmoid")
    check_norm(x, groups, None, b, z, "silu", center=True, gate_first=True)
    dense = x.contiguous()
    want = kda.kda_group_norm(dense, groups, None, b, None, center=True)
    assert torch.equal(kda.kda_group_norm(dense, groups, None, b, None, center=True, out=dense), want)


@pytest.mark.parametrize("dk,dv,H,G", [(32, 64, 2, 1), (16, 128, 1, 1), (128, 16, 3, 3), (32, 32, 4, 2)])
@pytest.mark.parametrize("lengths", [None, [1, 1700, 0, 64, 900], [3000]])
def test_bf16_scan_on_cuda_cores_in_pieces(dk, dv, H, G, lengths):
    T = sum(lengths) if lengths else 1500
    d, g = scan_inputs(dk + dv, (1 if lengths else 2, T), H, G, dk, dv, BF16, rate=0.05)
    cu = offsets(lengths) if lengths else None
    init = randn(g, len(lengths) if lengths else 2, H, dk, dv)
    out, fin = run(d, init, cu)
    compare(out, fin, d, init, cu)
    state = init.clone()
    again, _ = run(d, state, cu, final_state=state)
    assert torch.equal(again, out) and torch.equal(state, fin)


@pytest.mark.parametrize("T", [127, 128, 129, 255, 257, 513, 1025])
def test_bf16_scan_on_cuda_cores_around_the_pieces(T):
    d, g = scan_inputs(T, (1, T), 2, 1, 32, 16, BF16, rate=0.05)
    init = randn(g, 1, 2, 32, 16)
    compare(*run(d, init, None), d, init, None)
