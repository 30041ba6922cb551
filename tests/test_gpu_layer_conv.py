"""GPU parity of the short causal convolution (prompts and single tokens) with
the fp64 reference, element by element within the bound of its own terms."""
import pytest
import torch

import gated_delta_rule_121_b200 as kda
from layer_inputs import gen, offsets, randn, sliced
from oracle import layer as ref

pytestmark = pytest.mark.gpu
ACT = {"none": kda.KDA_ACT_NONE, "silu": kda.KDA_ACT_SILU}
BF16, F32 = torch.bfloat16, torch.float32


def check(x, w, b, init, cu, act, **kw):
    out, fin = kda.kda_conv_fwd(x, w, b, init, cu, activation=ACT[act], **kw)
    torch.cuda.synchronize()
    o, f, err = ref.conv(x, w, b, init, cu, act)
    own = ~torch.isnan(o)
    ref.assert_within(out.cpu()[own], o[own], err[own], "conv out")
    assert torch.equal(fin.cpu().double(), f), "conv state"
    return out, fin


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("C,pad", [(64, 0), (64, 8), (8, 0), (33, 0), (1, 0), (264, 4), (40, 3)])
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 67])
def test_batched(dtype, K, C, pad, T):
    g = gen(100 * K + C + T)
    x = sliced(g, (2, T), 16 if pad % 8 == 0 and pad else 0, (C,), pad, dtype)
    w, b = randn(g, C, K), randn(g, C)
    check(x, w, b, randn(g, 2, K - 1, C, dtype=dtype), None, "silu")
    check(x, w, None, None, None, "none")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("C", [72, 19])
@pytest.mark.parametrize("lengths", [[5], [0, 3, 0, 0, 1, 2, 70], [1] * 20, [64, 64], [7, 9, 8, 130, 1, 0], [200, 0]])
def test_packed(dtype, C, lengths):
    g = gen(7 + C + len(lengths))
    T = sum(lengths)
    x, w, b = randn(g, 1, T, C, dtype=dtype), randn(g, C, 4), randn(g, C)
    cu = offsets(lengths)
    check(x, w, b, randn(g, len(lengths), 3, C, dtype=dtype), cu, "silu")
    check(x, w, b, None, cu, "silu")


@pytest.mark.parametrize("C", [72, 19])
def test_state_in_place_and_rows_outside_the_sequences(C):
    """The final state over the initial one; a packed batch that leaves rows
    before and behind its sequences, which hold NaN: they are neither read for
    a sequence nor written."""
    g = gen(3)
    x, w, b = randn(g, 1, 60, C, dtype=BF16), randn(g, C, 4), randn(g, C)
    cu = torch.tensor([5, 6, 6, 30, 47], dtype=torch.int32, device="cuda")
    x[:, :5] = float("nan")
    x[:, 47:] = float("nan")
    init = randn(g, 4, 3, C, dtype=BF16)
    out0, fin0 = kda.kda_conv_fwd(x, w, b, init, cu)
    out = torch.full_like(x, 7.0)
    state = init.clone()
    kda.kda_conv_fwd(x, w, b, state, cu, out=out, final_state=state)
    torch.cuda.synchronize()
    assert torch.equal(state, fin0) and torch.equal(out[:, 5:47], out0[:, 5:47])
    assert bool((out[:, :5] == 7).all()) and bool((out[:, 47:] == 7).all())
    o, f, err = ref.conv(x, w, b, init, cu, "silu")
    ref.assert_within(out[:, 5:47], o[:, 5:47], err[:, 5:47], "conv out")
    assert torch.equal(state.cpu().double(), f)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("B,C,pad", [(1, 64, 0), (3, 1032, 24), (37, 33, 0), (5, 1, 0), (130, 16, 0)])
def test_steps_continue_a_prompt(dtype, K, B, C, pad):
    """A prompt, then single tokens from its state: the whole sequence's outputs."""
    g = gen(K + C)
    T, more = 5, 6
    x = sliced(g, (B, T + more), 0, (C,), pad, dtype)
    w, b = randn(g, C, K), randn(g, C)
    o, f, err = ref.conv(x, w, b, None, None, "silu")
    _, state = kda.kda_conv_fwd(x[:, :T].contiguous(), w, b)
    for t in range(T, T + more):
        out = kda.kda_conv_step(x[:, t], w, b, state)
        ref.assert_within(out, o[:, t], err[:, t], f"conv step {t}")
    torch.cuda.synchronize()
    assert torch.equal(state.cpu().double(), f)


def test_large_values_and_no_tokens():
    g = gen(5)
    x = randn(g, 1, 40, 24, dtype=BF16, std=1e4)
    check(x, randn(g, 24, 4), randn(g, 24), None, None, "silu")
    out, fin = kda.kda_conv_fwd(x[:, :0], randn(g, 24, 4), None, None, None)
    assert out.shape == (1, 0, 24) and not bool(fin.any())
    init = randn(g, 1, 3, 24, dtype=BF16)
    assert torch.equal(kda.kda_conv_fwd(x[:, :0], randn(g, 24, 4), None, init)[1], init)
    assert kda.kda_conv_step(x[0, :0], randn(g, 24, 4), None, x.new_zeros(0, 3, 24)).shape == (0, 24)


def test_offsets_beyond_32_bits():
    """Rows of a tensor of more than 2^31 elements: the bits of the dense rows' result."""
    wide = torch.empty(1, 70000, 32768, dtype=BF16, device="cuda")
    g = gen(9)
    for C in (64, 63):
        x, w = randn(g, 1, 70000, C, dtype=BF16), randn(g, C, 4)
        wide[..., -C:] = x
        for a, b in zip(kda.kda_conv_fwd(wide[..., -C:], w), kda.kda_conv_fwd(x, w)):
            assert torch.equal(a, b)


def test_long_rows():
    """Many runs per sequence."""
    g = gen(6)
    x = randn(g, 1, 3001, 520, dtype=BF16)
    check(x, randn(g, 520, 4), randn(g, 520), None, offsets([1000, 3, 1998]), "silu")
