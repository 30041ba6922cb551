"""GPU parity of the group norm with the fp64 reference, element by element
within the bound of its own rounding."""
import pytest
import torch

import gated_delta_rule_121_b200 as kda
from layer_inputs import gen, randn, sliced
from oracle import layer as ref

pytestmark = pytest.mark.gpu
ACT = {"none": kda.KDA_ACT_NONE, "silu": kda.KDA_ACT_SILU, "sigmoid": kda.KDA_ACT_SIGMOID}
BF16, F32 = torch.bfloat16, torch.float32


def check(x, groups, w, b, z, act, center=False, gate_first=False, eps=1e-5, **kw):
    out = kda.kda_group_norm(x, groups, w, b, z, eps, center, ACT[act], gate_first, **kw)
    torch.cuda.synchronize()
    y, err = ref.norm(x, groups, w, b, z, eps, center, act, gate_first)
    ref.assert_within(out, y, err, "norm")
    return out


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("groups,width", [(1, 1), (3, 7), (2, 16), (5, 33), (96, 128), (4, 64), (8, 24), (2, 450), (1, 1000),
                                          (3, 1024), (1, 2056), (1, 6144), (2, 5000), (1, 16384), (1, 9001)])
def test_widths(dtype, groups, width):
    g = gen(width)
    C, rows = groups * width, 5
    x, z = randn(g, rows, C, dtype=dtype), randn(g, rows, C, dtype=dtype)
    w, b = 1 + randn(g, C, std=0.2), randn(g, C)
    check(x, groups, w, None, z, "sigmoid")
    check(x, groups, w, b, z, "silu", center=True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("gate", ["none", "after", "first"])
@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("params", ["", "w", "b", "wb", "shared"])
def test_forms(dtype, gate, act, center, params):
    g = gen(11)
    x = sliced(g, (2, 9), 8, (4 * 32,), 8, dtype) + 3  # a mean of several deviations
    z = sliced(g, (2, 9), 0, (4 * 32,), 16, dtype) if gate != "none" else None
    n = 32 if params == "shared" else 128
    w = randn(g, n) if "w" in params or params == "shared" else None
    b = randn(g, n) if "b" in params or params == "shared" else None
    check(x, 4, w, b, z, act, center, gate == "first")


def test_unaligned_rows_and_strides():
    g = gen(12)
    x = sliced(g, (7,), 0, (3 * 40,), 5, BF16)      # row stride 125
    z = sliced(g, (7,), 8, (3 * 40,), 0, BF16)      # row stride 128
    check(x, 3, randn(g, 40), None, z, "silu")
    check(x, 3, None, None, None, "silu", center=True)


def test_in_place():
    g = gen(13)
    x, z = randn(g, 300, 256, dtype=BF16), randn(g, 300, 256, dtype=BF16)
    want = kda.kda_group_norm(x, 2, None, None, z)
    a, b = x.clone(), z.clone()
    assert torch.equal(kda.kda_group_norm(a, 2, None, None, z, out=a), want)
    assert torch.equal(kda.kda_group_norm(x, 2, None, None, b, out=b), want)


def test_rows_of_zeros_constants_and_large_values():
    g = gen(14)
    x = randn(g, 6, 128, dtype=F32)
    x[0] = 0
    x[1] = 5.0          # no variance
    x[2] = 1e15
    x[3] *= 1e-15
    for center in (False, True):
        out = kda.kda_group_norm(x, 1, None, None, None, 1e-5, center, kda.KDA_ACT_NONE)
        y, err = ref.norm(x, 1, None, None, None, 1e-5, center, "none", False)
        keep = [0, 1, 3, 4, 5] if center else [0, 1, 2, 3, 4, 5]  # centring 1e15 leaves only its rounding
        ref.assert_within(out[keep], y[keep], err[keep], "norm")
        assert bool(torch.isfinite(out).all())
    # a non-finite value spoils its own group and no other
    x[4, 3] = float("inf")
    out = kda.kda_group_norm(x, 2, None, None, None, activation=kda.KDA_ACT_NONE)
    assert not bool(torch.isfinite(out[4, :64]).all()) and bool(torch.isfinite(out[4, 64:]).all())
    assert bool(torch.isfinite(out[[0, 1, 3, 5]]).all())


def test_no_rows():
    assert kda.kda_group_norm(torch.empty(0, 3, 64, device="cuda", dtype=BF16), 2).shape == (0, 3, 64)


def test_offsets_beyond_32_bits():
    """Rows of a tensor of more than 2^31 elements: the bits of the dense rows' result."""
    wide = torch.empty(70000, 32768, dtype=BF16, device="cuda")
    x = randn(gen(15), 70000, 64, dtype=BF16)
    wide[:, -64:] = x
    assert torch.equal(kda.kda_group_norm(wide[:, -64:], 4), kda.kda_group_norm(x, 4))
    assert torch.equal(kda.kda_group_norm(x, 4, None, None, wide[:, -64:]), kda.kda_group_norm(x, 4, None, None, x))
