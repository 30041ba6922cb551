"""Magnitudes that the layer operators' header names: the scan's operands far from
one, and the norm's values up to where fp32 holds their squares' sum."""
import pytest
import torch

from layer_inputs import gen, randn, scan_inputs
from test_gpu_layer_norm import check
from test_gpu_layer_scan import compare, run

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,dk,dv", [(BF16, 128, 64), (BF16, 64, 128), (BF16, 32, 32), (F32, 32, 32)])
@pytest.mark.parametrize("xs,bs,cs", [(2.0 ** -85, 2.0 ** 60, 1.0), (2.0 ** 100, 2.0 ** -90, 1.0), (2.0 ** -85, 1.0, 2.0 ** 80),
                                      (1.0, 2.0 ** 100, 2.0 ** -100)])
def test_scan_operands(dtype, dk, dv, xs, bs, cs):
    d, g = scan_inputs(7, (1, 100), 2, 1, dk, dv, dtype)
    for k, s in (("x", xs), ("b", bs), ("c", cs)):
        d[k] *= s  # (a power of two: exact)
    init = randn(g, 1, 2, dk, dv) * (xs * bs)
    compare(*run(d, init, None), d, init, None)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("width", [128, 100, 16384])
def test_norm_of_large_values(dtype, center, width):
    g = gen(width)
    x = (1e17 * (2 * torch.rand(3, 2 * width, generator=g) - 1)).to("cuda", dtype).clamp(-1e17, 1e17)
    check(x, 2, randn(g, width), None, None, "none", center=center)
