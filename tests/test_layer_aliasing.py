"""Outputs that share memory with inputs: the layer operators refuse them on the
host (fake pointers: the refused calls never touch the device), and take an
output that lies between the rows of a slice."""
import pytest
import torch

import gated_delta_rule_121_b200 as kda
from layer_inputs import gen, randn, scan_inputs
from test_layer_host import CONV, CONV_STEP, INVALID, NORM, SSM, SSM_STEP, call

BF16, F32 = torch.bfloat16, torch.float32
# The pointers are made up: where a device is, only real tensors are passed.
host = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up pointers")


# CONV: 8 rows of 64 bf16 at 256; CONV_STEP: rows of 64 fp32 at 256
@host
@pytest.mark.parametrize("kw", [dict(out=256), dict(out=256, ldx=128), dict(out=272), dict(out=1264), dict(x=1280 - 1008, out=1264),
                                dict(x=2298, out=1280), dict(ldx=1 << 40, out=256), dict(ldx=72, out=256 + 144 * 7 + 112)])
def test_convolution_refuses_shared_memory(kw):
    assert call("kda_conv_fwd", CONV, **kw) == INVALID


@host
@pytest.mark.parametrize("kw", [dict(out=256), dict(out=496), dict(B=4, ldx=128, out=256), dict(B=4, ldx=128, out=512),
                                dict(B=4, ldx=512, out=256 + 2048 + 240), dict(B=2, x=1280 + 508, out=1280)])
def test_convolution_step_refuses_shared_memory(kw):
    assert call("kda_conv_step", CONV_STEP, **kw) == INVALID


FAR = dict(b=1 << 30, c=1 << 31, x=1 << 32, ldx=512, ldb=256, ldc=256)


@host
@pytest.mark.parametrize("name,spec,rows", [("kda_ssm_fwd", SSM, 64), ("kda_ssm_step", SSM_STEP, 64)])
@pytest.mark.parametrize("what,ld,width", [("x", 512, 256), ("b", 256, 128), ("c", 256, 128)])
def test_scan_refuses_shared_memory(name, spec, rows, what, ld, width):
    a = dict(FAR, **({"B": rows} if name == "kda_ssm_step" else {"T": rows}))
    at, size = a[what], rows * 256 * 2  # bytes of out
    for out in (at, at + 16, at + (rows - 1) * ld * 2 + width * 2 - 16, at - size + 16, at + 5 * ld * 2 + width * 2 - 16):
        assert call(name, spec, **a, out=out) == INVALID, out - at


# NORM: 4 rows of 256 bf16
@host
@pytest.mark.parametrize("kw", [dict(out=272), dict(out=256, ldx=512), dict(x=1 << 20, out=528), dict(x=1 << 20, out=512, ldg=300),
                                dict(x=1 << 20, gate=1 << 21, ldg=2048, out=(1 << 21) + 3 * 4096 + 496),
                                dict(x=(1 << 20) + 2, gate=None, out=1 << 20)])
def test_norm_refuses_shared_memory(kw):
    assert call("kda_group_norm", NORM, **kw) == INVALID


@pytest.mark.gpu
def test_outputs_between_the_rows_of_a_slice():
    """Three rows 4 C apart and a dense output that fills the gap behind the first one."""
    g, C = gen(1), 64
    w = randn(g, C, 4)
    for dtype in (BF16, F32):
        wide = randn(g, 3, 4 * C, dtype=dtype)
        keep = wide.clone()
        x, out = wide[:, :C], wide[0, C:].view(3, C)
        state = randn(g, 3, 3, C, dtype=dtype)
        want = kda.kda_conv_step(x.contiguous(), w, None, state.clone())
        assert torch.equal(kda.kda_conv_step(x, w, None, state.clone(), out=out), want) and torch.equal(x, keep[:, :C])
        want = kda.kda_conv_fwd(x[None].contiguous(), w)[0]
        assert torch.equal(kda.kda_conv_fwd(x[None], w, out=out[None])[0], want) and torch.equal(x, keep[:, :C])
        want = kda.kda_group_norm(x.contiguous(), 2)
        assert torch.equal(kda.kda_group_norm(x, 2, out=out), want) and torch.equal(x, keep[:, :C])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_shared_memory_raises(dtype):
    g, C = gen(2), 64
    w, wide = randn(g, C, 4), randn(g, 1, 12, 2 * C, dtype=dtype)
    x, start = wide[..., :C], wide.view(-1)[:12 * C]
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        kda.kda_conv_fwd(x, w, out=start.view(1, 12, C))
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        kda.kda_conv_step(x[0], w, None, randn(g, 12, 3, C, dtype=dtype), out=start.view(12, C))
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        kda.kda_group_norm(x[0], 2, out=start.view(12, C))
    d, _ = scan_inputs(3, (1, 12), 2, 1, 64, 64, dtype, wide=False)
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        kda.kda_ssm_fwd(*(d[k] for k in ("x", "b", "c", "delta", "A_log")), out=d["x"])
    a = [d[k][0] for k in ("x", "b", "c", "delta")] + [d["A_log"]]
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        kda.kda_ssm_step(*a, randn(g, 12, 2, 64, 64), out=a[0])
