"""Host-side checks of the layer operators (no GPU): the C entry points and the
binding refuse bad arguments before they touch the device, and the fp64
reference agrees with independent forms of the same formulas."""
import ctypes

import pytest
import torch

import gated_delta_rule_121_b200 as kda
from gated_delta_rule_121_b200 import layer
from oracle import layer as ref
from layer_inputs import gen, offsets, randn, scan_inputs

OK, INVALID, UNSUPPORTED, WORKSPACE = kda.KDA_OK, kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_WORKSPACE


def call(name, spec, **kw):
    unknown = set(kw) - set(spec)
    assert not unknown, unknown
    return layer._fn(name)(*{**spec, **kw}.values())


CONV = dict(x=256, ldx=64, weight=512, bias=768, init=1024, out=1280, fin=1536, B=1, T=8, C=64, K=4, cu=None,
            act=kda.KDA_ACT_SILU, stream=None, dt=kda.KDA_BF16)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), INVALID), (dict(weight=None), INVALID), (dict(out=None), INVALID), (dict(x=257), INVALID),
    (dict(bias=772), INVALID), (dict(init=1026), INVALID), (dict(fin=1540), INVALID), (dict(cu=20), INVALID),
    (dict(ldx=63), INVALID), (dict(C=0), INVALID), (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(dt=5), INVALID),
    (dict(act=2), INVALID), (dict(act=9), INVALID), (dict(K=1), UNSUPPORTED), (dict(K=5), UNSUPPORTED),
    (dict(out=256), INVALID), (dict(C=1 << 21, ldx=1 << 21), UNSUPPORTED), (dict(B=4, T=1 << 30), UNSUPPORTED), (dict(T=1 << 33), UNSUPPORTED),
    (dict(B=0), OK),
])
def test_conv_fwd_refusals(kw, code):
    assert call("kda_conv_fwd", CONV, **kw) == code


CONV_STEP = dict(x=256, ldx=64, weight=512, bias=None, state=1024, out=1280, B=1, C=64, K=4, act=kda.KDA_ACT_NONE,
                 stream=None, dt=kda.KDA_F32)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), INVALID), (dict(state=None), INVALID), (dict(state=1032), INVALID), (dict(out=None), INVALID),
    (dict(ldx=8), INVALID), (dict(B=-2), INVALID), (dict(K=6), UNSUPPORTED), (dict(act=2), INVALID),
    (dict(B=0, x=None, out=None, state=None), OK),
])
def test_conv_step_refusals(kw, code):
    assert call("kda_conv_step", CONV_STEP, **kw) == code


SSM = dict(x=256, ldx=256, b=512, ldb=128, c=768, ldc=128, delta=1024, A_log=1280, D=1536, dt_bias=1792, init=2048,
           out=2304, fin=2560, B=1, T=64, H=2, G=1, dk=128, dv=128, cu=None, stream=None, dt=kda.KDA_BF16, ws=4096,
           wsb=1 << 30)


@pytest.mark.parametrize("kw,code", [
    *[(dict([(p, None)]), INVALID) for p in ("x", "b", "c", "delta", "A_log", "out")],
    (dict(delta=1026), INVALID),
    *[(dict([(p, 264)]), INVALID) for p in ("x", "b", "c", "A_log", "D", "dt_bias", "init", "out", "fin", "cu")],
    (dict(ldx=255), INVALID), (dict(ldx=260), INVALID), (dict(ldb=120), INVALID), (dict(ldc=132), INVALID),
    (dict(H=0), INVALID), (dict(G=0), INVALID), (dict(H=3, G=2, ldx=512), INVALID), (dict(B=-1), INVALID),
    (dict(T=-1), INVALID), (dict(dt=3), INVALID), (dict(dk=96), UNSUPPORTED), (dict(dv=256, ldx=512), UNSUPPORTED),
    (dict(B=3, T=1 << 30), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED), (dict(ws=None), WORKSPACE),
    (dict(ws=4100), WORKSPACE), (dict(wsb=16), WORKSPACE),
])
def test_ssm_fwd_refusals(kw, code):
    assert call("kda_ssm_fwd", SSM, **kw) == code


SSM_STEP = dict(x=256, ldx=256, b=512, ldb=128, c=768, ldc=128, delta=1024, A_log=1280, D=None, dt_bias=None,
                state=2048, out=2304, B=1, H=2, G=1, dk=128, dv=128, stream=None, dt=kda.KDA_BF16)


@pytest.mark.parametrize("kw,code", [
    (dict(state=None), INVALID), (dict(state=2056), INVALID), (dict(x=None), INVALID), (dict(ldb=8), INVALID),
    (dict(G=3), INVALID), (dict(dk=8), UNSUPPORTED), (dict(B=1 << 30, H=4, ldx=512), UNSUPPORTED), (dict(B=-1), INVALID),
    (dict(B=0, state=None, x=None, b=None, c=None, delta=None, out=None), OK),
])
def test_ssm_step_refusals(kw, code):
    assert call("kda_ssm_step", SSM_STEP, **kw) == code


NORM = dict(x=256, ldx=256, gate=512, ldg=256, weight=768, bias=1024, out=1280, rows=4, groups=2, width=128, shared=1,
            eps=1e-5, center=0, act=kda.KDA_ACT_SIGMOID, gate_first=0, stream=None, dt=kda.KDA_BF16)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(x=257), INVALID), (dict(gate=513), INVALID),
    (dict(weight=776), INVALID), (dict(bias=1028), INVALID), (dict(out=1284), INVALID), (dict(ldx=255), INVALID),
    (dict(ldg=100), INVALID), (dict(groups=0), INVALID), (dict(width=0), INVALID), (dict(rows=-1), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(act=3), INVALID), (dict(dt=2), INVALID),
    (dict(gate=None, gate_first=1), INVALID), (dict(out=256, ldx=512), INVALID), (dict(out=512, ldg=512), INVALID),
    (dict(width=16385, groups=1, ldx=16385, ldg=16385), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED),
    (dict(rows=0, x=None, out=None, gate=None), OK),
])
def test_group_norm_refusals(kw, code):
    assert call("kda_group_norm", NORM, **kw) == code


def test_workspace_size_covers_the_status_word():
    for packed in (False, True):
        assert kda.kda_ssm_fwd_workspace_size(2, 4096, 16, 1, 128, 128, packed) >= 256
    assert kda.kda_ssm_fwd_workspace_size(0, 0, 16, 1, 128, 128) >= 16


# ---- the binding's own checks (CPU tensors never reach the library)

def test_binding_refuses_cpu_tensors():
    x = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_conv_fwd(x, torch.zeros(8, 4))
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_group_norm(x, 2)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_conv_step(x[:, 0], torch.zeros(8, 4), None, torch.zeros(1, 3, 8))


@pytest.mark.parametrize("what,match", [
    (lambda x: dict(x=x.half()), "bf16 or fp32"),
    (lambda x: dict(x=x[0]), r"\[B, T, C\]"),
    (lambda x: dict(x=x.transpose(1, 2), weight=torch.zeros(6, 4)), "contiguous"),
    (lambda x: dict(x=x[:, :1].expand(2, 6, 8)), "overlapping"),
    (lambda x: dict(x=torch.zeros(2, 9, 8)[:, :6]), "equal distance"),
    (lambda x: dict(weight=torch.zeros(8, 4, dtype=torch.float64)), "weight"),
    (lambda x: dict(bias=torch.zeros(7)), "bias"),
    (lambda x: dict(init_state=torch.zeros(2, 4, 8)), "init_state"),
    (lambda x: dict(cu_seqlens=torch.zeros(3, dtype=torch.int32)), "batch dimension"),
    (lambda x: dict(x=x[:1], cu_seqlens=torch.zeros(3, dtype=torch.int64)), "int32"),
])
def test_conv_binding_refusals(what, match):
    a = dict(x=torch.zeros(2, 6, 8), weight=torch.zeros(8, 4))
    a.update(what(a["x"]))
    with pytest.raises(ValueError, match=match):
        kda.kda_conv_fwd(**a)


def test_row_strides():
    f = layer._rows
    f32 = torch.float32
    wide = torch.zeros(2, 3, 40)
    assert f("x", wide[..., 8:24], (2, 3, 16), 2, f32, -1) == 40
    assert f("x", wide[..., 8:24].unflatten(-1, (2, 8)), (2, 3, 2, 8), 2, f32, -1) == 40
    assert f("x", wide, (2, 3, 40), 2, f32, -1) == 40
    assert f("x", wide[:1, :1], (1, 1, 40), 2, f32, -1) == 40
    assert f("x", wide[:, :1, :16], (2, 1, 16), 2, f32, -1) == 120
    assert f("x", torch.zeros(0, 3, 40), (0, 3, 40), 2, f32, -1) == 40
    assert f("x", torch.zeros(2, 0, 40), (2, 0, 40), 2, f32, -1) == 40


# ---- the reference against other forms

def test_reference_conv_is_torch_conv1d():
    g = gen(1)
    x, w, b = (randn(g, *s, device="cpu").double() for s in ((2, 9, 5), (5, 4), (5,)))
    out, fin, _ = ref.conv(x, w, b, None, None, "silu")
    y = torch.nn.functional.conv1d(x.transpose(1, 2), w[:, None], b, padding=3, groups=5)[..., :9].transpose(1, 2)
    assert torch.allclose(out, torch.nn.functional.silu(y), atol=1e-12)
    assert torch.equal(fin, x[:, -3:])
    # a sequence continued from its state is the whole sequence
    a, f, _ = ref.conv(x[:, :2], w, b, None, None, "silu")
    c, f2, _ = ref.conv(x[:, 2:], w, b, f, None, "silu")
    assert torch.allclose(torch.cat([a, c], 1), out, atol=1e-12) and torch.equal(f2, fin)


def test_reference_norm_is_torch_group_norm():
    g = gen(2)
    x, w, b = (randn(g, *s, device="cpu").double() for s in ((6, 24), (24,), (24,)))
    out, _ = ref.norm(x, 4, w, b, None, 1e-5, True, "none", False)
    assert torch.allclose(out, torch.nn.functional.group_norm(x, 4, w, b, 1e-5), atol=1e-12)
    out, _ = ref.norm(x, 1, w, None, None, 1e-5, False, "silu", False)
    assert torch.allclose(out, torch.nn.functional.silu(torch.nn.functional.rms_norm(x, (24,), w, 1e-5)), atol=1e-12)


def test_reference_scan_is_its_matrix_form():
    """y = (L * C B^T) (D x) with L_ts = prod of the decays between, and the
    state chained over a split."""
    d, g = scan_inputs(3, (1, 12), 4, 2, 16, 8, torch.float64, wide=False, device="cpu")
    init = randn(g, 1, 4, 16, 8, device="cpu").double()
    r = ref.scan(d["x"], d["b"], d["c"], d["delta"], d["A_log"], d["D"], d["dt_bias"], init, None)
    step = torch.nn.functional.softplus(d["delta"].double() + d["dt_bias"].double())[0]
    cum = (-torch.exp(d["A_log"].double()) * step).cumsum(0)
    for h in range(4):
        B, C, X = d["b"][0, :, h // 2].double(), d["c"][0, :, h // 2].double(), d["x"][0, :, h].double()
        L = torch.exp(cum[:, None, h] - cum[None, :, h]).tril()
        y = (L * (C @ B.t()) * step[:, h]) @ X + torch.exp(cum[:, h, None]) * (C @ init[0, h]) + d["D"][h].double() * X
        assert torch.allclose(r["out"][0, :, h], y, atol=1e-10)
    cut = lambda a, b_: [d[k][:, a:b_] for k in ("x", "b", "c", "delta")]  # noqa: E731
    r1 = ref.scan(*cut(0, 5), d["A_log"], d["D"], d["dt_bias"], init, None)
    r2 = ref.scan(*cut(5, 12), d["A_log"], d["D"], d["dt_bias"], r1["final"], None)
    assert torch.allclose(r2["final"], r["final"], atol=1e-12)
    packed = ref.scan(d["x"], d["b"], d["c"], d["delta"], d["A_log"], d["D"], d["dt_bias"], None, offsets([5, 0, 7], "cpu"))
    alone = ref.scan(*cut(5, 12), d["A_log"], d["D"], d["dt_bias"], None, None)
    assert torch.allclose(packed["out"][0, 5:], alone["out"][0], atol=1e-12)
    assert float(packed["final"][1].abs().max()) == 0.0
