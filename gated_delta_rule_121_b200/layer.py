"""Binding of the operators around a recurrent layer (include/kda.h): the short
causal convolution, the selective state-space scan and the group norm, for
prompts and for single tokens.

Argument marshalling only.  Token tensors may be slices of a wider one (a fused
projection, a convolution's output): the last dimensions are dense, tokens lie
any distance apart.  ``out`` shares no memory with them (kda_group_norm's may be x
or gate).  A tensor that an entry point cannot read as it lies raises
ValueError; nothing is copied behind the caller's back.

Each call runs on the tensors' device, on ``stream`` (its current stream by
default); outputs are allocated for that stream.  The checks are written for
decode steps, where a call's host time is what a user waits for.
"""
from __future__ import annotations

import ctypes

import torch

from . import _DT, _check, lib

KDA_ACT_NONE, KDA_ACT_SILU, KDA_ACT_SIGMOID = 0, 1, 2

_F32 = torch.float32
_vp, _int, _i64, _f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
_row = [_vp, _i64]  # a strided token tensor: pointer and row stride
_SIGNATURES = {
    "kda_conv_fwd": _row + [_vp] * 5 + [_int, _i64, _int, _int, _vp, _int, _vp, _int],
    "kda_conv_step": _row + [_vp] * 4 + [_int] * 4 + [_vp, _int],
    "kda_ssm_fwd": _row * 3 + [_vp] * 7 + [_int, _i64] + [_int] * 4 + [_vp, _vp, _int, _vp, ctypes.c_size_t],
    "kda_ssm_step": _row * 3 + [_vp] * 6 + [_int] * 5 + [_vp, _int],
    "kda_group_norm": _row * 2 + [_vp] * 3 + [_i64, _int, _int, _int, _f32, _int, _int, _int, _vp, _int],
    "kda_ssm_fwd_workspace_size": [_int, _i64] + [_int] * 6,
}
_fns = {}


def _fn(name):
    f = _fns.get(name)
    if f is None:
        f = getattr(lib(), name)
        f.argtypes = _SIGNATURES[name]
        f.restype = ctypes.c_size_t if name.endswith("_size") else ctypes.c_int
        _fns[name] = f
    return f


def _elsewhere(t, stream):
    """The context in which a call runs, None when that is the current one
    already: the tensors' device, and ``stream`` where one is given."""
    dev = t.device
    if dev.type != "cuda":
        raise ValueError("expected CUDA tensors")
    if stream is not None:
        if stream.device != dev:
            raise ValueError(f"the stream belongs to {stream.device}, the tensors to {dev}")
        return torch.cuda.stream(stream)
    return None if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def _raw_stream(index):
    """Handle of a device's current stream (torch.cuda.current_stream(index).cuda_stream, without the object)."""
    return torch._C._cuda_getCurrentRawStream(index)


def _p(t):
    return None if t is None else t.data_ptr()


def _bad(name, t, shape, dtype, how=""):
    return ValueError(f"{name}: expected {how}{dtype} {list(shape)} on the same device, got {t.dtype} {list(t.shape)} on {t.device}")


def _dense(name, t, shape, dtype, index):
    """``t`` is a dense tensor of this shape and type on this device (None passes)."""
    if t is not None and (t.shape != shape or t.dtype != dtype or t.get_device() != index or not t.is_contiguous()):
        raise _bad(name, t, shape, dtype, "contiguous ")


def _rows(name, t, shape, lead, dtype, index):
    """Row stride of a token tensor: the ``lead`` leading dimensions are tokens
    an equal distance apart, the others are dense."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != index:
        raise _bad(name, t, shape, dtype)
    if t.is_contiguous():
        width = 1
        for n in shape[lead:]:
            width *= n
        return width
    stride = t.stride()
    width = 1
    for i in range(len(shape) - 1, lead - 1, -1):
        if shape[i] > 1 and stride[i] != width:
            raise ValueError(f"{name}: each token's values must be contiguous")
        width *= shape[i]
    # the distance between tokens comes from the innermost leading dimension longer than one
    ld, span = None, 1
    for i in range(lead - 1, -1, -1):
        if shape[i] > 1:
            if ld is None:
                if stride[i] % span or stride[i] < width * span:
                    raise ValueError(f"{name}: overlapping or unevenly spaced tokens")
                ld = stride[i] // span
            elif stride[i] != ld * span:
                raise ValueError(f"{name}: tokens must lie an equal distance apart over the batch")
        span *= shape[i]
    return width if ld is None else ld


def _sequences(B, cu_seqlens, index):
    if cu_seqlens is None:
        return B
    if B != 1:
        raise ValueError("packed (cu_seqlens) inputs must have batch dimension 1")
    if (cu_seqlens.dtype != torch.int32 or cu_seqlens.get_device() != index or cu_seqlens.dim() != 1 or
            cu_seqlens.numel() < 1 or not cu_seqlens.is_contiguous()):
        raise ValueError("cu_seqlens: expected contiguous int32 [N + 1] on the same device")
    return cu_seqlens.numel() - 1


def _dtype(t, name="x"):
    dt = _DT.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name}: expected bf16 or fp32, got {t.dtype}")
    return dt


def kda_conv_fwd(x, weight, bias=None, init_state=None, cu_seqlens=None, activation=KDA_ACT_SILU, out=None,
                 final_state=None, output_final_state=True, stream=None):
    """Short depthwise causal convolution over whole sequences (include/kda.h,
    kda_conv_fwd).  x [B,T,C] (tokens any distance apart), weight [C,K] and bias
    [C] fp32, init_state [N,K-1,C] in x's type.  Returns ``(out, final_state)``;
    final_state [N,K-1,C] holds the last K-1 inputs of each sequence and may be
    init_state itself."""
    dt, dtype, dev = _dtype(x), x.dtype, x.get_device()
    if x.dim() != 3:
        raise ValueError("x must be [B, T, C]")
    B, T, C = x.shape
    if weight.dim() != 2:
        raise ValueError("weight must be [C, K]")
    K = weight.shape[1]
    N = _sequences(B, cu_seqlens, dev)
    ld = _rows("x", x, (B, T, C), 2, dtype, dev)
    _dense("weight", weight, (C, K), _F32, dev)
    _dense("bias", bias, (C,), _F32, dev)
    _dense("init_state", init_state, (N, K - 1, C), dtype, dev)
    _dense("out", out, (B, T, C), dtype, dev)
    _dense("final_state", final_state, (N, K - 1, C), dtype, dev)
    where = _elsewhere(x, stream)
    if where is not None:
        with where:
            return kda_conv_fwd(x, weight, bias, init_state, cu_seqlens, activation, out, final_state, output_final_state)
    if out is None:
        out = x.new_empty((B, T, C))
    if final_state is None and output_final_state:
        final_state = x.new_empty((N, K - 1, C))
    code = _fn("kda_conv_fwd")(x.data_ptr(), ld, weight.data_ptr(), _p(bias), _p(init_state), out.data_ptr(), _p(final_state),
                               N, T, C, K, _p(cu_seqlens), activation, _raw_stream(dev), dt)
    if code:
        _check(code, "kda_conv_fwd")
    return out, final_state


def kda_conv_step(x, weight, bias, state, activation=KDA_ACT_SILU, out=None, stream=None):
    """One token of the convolution for each sequence: x [B,C], ``state``
    [B,K-1,C] is shifted in place.  Returns out [B,C]."""
    dt, dtype, dev = _dtype(x), x.dtype, x.get_device()
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x must be [B, C] and weight [C, K]")
    B, C = x.shape
    K = weight.shape[1]
    ld = _rows("x", x, (B, C), 1, dtype, dev)
    _dense("weight", weight, (C, K), _F32, dev)
    _dense("bias", bias, (C,), _F32, dev)
    _dense("state", state, (B, K - 1, C), dtype, dev)
    _dense("out", out, (B, C), dtype, dev)
    where = _elsewhere(x, stream)
    if where is not None:
        with where:
            return kda_conv_step(x, weight, bias, state, activation, out)
    if out is None:
        out = x.new_empty((B, C))
    code = _fn("kda_conv_step")(x.data_ptr(), ld, weight.data_ptr(), _p(bias), state.data_ptr(), out.data_ptr(), B, C, K,
                                activation, _raw_stream(dev), dt)
    if code:
        _check(code, "kda_conv_step")
    return out


def kda_ssm_fwd_workspace_size(B, T, H, G, dk, dv, packed=False, dtype=torch.bfloat16) -> int:
    """Workspace bytes of kda_ssm_fwd; with ``packed``, B is the number of
    sequences and T the total token count."""
    return int(_fn("kda_ssm_fwd_workspace_size")(B, T, H, G, dk, dv, int(bool(packed)), _DT[dtype]))


def _ssm_args(x, b, c, delta, A_log, D, dt_bias, lead):
    dt, dtype, dev = _dtype(x), x.dtype, x.get_device()
    shape = x.shape
    tokens, H, dv = shape[:lead], shape[-2], shape[-1]
    G, dk = b.shape[-2], b.shape[-1]
    ldx = _rows("x", x, shape, lead, dtype, dev)
    bc = tokens + (G, dk)
    ldb, ldc = _rows("b", b, bc, lead, dtype, dev), _rows("c", c, bc, lead, dtype, dev)
    _dense("delta", delta, tokens + (H,), _F32, dev)
    _dense("A_log", A_log, (H,), _F32, dev)
    _dense("D", D, (H,), _F32, dev)
    _dense("dt_bias", dt_bias, (H,), _F32, dev)
    head = (x.data_ptr(), ldx, b.data_ptr(), ldb, c.data_ptr(), ldc, delta.data_ptr(), A_log.data_ptr(), _p(D), _p(dt_bias))
    return dt, dev, H, G, dk, dv, head


def kda_ssm_fwd(x, b, c, delta, A_log, D=None, dt_bias=None, init_state=None, cu_seqlens=None, out=None,
                final_state=None, output_final_state=True, workspace=None, stream=None):
    """Selective state-space scan over whole sequences (include/kda.h,
    kda_ssm_fwd).  x [B,T,H,dv], b and c [B,T,G,dk] (tokens any distance apart),
    delta [B,T,H], A_log, D and dt_bias [H] fp32, states [N,H,dk,dv] fp32.
    Returns ``(out, final_state)``.  With a ``workspace`` of one's own,
    kda_workspace_status tells afterwards whether a device-side wait gave up."""
    if x.dim() != 4 or b.dim() != 4 or c.dim() != 4:
        raise ValueError("x must be [B, T, H, dv], b and c [B, T, G, dk]")
    dt, dev, H, G, dk, dv, head = _ssm_args(x, b, c, delta, A_log, D, dt_bias, 2)
    B, T = x.shape[0], x.shape[1]
    N = _sequences(B, cu_seqlens, dev)
    _dense("init_state", init_state, (N, H, dk, dv), _F32, dev)
    _dense("out", out, (B, T, H, dv), x.dtype, dev)
    _dense("final_state", final_state, (N, H, dk, dv), _F32, dev)
    where = _elsewhere(x, stream)
    if where is not None:
        with where:
            return kda_ssm_fwd(x, b, c, delta, A_log, D, dt_bias, init_state, cu_seqlens, out, final_state,
                               output_final_state, workspace)
    if out is None:
        out = x.new_empty((B, T, H, dv))
    if final_state is None and output_final_state:
        final_state = A_log.new_empty((N, H, dk, dv))
    if workspace is None:
        n = _fn("kda_ssm_fwd_workspace_size")(N, T, H, G, dk, dv, int(cu_seqlens is not None), dt)
        workspace = torch.empty(n, dtype=torch.uint8, device=x.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace: expected a contiguous tensor on the same device")
    code = _fn("kda_ssm_fwd")(*head, _p(init_state), out.data_ptr(), _p(final_state), N, T, H, G, dk, dv, _p(cu_seqlens),
                              _raw_stream(dev), dt, workspace.data_ptr(), workspace.numel() * workspace.element_size())
    if code:
        _check(code, "kda_ssm_fwd")
    return out, final_state


def kda_ssm_step(x, b, c, delta, A_log, state, D=None, dt_bias=None, out=None, stream=None):
    """One token of the scan for each sequence: x [B,H,dv], b and c [B,G,dk],
    delta [B,H]; ``state`` [B,H,dk,dv] fp32 is updated in place.  Returns out
    [B,H,dv]."""
    if x.dim() != 3 or b.dim() != 3 or c.dim() != 3:
        raise ValueError("x must be [B, H, dv], b and c [B, G, dk]")
    dt, dev, H, G, dk, dv, head = _ssm_args(x, b, c, delta, A_log, D, dt_bias, 1)
    B = x.shape[0]
    _dense("state", state, (B, H, dk, dv), _F32, dev)
    _dense("out", out, (B, H, dv), x.dtype, dev)
    where = _elsewhere(x, stream)
    if where is not None:
        with where:
            return kda_ssm_step(x, b, c, delta, A_log, state, D, dt_bias, out)
    if out is None:
        out = x.new_empty((B, H, dv))
    code = _fn("kda_ssm_step")(*head, state.data_ptr(), out.data_ptr(), B, H, G, dk, dv, _raw_stream(dev), dt)
    if code:
        _check(code, "kda_ssm_step")
    return out


def kda_group_norm(x, groups, weight=None, bias=None, gate=None, eps=1e-5, center=False, activation=KDA_ACT_SIGMOID,
                   gate_first=False, out=None, stream=None):
    """Group norm over the last dimension's channels with an activation
    (include/kda.h, kda_group_norm).  x [..., C] and gate like x (rows any
    distance apart), weight and bias fp32 [C], or [C / groups] shared by all
    groups.  Returns ``out`` like x, dense; it may be x or gate themselves."""
    dt, dtype, dev = _dtype(x), x.dtype, x.get_device()
    shape = x.shape
    lead = len(shape) - 1
    if lead < 0 or groups <= 0 or shape[-1] % groups or shape[-1] == 0:
        raise ValueError("the channels must divide into the groups")
    C = shape[-1]
    width = C // groups
    ldx = _rows("x", x, shape, lead, dtype, dev)
    ldg = C if gate is None else _rows("gate", gate, shape, lead, dtype, dev)
    shared = (weight is not None and weight.shape == (width,)) or (bias is not None and bias.shape == (width,))
    _dense("weight", weight, (width,) if shared else (C,), _F32, dev)
    _dense("bias", bias, (width,) if shared else (C,), _F32, dev)
    _dense("out", out, shape, dtype, dev)
    where = _elsewhere(x, stream)
    if where is not None:
        with where:
            return kda_group_norm(x, groups, weight, bias, gate, eps, center, activation, gate_first, out)
    if out is None:
        out = x.new_empty(shape)
    code = _fn("kda_group_norm")(x.data_ptr(), ldx, _p(gate), ldg, _p(weight), _p(bias), out.data_ptr(), x.numel() // C,
                                 groups, width, int(shared), eps, int(bool(center)), activation, int(bool(gate_first)),
                                 _raw_stream(dev), dt)
    if code:
        _check(code, "kda_group_norm")
    return out
