"""Binding of the operators around a recurrent layer (include/kda.h): the short
causal convolution, the selective state-space scan and the group norm, for
prompts and for single tokens.

Argument marshalling only.  Token tensors may be slices of a wider one (a fused
projection, a convolution's output): the last dimensions are dense, tokens lie
any distance apart.  A tensor that an entry point cannot read as it lies raises
ValueError; nothing is copied behind the caller's back.

Each call runs on the tensors' device, on ``stream`` (its current stream by
default); outputs are allocated for that stream.
"""
from __future__ import annotations

import ctypes

import torch

from . import _DT, _check, lib

KDA_ACT_NONE, KDA_ACT_SILU, KDA_ACT_SIGMOID = 0, 1, 2

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


class _On:
    """Makes the tensors' device current (and ``stream``, where one is given)
    around allocations and the launch; ``raw`` is the stream's handle."""
    __slots__ = ("raw", "_ctx")

    def __init__(self, t, stream):
        dev = t.device
        if dev.type != "cuda":
            raise ValueError("expected CUDA tensors")
        self._ctx = None
        if stream is not None:
            if stream.device != dev:
                raise ValueError(f"the stream belongs to {stream.device}, the tensors to {dev}")
            self._ctx = torch.cuda.stream(stream)
        elif torch.cuda.current_device() != dev.index:
            self._ctx = torch.cuda.device(dev)
        self.raw = (stream if stream is not None else torch.cuda.current_stream(dev)).cuda_stream

    def __enter__(self):
        if self._ctx is not None:
            self._ctx.__enter__()
        return self.raw

    def __exit__(self, *exc):
        if self._ctx is not None:
            self._ctx.__exit__(*exc)


def _p(t):
    return None if t is None else t.data_ptr()


def _dense(name, t, shape, dtype, dev):
    """``t`` as a dense tensor of this shape and type on this device (None passes)."""
    if t is None:
        return
    if t.dtype != dtype or t.device != dev or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} {list(shape)} on {dev}, "
                         f"got {t.dtype} {list(t.shape)} on {t.device}")


def _rows(name, t, shape, lead, dtype, dev):
    """Row stride of a token tensor: the ``lead`` leading dimensions are tokens
    an equal distance apart, the others are dense."""
    if t.dtype != dtype or t.device != dev or tuple(t.shape) != shape:
        raise ValueError(f"{name}: expected {dtype} {list(shape)} on {dev}, got {t.dtype} {list(t.shape)} on {t.device}")
    stride = t.stride()
    width = 1
    for i in range(len(shape) - 1, lead - 1, -1):
        if shape[i] > 1 and stride[i] != width:
            raise ValueError(f"{name}: each token's values must be contiguous")
        width *= shape[i]
    if t.numel() == 0:
        return width
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


def _sequences(B, cu_seqlens, dev):
    if cu_seqlens is None:
        return B
    if B != 1:
        raise ValueError("packed (cu_seqlens) inputs must have batch dimension 1")
    if (cu_seqlens.dtype != torch.int32 or cu_seqlens.device != dev or cu_seqlens.dim() != 1 or
            cu_seqlens.numel() < 1 or not cu_seqlens.is_contiguous()):
        raise ValueError(f"cu_seqlens: expected contiguous int32 [N + 1] on {dev}")
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
    init_state itself.  ``out`` must not overlap x."""
    dt, dev = _dtype(x), x.device
    if x.dim() != 3:
        raise ValueError("x must be [B, T, C]")
    B, T, C = x.shape
    if weight.dim() != 2:
        raise ValueError("weight must be [C, K]")
    K = weight.shape[1]
    N = _sequences(B, cu_seqlens, dev)
    ld = _rows("x", x, (B, T, C), 2, x.dtype, dev)
    _dense("weight", weight, (C, K), torch.float32, dev)
    _dense("bias", bias, (C,), torch.float32, dev)
    _dense("init_state", init_state, (N, K - 1, C), x.dtype, dev)
    _dense("out", out, (B, T, C), x.dtype, dev)
    _dense("final_state", final_state, (N, K - 1, C), x.dtype, dev)
    with _On(x, stream) as s:
        if out is None:
            out = torch.empty((B, T, C), dtype=x.dtype, device=dev)
        if final_state is None and output_final_state:
            final_state = torch.empty((N, K - 1, C), dtype=x.dtype, device=dev)
        _check(_fn("kda_conv_fwd")(_p(x), ld, _p(weight), _p(bias), _p(init_state), _p(out), _p(final_state), N, T, C,
                                   K, _p(cu_seqlens), activation, s, dt), "kda_conv_fwd")
    return out, final_state


def kda_conv_step(x, weight, bias, state, activation=KDA_ACT_SILU, out=None, stream=None):
    """One token of the convolution for each sequence: x [B,C], ``state``
    [B,K-1,C] is shifted in place.  Returns out [B,C]."""
    dt, dev = _dtype(x), x.device
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x must be [B, C] and weight [C, K]")
    B, C = x.shape
    K = weight.shape[1]
    ld = _rows("x", x, (B, C), 1, x.dtype, dev)
    _dense("weight", weight, (C, K), torch.float32, dev)
    _dense("bias", bias, (C,), torch.float32, dev)
    _dense("state", state, (B, K - 1, C), x.dtype, dev)
    _dense("out", out, (B, C), x.dtype, dev)
    with _On(x, stream) as s:
        if out is None:
            out = torch.empty((B, C), dtype=x.dtype, device=dev)
        _check(_fn("kda_conv_step")(_p(x), ld, _p(weight), _p(bias), _p(state), _p(out), B, C, K, activation, s, dt),
               "kda_conv_step")
    return out


def kda_ssm_fwd_workspace_size(B, T, H, G, dk, dv, packed=False, dtype=torch.bfloat16) -> int:
    """Workspace bytes of kda_ssm_fwd; with ``packed``, B is the number of
    sequences and T the total token count."""
    return int(_fn("kda_ssm_fwd_workspace_size")(B, T, H, G, dk, dv, int(bool(packed)), _DT[dtype]))


def _ssm_args(x, b, c, delta, A_log, D, dt_bias, lead):
    dt, dev = _dtype(x), x.device
    H, dv = x.shape[-2:]
    G, dk = b.shape[-2:]
    tokens = tuple(x.shape[:lead])
    lds = [_rows("x", x, tokens + (H, dv), lead, x.dtype, dev), _rows("b", b, tokens + (G, dk), lead, x.dtype, dev),
           _rows("c", c, tokens + (G, dk), lead, x.dtype, dev)]
    _dense("delta", delta, tokens + (H,), torch.float32, dev)
    _dense("A_log", A_log, (H,), torch.float32, dev)
    _dense("D", D, (H,), torch.float32, dev)
    _dense("dt_bias", dt_bias, (H,), torch.float32, dev)
    head = (_p(x), lds[0], _p(b), lds[1], _p(c), lds[2], _p(delta), _p(A_log), _p(D), _p(dt_bias))
    return dt, dev, H, G, dk, dv, head


def kda_ssm_fwd(x, b, c, delta, A_log, D=None, dt_bias=None, init_state=None, cu_seqlens=None, out=None,
                final_state=None, output_final_state=True, workspace=None, stream=None):
    """Selective state-space scan over whole sequences (include/kda.h,
    kda_ssm_fwd).  x [B,T,H,dv], b and c [B,T,G,dk] (tokens any distance apart),
    delta [B,T,H], A_log, D and dt_bias [H] fp32, states [N,H,dk,dv] fp32.
    Returns ``(out, final_state)``."""
    if x.dim() != 4 or b.dim() != 4 or c.dim() != 4:
        raise ValueError("x must be [B, T, H, dv], b and c [B, T, G, dk]")
    dt, dev, H, G, dk, dv, head = _ssm_args(x, b, c, delta, A_log, D, dt_bias, 2)
    B, T = x.shape[:2]
    N = _sequences(B, cu_seqlens, dev)
    _dense("init_state", init_state, (N, H, dk, dv), torch.float32, dev)
    _dense("out", out, (B, T, H, dv), x.dtype, dev)
    _dense("final_state", final_state, (N, H, dk, dv), torch.float32, dev)
    with _On(x, stream) as s:
        if out is None:
            out = torch.empty((B, T, H, dv), dtype=x.dtype, device=dev)
        if final_state is None and output_final_state:
            final_state = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
        if workspace is None:
            n = kda_ssm_fwd_workspace_size(N, T, H, G, dk, dv, cu_seqlens is not None, x.dtype)
            workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
        elif workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace: expected a contiguous tensor on {dev}")
        _check(_fn("kda_ssm_fwd")(*head, _p(init_state), _p(out), _p(final_state), N, T, H, G, dk, dv, _p(cu_seqlens),
                                  s, dt, _p(workspace), workspace.numel() * workspace.element_size()), "kda_ssm_fwd")
    return out, final_state


def kda_ssm_step(x, b, c, delta, A_log, state, D=None, dt_bias=None, out=None, stream=None):
    """One token of the scan for each sequence: x [B,H,dv], b and c [B,G,dk],
    delta [B,H]; ``state`` [B,H,dk,dv] fp32 is updated in place.  Returns out
    [B,H,dv]."""
    if x.dim() != 3 or b.dim() != 3 or c.dim() != 3:
        raise ValueError("x must be [B, H, dv], b and c [B, G, dk]")
    dt, dev, H, G, dk, dv, head = _ssm_args(x, b, c, delta, A_log, D, dt_bias, 1)
    B = x.shape[0]
    _dense("state", state, (B, H, dk, dv), torch.float32, dev)
    _dense("out", out, (B, H, dv), x.dtype, dev)
    with _On(x, stream) as s:
        if out is None:
            out = torch.empty((B, H, dv), dtype=x.dtype, device=dev)
        _check(_fn("kda_ssm_step")(*head, _p(state), _p(out), B, H, G, dk, dv, s, dt), "kda_ssm_step")
    return out


def kda_group_norm(x, groups, weight=None, bias=None, gate=None, eps=1e-5, center=False, activation=KDA_ACT_SIGMOID,
                   gate_first=False, out=None, stream=None):
    """Group norm over the last dimension's channels with an activation
    (include/kda.h, kda_group_norm).  x [..., C] and gate like x (rows any
    distance apart), weight and bias fp32 [C], or [C / groups] shared by all
    groups.  Returns ``out`` like x, dense; it may be x or gate themselves."""
    dt, dev = _dtype(x), x.device
    if x.dim() < 1 or groups <= 0 or x.shape[-1] % groups or x.shape[-1] == 0:
        raise ValueError("the channels must divide into the groups")
    shape, lead, C = tuple(x.shape), x.dim() - 1, x.shape[-1]
    width = C // groups
    ldx = _rows("x", x, shape, lead, x.dtype, dev)
    ldg = C if gate is None else _rows("gate", gate, shape, lead, x.dtype, dev)
    shared = any(p is not None and tuple(p.shape) == (width,) for p in (weight, bias))
    for name, p in (("weight", weight), ("bias", bias)):
        _dense(name, p, (width,) if shared else (C,), torch.float32, dev)
    _dense("out", out, shape, x.dtype, dev)
    with _On(x, stream) as s:
        if out is None:
            out = torch.empty(shape, dtype=x.dtype, device=dev)
        _check(_fn("kda_group_norm")(_p(x), ldx, _p(gate), ldg, _p(weight), _p(bias), _p(out), x.numel() // C, groups,
                                     width, int(shared), eps, int(bool(center)), activation, int(bool(gate_first)), s,
                                     dt), "kda_group_norm")
    return out
