"""fp64 reference of the operators around a recurrent layer (short convolution,
selective scan, group norm), on the CPU.

TEST INFRASTRUCTURE ONLY, like the rest of this package: nothing here imports
the library.  Written from the definitions, token by token where the operator
is a recurrence.  ``scan`` also runs the recurrence of a bound on the rounding
error of an fp32 evaluation, so that tests hold every element to what its own
terms allow.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24  # half an fp32 step, relative
HALF_STEP = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def _d(t):
    return None if t is None else t.detach().cpu().double()


def bounds_of(B, T, cu=None):
    """[(start, end)] of every sequence in the flattened token axis."""
    if cu is None:
        return [(i * T, (i + 1) * T) for i in range(B)]
    c = cu.cpu().tolist()
    return list(zip(c[:-1], c[1:]))


def _act(v, act):
    if act == "none":
        return v
    s = torch.where(v >= 0, 1 / (1 + torch.exp(-v.abs())), torch.exp(-v.abs()) / (1 + torch.exp(-v.abs())))
    return v * s if act == "silu" else s


def act_error(v, act):
    """Relative error of an fp32 activation at v: the exponential is within
    2 + 1.2 |v| steps, the reciprocal and its argument within 3, one product (a step is 2 U)."""
    return 0.0 * v if act == "none" else 2 * U * (6 + 1.2 * v.abs().clamp(max=90))


def conv(x, weight, bias, init, cu, act):
    """(out, final_state, bound): bound on |result - out| before the output's
    own rounding.  x [B,T,C]; rows of no sequence come out as NaN."""
    x, w, b, init = _d(x), _d(weight), _d(bias), _d(init)
    B, T, C = x.shape
    K = w.shape[1]
    flat = x.reshape(B * T, C)
    out = torch.full_like(flat, float("nan"))
    err = torch.zeros_like(flat)
    fins = []
    for n, (s, e) in enumerate(bounds_of(B, T, cu)):
        head = init[n] if init is not None else torch.zeros(K - 1, C, dtype=torch.float64)
        rows = torch.cat([head, flat[s:e]])
        acc = torch.zeros(e - s, C, dtype=torch.float64)
        mag = torch.zeros_like(acc)
        if b is not None:
            acc, mag = acc + b, mag + b.abs()
        for j in range(K):
            acc = acc + rows[j:j + e - s] * w[:, j]
            mag = mag + (rows[j:j + e - s] * w[:, j]).abs()
        y = _act(acc, act)
        out[s:e] = y
        # K fused multiply-adds (one rounding each, of partial sums up to mag);
        # the activation's slope is at most 1.1
        err[s:e] = 1.1 * K * U * mag + act_error(acc, act) * y.abs()
        fins.append(rows[rows.shape[0] - (K - 1):])
    fin = torch.stack(fins) if fins else torch.zeros(0, K - 1, C, dtype=torch.float64)
    return out.view(B, T, C), fin, err.view(B, T, C)


def norm(x, groups, weight, bias, gate, eps, center, act, gate_first):
    """(out, bound)."""
    x, w, b, z = _d(x), _d(weight), _d(bias), _d(gate)
    shape = x.shape
    C = shape[-1]
    width = C // groups
    g, ge = (_act(z, act), act_error(z, act)) if z is not None else (None, None)
    u = x * g if gate_first else x
    # relative error of u, then of the centred value against the group's largest
    eu = (ge + U) * u.abs() if gate_first else 0.0 * u
    u = u.reshape(-1, groups, width)
    eu = eu.reshape(u.shape)
    if center:
        mu = u.mean(-1, keepdim=True)
        # the mean: width sums of magnitudes |u|, a product; then a subtraction
        eu = eu + eu.mean(-1, keepdim=True) + (width + 2) * U * u.abs().mean(-1, keepdim=True) + U * (u - mu).abs()
        u = u - mu
    ms = (u * u).mean(-1, keepdim=True)
    r = 1 / torch.sqrt(ms + eps)
    # relative error of r: half that of the mean square (width sums, twice the values' errors), 2 steps of its own
    er = 0.5 * ((width + 3) * U + 2 * (eu * u.abs()).mean(-1, keepdim=True) / (ms + eps)) + 4 * U
    v = u * r
    ev = eu * r + v.abs() * (er + U)
    per = lambda p: p if p.numel() == C else p.repeat(groups)  # noqa: E731
    if w is not None:
        ww = per(w).view(groups, width)
        ev = ev * ww.abs() + U * (v * ww).abs()
        v = v * ww
    if b is not None:
        v = v + per(b).view(groups, width)
        ev = ev + U * v.abs()
    v, ev = v.reshape(shape), ev.reshape(shape)
    if z is None:
        y = _act(v, act)
        return y, 1.1 * ev + act_error(v, act) * y.abs()
    if gate_first:
        return v, ev
    return v * g, ev * g.abs() + (ge + U) * (v * g).abs()


def scan(x, b, c, delta, A_log, D, dt_bias, init, cu):
    """dict: out, final, and bounds of an fp32 evaluation: ``err_state`` per
    state element, ``err_out`` per output before its own rounding, and
    ``terms`` = sum_n |c_n| |S_n| with every product taken by magnitude (what a
    relative error of the operands multiplies).

    Per step, a_t carries a relative error of |log a| (eD + 16 U) + 4 U: eD that
    of D_t (softplus within 10 steps, its argument within |d| of them), sums of
    log decays and the exponential; the new term carries 64 U: products, the
    split of its weight and the sums of a 64-token chunk on the tensor cores.
    """
    x, b, c, delta, A_log, D, dt_bias, init = (_d(t) for t in (x, b, c, delta, A_log, D, dt_bias, init))
    B, T, H, dv = x.shape
    G, dk = b.shape[-2:]
    R = H // G
    seqs = bounds_of(B, T, cu)
    N = len(seqs)
    fx, fb, fc, fd = x.reshape(B * T, H, dv), b.reshape(B * T, G, dk), c.reshape(B * T, G, dk), delta.reshape(B * T, H)
    out = torch.full((B * T, H, dv), float("nan"), dtype=torch.float64)
    err_out, terms = torch.zeros_like(out), torch.zeros_like(out)
    fin = torch.zeros(N, H, dk, dv, dtype=torch.float64)
    err_state = torch.zeros_like(fin)
    for n, (s, e) in enumerate(seqs):
        S = init[n].clone() if init is not None else torch.zeros(H, dk, dv, dtype=torch.float64)
        M, E = S.abs(), torch.zeros_like(S)
        for t in range(s, e):
            arg = fd[t] + (dt_bias if dt_bias is not None else 0)
            step = torch.log1p(torch.exp(-arg.abs())) + arg.clamp(min=0) if dt_bias is not None else fd[t]
            la = -torch.exp(A_log) * step
            a = torch.exp(la)[:, None, None]
            eD = U * (arg.abs() + 10)
            ea = (la.abs() * (eD + 16 * U) + 4 * U)[:, None, None]
            bt, ct = fb[t].repeat_interleave(R, 0)[:, :, None], fc[t].repeat_interleave(R, 0)[:, :, None]
            new = bt * (step[:, None] * fx[t])[:, None, :]
            E = a * (E + ea * M) + (64 * U + eD[:, None, None]) * new.abs()
            S = a * S + new
            M = a * M + new.abs()
            y = (S * ct).sum(1)
            skip = D[:, None] * fx[t] if D is not None else 0 * fx[t]
            out[t] = y + skip
            terms[t] = (M * ct.abs()).sum(1)
            err_out[t] = (E * ct.abs()).sum(1) + (dk + 4) * U * terms[t] + 2 * U * (y + skip).abs() + U * skip.abs()
        fin[n], err_state[n] = S, E + 2 * U * S.abs()
    shape = (B, T, H, dv)
    return dict(out=out.view(shape), final=fin, err_out=err_out.view(shape), err_state=err_state,
                terms=terms.view(shape))


def scan_step(x, b, c, delta, A_log, D, dt_bias, state):
    """One token: scan() over sequences of length one."""
    r = scan(x[:, None], b[:, None], c[:, None], delta[:, None], A_log, D, dt_bias, state, None)
    return {k: (v[:, 0] if k in ("out", "err_out", "terms") else v) for k, v in r.items()}


def assert_within(got, ref, bound, what=""):
    """Every element of ``got`` within ``bound`` of the fp64 ``ref``, plus the
    rounding of got's own type (half a step of the reference and of the bound)."""
    h = HALF_STEP[got.dtype]
    d = (got.detach().cpu().double() - ref).abs()
    # values below the type's normal range round by at most half of its smallest step
    tiny = float(torch.finfo(got.dtype).tiny)
    allow = bound + h * (ref.abs() + bound) + tiny
    assert torch.isfinite(got).all(), f"{what}: non-finite values"
    bad = d > allow
    if bad.any():
        i = int((d / allow).flatten().argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} elements off; worst {float(d.flatten()[i]):.3e} "
                             f"allowed {float(allow.flatten()[i]):.3e} at flat index {i}, reference "
                             f"{float(ref.flatten()[i]):.6e}")
