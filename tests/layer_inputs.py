"""Seeded inputs of the layer operators' tests."""
import math

import torch


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=torch.float32, std=1.0, device="cuda"):
    return (torch.randn(shape, generator=g) * std).to(device=device, dtype=dtype)


def offsets(lengths, device="cuda"):
    c = [0]
    for n in lengths:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device=device)


def sliced(g, lead, before, shape, after, dtype, device="cuda"):
    """A token tensor [*lead, *shape] lying inside wider rows, with other values on both sides."""
    width = math.prod(shape)
    wide = randn(g, *lead, before + width + after, dtype=dtype, device=device)
    return wide[..., before:before + width].unflatten(-1, shape)


def scan_inputs(seed, lead, H, G, dk, dv, dtype, rate=1.0, wide=True, device="cuda"):
    """x, b, c (slices of wider rows, or dense), delta, and A_log, D, dt_bias.
    ``rate`` scales the decay: exp(A_log) is log-uniform in rate * [1/16, 1]."""
    g = gen(seed)
    pad = 16 if wide else 0
    d = dict(x=sliced(g, lead, pad, (H, dv), pad, dtype, device), b=sliced(g, lead, pad, (G, dk), 2 * pad, dtype, device),
             c=sliced(g, lead, 0, (G, dk), pad, dtype, device), delta=randn(g, *lead, H, device=device))
    d["A_log"] = (torch.rand(H, generator=g) * math.log(1 / 16) + math.log(rate)).to(device)
    d["D"] = randn(g, H, device=device)
    d["dt_bias"] = randn(g, H, device=device) - 1
    return d, g
