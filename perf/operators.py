"""Cases for measuring the operators of a state-space layer: the short causal
convolution, the selective state-space scan and the group norm, each for
prompts and for single tokens.

A case names one operator and its sizes.  ``run`` computes it in a plain form
(elementary torch operations in fp32, the decays' exponents in fp64, rounded
once at the end) or, where ``own`` is true, by the library's entry points.

Formulas (per sequence; h a head, c a channel, n a group of channels):
  conv   y_t[c] = act(bias[c] + sum_j w[c, j] x_{t-K+1+j}[c]); inputs before the
         first token come from the state (its K - 1 rows) or are zero
  scan   D_t = softplus(delta_t + dt_bias), a_t = exp(-exp(A_log) D_t),
         S_t = a_t S_{t-1} + D_t B_t x_t^T,   y_t = S_t^T C_t + D x_t
  norm   u = x, or x act(gate);  n = (u - mu) / sqrt(mean((u - mu)^2) + eps) w + b
         over each group's channels (mu = 0 for the RMS form);
         y = n act(gate), or n where the gate came first
"""
import math
import random

import torch

own = False

DEV = "cuda"
CHUNK = 128  # tokens per block of the plain scan
EPS = 1e-5
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one projection's channels (96 heads of 128) of a 64K prompt, read as a slice of the fused q, k, v projection
        dict(name="conv 64K", op="conv", B=1, T=65536, C=12288, K=4, dtype="bf16", fused=True, init=False, act="silu"),
        # a packed batch of short prompts continued from cached states, a channel count that no vector width divides
        dict(name="conv packed odd", op="conv", total=5000, lo=1, hi=900, pack=3, C=1111, K=3, dtype="bf16",
             fused=False, init=True, act="silu"),
        # one decode step of a large batch: q, k and v channels of 96 heads of 128
        dict(name="conv step 512", op="conv_step", B=512, C=36864, K=4, dtype="bf16", act="silu"),
        # one decode step of a single sequence, where latency counts
        dict(name="conv step 1", op="conv_step", B=1, C=4096, K=4, dtype="bf16", act="silu"),
        # a 64K prompt through 96 heads
        dict(name="scan 64K", op="scan", B=1, T=65536, H=96, G=8, dk=128, dv=64, dtype="bf16", init=False),
        # a mid-size prompt batch from cached states, 128 x 128 states
        dict(name="scan mid", op="scan", B=2, T=4096, H=16, G=1, dk=128, dv=128, dtype="bf16", init=True),
        # packed prompts of very different lengths
        dict(name="scan packed", op="scan", total=65536, lo=64, hi=16384, pack=5, H=32, G=1, dk=128, dv=64,
             dtype="bf16", init=True),
        # a short fp32 prompt with small states
        dict(name="scan fp32", op="scan", B=2, T=1000, H=4, G=2, dk=16, dv=16, dtype="f32", init=True),
        # one decode step of a large batch: the whole cost is the resident state
        dict(name="scan step 512", op="scan_step", B=512, H=96, G=8, dk=128, dv=128, dtype="bf16"),
        # one decode step of a few sequences
        dict(name="scan step 4", op="scan_step", B=4, H=96, G=8, dk=128, dv=64, dtype="bf16"),
        # the head-wise output norm with its sigmoid gate over a 64K prompt's 96 heads of 128
        dict(name="norm heads 64K", op="norm", rows=65536, C=12288, groups=96, dtype="bf16", act="sigmoid",
             gate="after", center=False, bias=False, shared=True),
        # a decode batch: the gate first, one norm over all channels of 96 heads of 64
        dict(name="norm step 512", op="norm", rows=512, C=6144, groups=1, dtype="bf16", act="silu", gate="first",
             center=False, bias=False, shared=False),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv_step", "scan", "scan", "scan_step", "norm"])
    dtype = "bf16" if rng.random() < 0.75 else "f32"
    act = rng.choice(["silu", "none"])
    if op == "conv":
        C, K = _logu(rng, 16, 12288), rng.choice([2, 3, 4])
        if rng.random() < 0.5:
            total = _logu(rng, 1, 65536)
            return dict(op=op, total=total, lo=1, hi=max(1, total // 2), pack=rng.randrange(1000), C=C, K=K,
                        dtype=dtype, fused=rng.random() < 0.5, init=rng.random() < 0.5, act=act)
        B = rng.randint(1, 4)
        return dict(op=op, B=B, T=_logu(rng, 1, 65536 // B), C=C, K=K, dtype=dtype, fused=rng.random() < 0.5,
                    init=rng.random() < 0.5, act=act)
    if op == "conv_step":
        return dict(op=op, B=_logu(rng, 1, 512), C=_logu(rng, 16, 36864), K=rng.choice([2, 3, 4]), dtype=dtype, act=act)
    if op == "norm":
        groups, width = _logu(rng, 1, 96), _logu(rng, 8, 512)
        gate = rng.choice(["after", "first", "none"])
        return dict(op=op, rows=_logu(rng, 1, 16384), C=groups * width, groups=groups, dtype=dtype,
                    act=rng.choice(["silu", "sigmoid"]), gate=gate, center=rng.random() < 0.5, bias=rng.random() < 0.5,
                    shared=rng.random() < 0.5)
    dk, dv = rng.choice([16, 32, 64, 128, 128]), rng.choice([16, 32, 64, 64, 128])
    G = rng.choice([1, 1, 2, 8])
    if op == "scan_step":
        return dict(op=op, B=_logu(rng, 1, 256), H=G * rng.randint(1, 96 // G), G=G, dk=dk, dv=dv, dtype=dtype)
    if dtype == "f32":  # prompts checked in full precision: short ones
        return dict(op=op, B=rng.randint(1, 2), T=_logu(rng, 1, 4096), H=G * rng.randint(1, 2), G=G, dk=dk, dv=dv,
                    dtype=dtype, init=rng.random() < 0.5)
    H = G * rng.randint(1, 48 // G)
    if rng.random() < 0.4:
        total = _logu(rng, 64, 32768)
        return dict(op=op, total=total, lo=1, hi=max(1, total // 3), pack=rng.randrange(1000), H=H, G=G, dk=dk, dv=dv,
                    dtype=dtype, init=rng.random() < 0.5)
    B = rng.randint(1, 4)
    return dict(op=op, B=B, T=_logu(rng, 1, 32768 // B), H=H, G=G, dk=dk, dv=dv, dtype=dtype, init=rng.random() < 0.5)


def _lengths(case):
    """Packed lengths, log-uniform in [lo, hi], cut off at the total."""
    rng, out, acc = random.Random(case["pack"]), [], 0
    while acc < case["total"]:
        n = min(_logu(rng, case["lo"], case["hi"]), case["total"] - acc)
        out.append(n)
        acc += n
    return out


def _shape(case):
    """(B, T, N, lengths): the tensors' two leading sizes and the sequences in them."""
    if "total" in case:
        lens = _lengths(case)
        return 1, case["total"], len(lens), lens
    return case["B"], case["T"], case["B"], [case["T"]] * case["B"]


def _randn(gen, *shape, std=1.0):
    return torch.randn(shape, generator=gen, device=DEV) * std


def _decay_parameters(gen, H):
    """A_log = log U[1, 16]; dt_bias puts softplus(dt_bias) log-uniform in [1e-3, 1e-1]; D near one."""
    A_log = torch.log(1 + 15 * torch.rand(H, generator=gen, device=DEV))
    dt = torch.exp(torch.rand(H, generator=gen, device=DEV) * math.log(100.0) + math.log(1e-3))
    return A_log, dt + torch.log(-torch.expm1(-dt)), 1 + _randn(gen, H, std=0.2)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    dt, op = DT[case["dtype"]], case["op"]
    s = dict(case=case)
    if op in ("conv", "conv_step"):
        C, K = case["C"], case["K"]
        s["weight"] = _randn(gen, C, K, std=K ** -0.5)
        s["bias"] = _randn(gen, C, std=0.1)
    if op == "conv":
        B, T, N, lens = _shape(case)
        ld = 3 * (-(-C // 8) * 8) if case["fused"] else C
        s["x"] = _randn(gen, B, T, ld).to(dt)[..., :C]
        s["init"] = _randn(gen, N, K - 1, C).to(dt) if case["init"] else None
        s["cu"] = _offsets(lens) if "total" in case else None
    elif op == "conv_step":
        s["x"] = _randn(gen, case["B"], C).to(dt)
        s["state"] = _randn(gen, case["B"], K - 1, C).to(dt)
    elif op == "norm":
        C, rows = case["C"], case["rows"]
        s["x"] = _randn(gen, rows, C).to(dt)
        s["gate"] = _randn(gen, rows, C).to(dt) if case["gate"] != "none" else None
        width = C // case["groups"] if case["shared"] else C
        s["weight"] = 1 + _randn(gen, width, std=0.1)
        s["bias"] = _randn(gen, width, std=0.1) if case["bias"] else None
    else:
        B, T, N, lens = _shape(case) if op == "scan" else (case["B"], 1, case["B"], None)
        H, G, dk, dv = case["H"], case["G"], case["dk"], case["dv"]
        s["A_log"], s["dt_bias"], s["D"] = _decay_parameters(gen, H)
        # x, B and C are slices of one convolution's output, as the layer has them
        lead = (B, T) if op == "scan" else (B,)
        xbc = torch.nn.functional.silu(_randn(gen, *lead, H * dv + 2 * G * dk)).to(dt)
        s["x"] = xbc[..., :H * dv].unflatten(-1, (H, dv))
        s["b"] = xbc[..., H * dv:H * dv + G * dk].unflatten(-1, (G, dk))
        s["c"] = xbc[..., H * dv + G * dk:].unflatten(-1, (G, dk))
        s["delta"] = _randn(gen, *lead, H, std=0.5)
        if op == "scan":
            s["init"] = _randn(gen, N, H, dk, dv, std=0.1) if case["init"] else None
            s["cu"] = _offsets(lens) if "total" in case else None
            s["longest"] = max(lens)
        else:
            s["state"] = _randn(gen, N, H, dk, dv, std=0.1)
    return s


def _offsets(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(DEV)


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import gated_delta_rule_121_b200 as kda
        act = {"none": kda.KDA_ACT_NONE, "silu": kda.KDA_ACT_SILU, "sigmoid": kda.KDA_ACT_SIGMOID}
        if op == "conv":
            return kda.kda_conv_fwd(s["x"], s["weight"], s["bias"], s["init"], s["cu"], activation=act[case["act"]])
        if op == "conv_step":
            return kda.kda_conv_step(s["x"], s["weight"], s["bias"], s["state"], activation=act[case["act"]]), s["state"]
        if op == "scan":
            return kda.kda_ssm_fwd(s["x"], s["b"], s["c"], s["delta"], s["A_log"], s["D"], s["dt_bias"], s["init"], s["cu"])
        if op == "scan_step":
            return kda.kda_ssm_step(s["x"], s["b"], s["c"], s["delta"], s["A_log"], s["state"], s["D"], s["dt_bias"]), s["state"]
        return kda.kda_group_norm(s["x"], case["groups"], s["weight"], s["bias"], s["gate"], eps=EPS, center=case["center"],
                                  activation=act[case["act"]], gate_first=case["gate"] == "first")
    return dict(conv=_conv, conv_step=_conv_step, scan=_scan, scan_step=_scan_step, norm=_norm)[op](s, case)


# ---- plain forms

def _act(x, name):
    return x * torch.sigmoid(x) if name == "silu" else torch.sigmoid(x) if name == "sigmoid" else x


def _sequence_of(s):
    """Sequence, position in it and length of it for every token of a packed batch."""
    cu = s["cu"].long()
    t = torch.arange(s["x"].shape[1], device=DEV)
    n = torch.searchsorted(cu, t, right=True) - 1
    return n, t - cu[n], cu[1:] - cu[:-1]


def _conv(s, case):
    x, K = s["x"], case["K"]
    B, T, C = x.shape
    w, taps = s["weight"], torch.arange(K, device=DEV)
    if s["cu"] is None:
        head = s["init"] if s["init"] is not None else torch.zeros(B, K - 1, C, dtype=x.dtype, device=DEV)
        rows = torch.cat([head, x], 1).float()
        acc = sum(rows[:, j:j + T] * w[:, j] for j in range(K)) + s["bias"]
        last = rows[:, T:]
    else:  # a row of the table for every tap: the sequence's own token, or a row of its state
        n, pos, length = _sequence_of(s)
        N = length.numel()
        head = s["init"] if s["init"] is not None else torch.zeros(N, K - 1, C, dtype=x.dtype, device=DEV)
        rows = torch.cat([head.flatten(0, 1), x[0]]).float()

        def at(n, start, p):  # table row of position p of sequence n
            return torch.where(p < 0, n * (K - 1) + p + K - 1, N * (K - 1) + start + p)

        start = s["cu"].long()
        src = at(n[:, None], start[n][:, None], pos[:, None] - (K - 1) + taps)
        acc = sum(rows[src[:, j]] * w[:, j] for j in range(K))[None] + s["bias"]
        seq = torch.arange(N, device=DEV)[:, None]
        last = rows[at(seq, start[:-1, None], length[:, None] - (K - 1) + taps[:-1])]
    return _act(acc, case["act"]).to(x.dtype), last.to(x.dtype)


def _conv_step(s, case):
    rows = torch.cat([s["state"], s["x"][:, None]], 1)
    out = _act((rows.float() * s["weight"].t()).sum(1) + s["bias"], case["act"]).to(s["x"].dtype)
    s["state"].copy_(rows[:, 1:])
    return out, s["state"]


def _steps(s):
    """D_t and the log decay of every token and head, in fp64."""
    d = s["delta"].double() + s["dt_bias"].double()
    d = torch.clamp(d, min=0) + torch.log1p(torch.exp(-d.abs()))
    return d, -torch.exp(s["A_log"].double()) * d


def _scan(s, case):
    x, b, c = s["x"].float(), s["b"].float(), s["c"].float()
    step, g = _steps(s)
    H, G, dk, dv = case["H"], case["G"], case["dk"], case["dv"]
    if s["cu"] is not None:  # one padded row per sequence
        n, pos, length = _sequence_of(s)
        N, L = length.numel(), s["longest"]
        pad = lambda v: v.new_zeros((N, L) + v.shape[2:]).index_put((n, pos), v[0])  # noqa: E731
        x, b, c, step, g = pad(x), pad(b), pad(c), pad(step), pad(g)
    N, L = x.shape[:2]
    Q = min(CHUNK, L)
    more = -L % Q
    grow = lambda v: torch.cat([v, v.new_zeros((N, more) + v.shape[2:])], 1) if more else v  # noqa: E731
    cut = lambda v: grow(v).unflatten(1, (-1, Q))  # noqa: E731
    xs, bs, cs, step, g = cut(x), cut(b), cut(c), cut(step), cut(g)       # [N, M, Q, ...]
    M, R = xs.shape[1], H // G
    cum = g.cumsum(2)                                                      # [N, M, Q, H]
    rest = g.flip(2).cumsum(2).flip(2) - g                                 # log decay from after t to the chunk's end
    xs = xs.unflatten(3, (G, R))                                           # [N, M, Q, G, R, dv]
    # inside a chunk
    gram = torch.einsum("nmtgk,nmsgk->nmgts", cs, bs)
    t = torch.arange(Q, device=DEV)
    ch = cum.permute(0, 1, 3, 2)                                           # [N, M, H, Q]
    diff = ch[..., :, None] - ch[..., None, :]
    decay = diff.masked_fill_(t[:, None] < t, float("-inf")).float().exp_()
    decay *= step.float().permute(0, 1, 3, 2)[..., None, :]
    del diff
    score = gram[:, :, :, None] * decay.unflatten(2, (G, R))
    y = torch.einsum("nmgrts,nmsgrv->nmtgrv", score, xs)
    del score, decay, gram
    # the chunks' own states, and the state before each chunk
    weight = (rest.exp() * step).float().unflatten(3, (G, R))
    own_state = torch.einsum("nmsgk,nmsgrv->nmgrkv", bs, xs * weight[..., None])
    first = s["init"] if s["init"] is not None else torch.zeros(N, H, dk, dv, device=DEV)
    states = torch.cat([first.view(N, 1, G, R, dk, dv), own_state], 1).flatten(2, 3)  # [N, M + 1, H, dk, dv]
    total = torch.cat([cum.new_zeros(N, 1, H), cum[:, :, -1].cumsum(1)], 1).permute(0, 2, 1)  # [N, H, M + 1]
    m = torch.arange(M + 1, device=DEV)
    passed = (total[..., :, None] - total[..., None, :]).masked_fill_(m[:, None] < m, float("-inf")).exp_().float()
    states = torch.einsum("nhij,njhkv->nihkv", passed, states)
    before = states[:, :-1].unflatten(2, (G, R))
    y += torch.einsum("nmtgk,nmgrkv->nmtgrv", cs, before) * cum.exp().float().unflatten(3, (G, R))[..., None]
    y += xs * s["D"].view(G, R, 1)
    y = y.flatten(1, 2)[:, :L].flatten(2, 3)
    if s["cu"] is not None:
        y = y[n, pos][None]
    return y.to(s["x"].dtype), states[:, -1]


def _scan_step(s, case):
    step, g = _steps(s)
    R = case["H"] // case["G"]
    x, b, c = s["x"].float(), s["b"].float().repeat_interleave(R, 1), s["c"].float().repeat_interleave(R, 1)
    state = s["state"]
    state.mul_(g.exp().float()[..., None, None]).add_((b * step.float()[..., None])[..., None] * x[..., None, :])
    y = torch.einsum("bhkv,bhk->bhv", state, c) + s["D"][:, None] * x
    return y.to(s["x"].dtype), state


def _norm(s, case):
    x, act = s["x"].float(), case["act"]
    gate = _act(s["gate"].float(), act) if s["gate"] is not None else None
    u = x * gate if case["gate"] == "first" else x
    u = u.unflatten(-1, (case["groups"], -1))
    if case["center"]:
        u = u - u.mean(-1, keepdim=True)
    u = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + EPS)
    wide = lambda v: v if case["shared"] else v.view(case["groups"], -1)  # noqa: E731
    u = u * wide(s["weight"])
    if s["bias"] is not None:
        u = u + wide(s["bias"])
    u = u.flatten(-2)
    if case["gate"] == "after":
        u = u * gate
    elif case["gate"] == "none":
        u = _act(u, act)
    return u.to(s["x"].dtype)


# ---- the definitions in fp64

def exact(case, seed):
    s = prepare(case, seed)
    f = lambda v: None if v is None else v.double()  # noqa: E731
    op = case["op"]
    if op == "norm":
        x, w, b, z = f(s["x"]), f(s["weight"]), f(s["bias"]), f(s["gate"])
        squash = lambda v: torch.sigmoid(v) * (v if case["act"] == "silu" else 1)  # noqa: E731
        if case["gate"] == "first":
            x = x * squash(z)
        groups = torch.stack(x.chunk(case["groups"], -1), 1)
        mean = groups.mean(-1, keepdim=True) if case["center"] else 0.0
        groups = (groups - mean) / torch.sqrt(((groups - mean) ** 2).mean(-1, keepdim=True) + EPS)
        per = case["groups"] if case["shared"] else 1
        out = groups.reshape(x.shape) * w.repeat(per)
        if b is not None:
            out = out + b.repeat(per)
        return out * squash(z) if case["gate"] == "after" else out if case["gate"] == "first" else squash(out)
    if op in ("conv", "conv_step"):
        K = case["K"]
        if op == "conv_step":
            seqs, heads = list(f(s["x"])[:, None]), f(s["state"])
        else:
            B, T, N, lens = _shape(case)
            seqs = list(s["x"].reshape(B * T, -1).split(lens))
            heads = s["init"] if s["init"] is not None else [None] * N
        outs, lasts = [], []
        for x, head in zip(seqs, heads):
            head = torch.zeros(K - 1, x.shape[1], device=DEV) if head is None else head
            rows = torch.cat([head.double(), x.double()])
            y = torch.zeros(x.shape, dtype=torch.float64, device=DEV) + f(s["bias"])
            for j in range(K):
                y.addcmul_(rows[j:j + x.shape[0]], f(s["weight"])[:, j])
            outs.append(y / (1 + torch.exp(-y)) if case["act"] == "silu" else y)
            lasts.append(rows[rows.shape[0] - (K - 1):])
        out = torch.cat(outs)
        return (out if op == "conv_step" else out.view(s["x"].shape)), torch.stack(lasts)
    # the scan, token by token
    H, G, dk, dv = case["H"], case["G"], case["dk"], case["dv"]
    d = f(s["delta"]) + f(s["dt_bias"])
    d = torch.where(d > 40, d, torch.log1p(torch.exp(d.clamp(max=40))))
    a = torch.exp(-torch.exp(f(s["A_log"])) * d)
    if op == "scan_step":
        lens, x, b, c, a, d = None, f(s["x"])[:, None], f(s["b"])[:, None], f(s["c"])[:, None], a[:, None], d[:, None]
        S = f(s["state"])
    else:
        B, T, N, lens = _shape(case)
        if max(lens) * max(1.0, N * H * dk * dv / 2e6) > 250_000:
            return None  # the token loop would take too long
        split = lambda v: torch.nn.utils.rnn.pad_sequence(list(v.reshape(B * T, *v.shape[2:]).split(lens)), batch_first=True)  # noqa: E731
        # padding tokens keep the state: a decay of one and a step of zero
        x, b, c, d = split(f(s["x"])), split(f(s["b"])), split(f(s["c"])), split(d)
        a = 1 - split(1 - a)
        S = f(s["init"]) if s["init"] is not None else torch.zeros(N, H, dk, dv, dtype=torch.float64, device=DEV)
    S = S.view(-1, G, H // G, dk, dv).clone()
    x, a, d = (v.unflatten(2, (G, H // G)) for v in (x, a, d))
    dx, a = (x * d[..., None])[..., None, :], a[..., None, None]
    b, c = b[:, :, :, None, :, None], c[:, :, :, None, None, :]
    outs = []
    for t in range(x.shape[1]):
        S.mul_(a[:, t]).addcmul_(b[:, t], dx[:, t])
        outs.append(torch.matmul(c[:, t], S)[..., 0, :])
    y = torch.stack(outs, 1) + f(s["D"]).view(G, H // G, 1) * x
    y = y.flatten(2, 3)
    if lens is None:
        y = y[:, 0]
    else:
        y = torch.cat([y[i, :n] for i, n in enumerate(lens)]).view(s["x"].shape)
    return y, S.flatten(1, 2)


def work(case):
    """Bytes and operations of one pass: every input read once, every output written once."""
    e, op = (2 if case["dtype"] == "bf16" else 4), case["op"]
    if op == "norm":
        n = case["rows"] * case["C"]
        return dict(bytes=n * e * (2 if case["gate"] == "none" else 3), flops=8 * n)
    if op == "conv_step":
        n = case["B"] * case["C"]
        return dict(bytes=n * e * 2 * case["K"] + 4 * case["C"] * (case["K"] + 1), flops=2 * case["K"] * n)
    if op == "conv":
        B, T, N, _ = _shape(case)
        state = N * (case["K"] - 1) * case["C"] * e
        return dict(bytes=2 * B * T * case["C"] * e + state * (2 if case["init"] else 1) + 4 * case["C"] * (case["K"] + 1),
                    flops=2 * case["K"] * B * T * case["C"])
    H, G, dk, dv = case["H"], case["G"], case["dk"], case["dv"]
    B, T, N, _ = _shape(case) if op == "scan" else (case["B"], 1, case["B"], None)
    token = e * (2 * H * dv + 2 * G * dk) + 4 * H
    states = 4 * N * H * dk * dv * (2 if op == "scan_step" or case["init"] else 1)
    # the recurrence's own products: the state's update and its read
    return dict(bytes=B * T * token + states, flops=4 * B * T * H * dk * dv)
