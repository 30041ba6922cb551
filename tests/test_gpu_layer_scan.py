"""GPU parity of the selective state-space scan (prompts and single tokens) with
the fp64 reference.

CUDA-core path: every element within the bound that the reference runs beside
the recurrence.  Tensor-core path: the state within the same bound (its operands
carry 24 bits); the outputs' products are taken with bf16 operands, so an output
may be off by half a bf16 step of the sum of its terms' magnitudes on top, and
in the norm by the framework's bf16 contract."""
import pytest
import torch

import gated_delta_rule_121_b200 as kda
from layer_inputs import offsets, randn, scan_inputs
from oracle import layer as ref
from parity import errors

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def on_tensor_cores(dtype, dk, dv):
    return dtype == BF16 and dk in (64, 128) and dv in (64, 128)


def compare(out, fin, d, init, cu, r=None):
    dtype, (dk, dv) = out.dtype, (d["b"].shape[-1], d["x"].shape[-1])
    r = r or ref.scan(d["x"], d["b"], d["c"], d["delta"], d["A_log"], d["D"], d["dt_bias"], init, cu)
    own = ~torch.isnan(r["out"])
    extra = 0.0
    if on_tensor_cores(dtype, dk, dv):
        # operands: half a bf16 step each; a score's decay: the rounding of a
        # 64-token sum of log decays, at most a third of such a step for sums up to 2^13
        extra = (ref.HALF_STEP[BF16] * 4 / 3) * r["terms"][own]
    o = out.cpu()
    ref.assert_within(o[own], r["out"][own], r["err_out"][own] + extra, "scan out")
    if fin is not None:
        ref.assert_within(fin, r["final"], r["err_state"], "scan state")
    if own.sum() > 1000:
        e = errors(o[own], r["out"][own])
        assert e["rel_fro"] <= (5e-3 if dtype == BF16 else 1e-5), e
    return r


def run(d, init, cu, **kw):
    return kda.kda_ssm_fwd(d["x"], d["b"], d["c"], d["delta"], d["A_log"], d["D"], d["dt_bias"], init, cu, **kw)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dk,dv", [(16, 16), (16, 128), (32, 64), (64, 32), (64, 64), (64, 128), (128, 16), (128, 64),
                                   (128, 128)])
def test_sizes(dtype, dk, dv):
    d, g = scan_inputs(dk + dv, (2, 75), 4, 2, dk, dv, dtype)
    init = randn(g, 2, 4, dk, dv)
    compare(*run(d, init, None), d, init, None)


@pytest.mark.parametrize("dtype,dk,dv", [(BF16, 128, 64), (BF16, 64, 128), (F32, 32, 32)])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 321])
def test_lengths(dtype, dk, dv, T):
    d, g = scan_inputs(T, (1, T), 2, 1, dk, dv, dtype)
    compare(*run(d, None, None), d, None, None)


@pytest.mark.parametrize("dtype,dk,dv", [(BF16, 128, 64), (BF16, 128, 128), (BF16, 32, 64), (F32, 64, 64)])
@pytest.mark.parametrize("lengths", [[5], [0, 3, 0, 0, 1, 2, 70], [1] * 9, [64, 64, 128], [63, 65, 130, 1, 0], [200, 0]])
def test_packed(dtype, dk, dv, lengths):
    d, g = scan_inputs(len(lengths) + sum(lengths), (1, sum(lengths)), 3, 1, dk, dv, dtype)
    cu = offsets(lengths)
    init = randn(g, len(lengths), 3, dk, dv)
    compare(*run(d, init, cu), d, init, cu)
    compare(*run(d, None, cu), d, None, cu)


@pytest.mark.parametrize("H,G", [(1, 1), (2, 2), (3, 3), (6, 2), (6, 3), (5, 1), (16, 1)])
@pytest.mark.parametrize("dtype,dk,dv", [(BF16, 64, 64), (BF16, 128, 64), (BF16, 128, 128), (F32, 16, 32)])
def test_heads_and_groups(H, G, dtype, dk, dv):
    d, g = scan_inputs(H * 10 + G, (2, 70), H, G, dk, dv, dtype)
    compare(*run(d, None, None), d, None, None)


@pytest.mark.parametrize("dtype,dk,dv", [(BF16, 128, 64), (BF16, 128, 128), (F32, 64, 64)])
@pytest.mark.parametrize("rate", [1e-4, 30.0, 1000.0])
def test_decays_from_none_to_all(dtype, dk, dv, rate):
    """Decays near one, and decays that leave nothing of a state after a token."""
    d, g = scan_inputs(31, (1, 150), 4, 2, dk, dv, dtype, rate=rate)
    d["delta"][:, 40:60] = -60.0   # steps of zero: the state stands still
    d["delta"][:, 90:93] = 60.0
    init = randn(g, 1, 4, dk, dv)
    compare(*run(d, init, None), d, init, None)


@pytest.mark.parametrize("dtype,dk,dv", [(BF16, 128, 64), (F32, 32, 16)])
def test_optional_parameters_and_dense_inputs(dtype, dk, dv):
    d, g = scan_inputs(32, (2, 66), 4, 1, dk, dv, dtype, wide=False)
    d["D"], d["dt_bias"] = None, None
    d["delta"] = d["delta"].abs().contiguous()  # steps given as they are
    compare(*run(d, None, None), d, None, None)
    out, fin = run(d, None, None, output_final_state=False)
    assert fin is None
    compare(out, None, d, None, None)


@pytest.mark.parametrize("dtype,dk,dv", [(BF16, 128, 64), (BF16, 64, 128), (BF16, 16, 16), (F32, 128, 128)])
def test_rows_outside_the_sequences(dtype, dk, dv):
    """Rows that no sequence holds contain NaN and infinities: no sequence reads
    them (a last chunk shorter than its tile among them), and they stay unwritten."""
    d, g = scan_inputs(33, (1, 160), 2, 1, dk, dv, dtype)
    cu = torch.tensor([3, 73, 73, 139], dtype=torch.int32, device="cuda")
    for k in ("x", "b", "c", "delta"):
        d[k][:, :3] = float("nan")
        d[k][:, 139:150] = float("nan")
        d[k][:, 150:] = float("inf")
    init = randn(g, 3, 2, dk, dv)
    out = torch.full((1, 160, 2, dv), 9.0, dtype=dtype, device="cuda")
    _, fin = run(d, init, cu, out=out)
    compare(out, fin, d, init, cu)
    assert bool((out[:, :3] == 9).all()) and bool((out[:, 139:] == 9).all())


@pytest.mark.parametrize("dtype,dk,dv", [(BF16, 128, 64), (BF16, 128, 128), (F32, 64, 64)])
def test_a_spoilt_sequence_leaves_the_others(dtype, dk, dv):
    d, g = scan_inputs(34, (1, 200), 2, 1, dk, dv, dtype)
    cu = offsets([70, 60, 70])
    want, wf = run(d, None, cu)
    d["x"][0, 75] = float("nan")
    d["b"][0, 100] = float("inf")
    out, fin = run(d, None, cu)
    assert torch.equal(out[:, :70], want[:, :70]) and torch.equal(out[:, 130:], want[:, 130:])
    assert torch.equal(fin[0], wf[0]) and torch.equal(fin[2], wf[2])
    assert not bool(torch.isfinite(out[:, 75:130]).all())


@pytest.mark.parametrize("dtype,dk,dv", [(BF16, 128, 64), (BF16, 64, 128), (F32, 32, 32)])
def test_states_chain_in_place(dtype, dk, dv):
    """Two calls over the halves, the state in place, against the whole."""
    d, g = scan_inputs(35, (2, 130), 4, 2, dk, dv, dtype)
    init = randn(g, 2, 4, dk, dv)
    r = ref.scan(d["x"], d["b"], d["c"], d["delta"], d["A_log"], d["D"], d["dt_bias"], init, None)
    state, outs = init.clone(), []
    for s, e in ((0, 71), (71, 130)):
        part = dict(d, **{k: d[k][:, s:e].contiguous() for k in ("x", "b", "c", "delta")})
        outs.append(run(part, state, None, final_state=state)[0])
    compare(torch.cat(outs, 1), state, d, init, None, r)


@pytest.mark.parametrize("H,G,dk,dv,B,T", [(2, 1, 128, 64, 1, 3000), (1, 1, 64, 64, 1, 2500), (2, 2, 128, 128, 2, 1500)])
def test_long_sequences(H, G, dk, dv, B, T):
    """Few heads, long sequences: the split over the SMs."""
    d, g = scan_inputs(T, (B, T), H, G, dk, dv, BF16, rate=0.05)
    init = randn(g, B, H, dk, dv)
    compare(*run(d, init, None), d, init, None)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_long_packed(dtype):
    d, g = scan_inputs(41, (1, 4000), 2, 1, 128, 64, dtype, rate=0.1)
    cu = offsets([1, 1700, 0, 64, 900, 3, 1332])
    init = randn(g, 7, 2, 128, 64)
    compare(*run(d, init, cu), d, init, cu)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dk,dv", [(16, 16), (128, 16), (16, 128), (32, 64), (64, 64), (128, 64), (128, 128)])
@pytest.mark.parametrize("B,H,G", [(1, 2, 1), (5, 6, 3)])
def test_steps_match_reference(dtype, dk, dv, B, H, G):
    d, g = scan_inputs(dk + B, (B, 4), H, G, dk, dv, dtype)
    state = randn(g, B, H, dk, dv)
    ref_state = state.clone()
    for t in range(4):
        a = [d[k][:, t] for k in ("x", "b", "c")]
        delta = d["delta"][:, t].contiguous()
        r = ref.scan_step(*a, delta, d["A_log"], d["D"], d["dt_bias"], ref_state)
        out = kda.kda_ssm_step(*a, delta, d["A_log"], state, d["D"], d["dt_bias"])
        ref.assert_within(out, r["out"], r["err_out"], f"step {t} out")
        ref.assert_within(state, r["final"], r["err_state"], f"step {t} state")
        ref_state = state.clone()
    out = kda.kda_ssm_step(*a, delta.abs(), d["A_log"], state)  # no skip, steps as given
    r = ref.scan_step(*a, delta.abs(), d["A_log"], None, None, ref_state)
    ref.assert_within(out, r["out"], r["err_out"], "step without D and dt_bias")


@pytest.mark.parametrize("dtype,dk,dv", [(BF16, 128, 64), (F32, 32, 32)])
def test_steps_continue_a_prompt(dtype, dk, dv):
    d, g = scan_inputs(51, (2, 75), 4, 2, dk, dv, dtype)
    r = ref.scan(d["x"], d["b"], d["c"], d["delta"], d["A_log"], d["D"], d["dt_bias"], None, None)
    part = dict(d, **{k: d[k][:, :70] for k in ("b", "c", "delta")}, x=d["x"][:, :70])
    part = {k: (v.contiguous() if k in ("x", "b", "c", "delta") else v) for k, v in part.items()}
    _, state = run(part, None, None)
    for t in range(70, 75):
        out = kda.kda_ssm_step(d["x"][:, t], d["b"][:, t], d["c"][:, t], d["delta"][:, t].contiguous(), d["A_log"], state,
                               d["D"], d["dt_bias"])
        ref.assert_within(out, r["out"][:, t], r["err_out"][:, t], f"token {t}")
    ref.assert_within(state, r["final"], r["err_state"], "state")


def test_no_tokens():
    d, g = scan_inputs(61, (2, 5), 2, 1, 128, 64, BF16)
    none = {k: (d[k][:, :0].contiguous() if k in ("x", "b", "c", "delta") else d[k]) for k in d}
    init = randn(g, 2, 2, 128, 64)
    out, fin = run(none, init, None)
    assert out.shape == (2, 0, 2, 64) and torch.equal(fin, init)
    assert not bool(run(none, None, None)[1].any())


@pytest.mark.parametrize("dtype,H,G,dk,dv", [(BF16, 2, 1, 128, 64), (BF16, 3, 3, 64, 64), (BF16, 1, 1, 128, 128),
                                             (F32, 2, 2, 32, 16)])
@pytest.mark.parametrize("lengths", [None, [1, 1700, 0, 64, 900]])
def test_long_sequences_in_place(dtype, H, G, dk, dv, lengths):
    """Split sequences whose final states go over their initial ones: the bits of
    the call that keeps them apart."""
    T = 2665 if lengths else 1500
    d, g = scan_inputs(71, (1 if lengths else 2, T), H, G, dk, dv, dtype, rate=0.02)
    cu = offsets(lengths) if lengths else None
    init = randn(g, len(lengths) if lengths else 2, H, dk, dv)
    out, fin = run(d, init, cu)
    state = init.clone()
    out2, _ = run(d, state, cu, final_state=state)
    assert torch.equal(out, out2) and torch.equal(fin, state)
    assert not torch.equal(fin, init)


@pytest.mark.parametrize("T", [255, 256, 257, 511, 512, 513, 1025])
@pytest.mark.parametrize("dtype,dv", [(BF16, 64), (F32, 16)])
def test_lengths_around_the_pieces(dtype, dv, T):
    d, g = scan_inputs(T, (1, T), 2, 1, 64, dv, dtype, rate=0.05)
    init = randn(g, 1, 2, 64, dv)
    compare(*run(d, init, None), d, init, None)


def test_offsets_beyond_32_bits():
    """Rows of a tensor of more than 2^31 elements: the bits of the dense rows' result."""
    T, wide = 70000, torch.empty(1, 70000, 32768, dtype=BF16, device="cuda")
    d, g = scan_inputs(81, (1, T), 2, 1, 128, 64, BF16, wide=False)
    dense, dfin = run(d, None, None)
    far = dict(d)
    at = 32768 - 512
    for k in ("x", "b", "c"):
        n = d[k].shape[2] * d[k].shape[3]
        wide[..., at:at + n] = d[k].flatten(2)
        far[k] = wide[..., at:at + n].unflatten(-1, d[k].shape[2:])
        at += n
    out, fin = run(far, None, None)
    assert torch.equal(out, dense) and torch.equal(fin, dfin)


@pytest.mark.parametrize("dv,H,G", [(64, 2, 1), (128, 2, 2)])
@pytest.mark.parametrize("in_place", [False, True])
def test_many_sequences(dv, H, G, in_place):
    """More sequences than blocks, so that a block goes from one to the next: empty
    ones, single tokens and odd lengths among them."""
    lengths = [(7 * i * i + 3) % 83 if i % 11 else 0 for i in range(210)]
    d, g = scan_inputs(51, (1, sum(lengths)), H, G, 64, dv, BF16)
    cu = offsets(lengths)
    init = randn(g, len(lengths), H, 64, dv)
    state = init.clone()
    out, fin = run(d, state, cu, final_state=state if in_place else None)
    compare(out, fin, d, init, cu)


def test_many_short_sequences():
    """More items than blocks take in one wave."""
    d, g = scan_inputs(52, (1100, 3), 1, 1, 64, 64, BF16)
    init = randn(g, 1100, 1, 64, 64)
    compare(*run(d, init, None), d, init, None)


def test_spoilt_sequences_among_many():
    """A block that goes on after a sequence with NaN and infinities carries nothing over."""
    lengths = [64, 65, 3] * 80
    d, g = scan_inputs(53, (1, sum(lengths)), 2, 1, 64, 64, BF16)
    cu = offsets(lengths)
    init = randn(g, len(lengths), 2, 64, 64)
    ok_out, ok_fin = run(d, init, cu)
    bad = torch.zeros(len(lengths), dtype=torch.bool)
    bad[::4] = True
    rows = torch.repeat_interleave(bad, torch.tensor(lengths)).cuda()
    for k, v in (("x", float("nan")), ("b", float("inf")), ("c", float("-inf")), ("delta", float("nan"))):
        d[k][0, rows] = v
    out, fin = run(d, init, cu)
    assert torch.equal(out[0, ~rows], ok_out[0, ~rows])
    assert torch.equal(fin[~bad.cuda()], ok_fin[~bad.cuda()])
