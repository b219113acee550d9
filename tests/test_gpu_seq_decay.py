"""GPU parity of linear attention with a decay (dlrm_seq_decay.h; needs an MI355X) against oracle/decay.py.

Error measure: |gpu - oracle| over the sum of the absolute values of the terms (the oracle's scales).  Gates, from the
arithmetic, for sequences of n events and heads of d:
  - a state's value is a sum of products y_j z_j w_j: w of up to n / 64 + 3 factors e^g, each right to 2^-21 (exp2, its
    argument and the product), at most 80 fp32 additions of 2^-24 a chunk of terms that are its own: f = (n / 64 + 3) 2^-21 + 80 2^-23;
  - o, dq, dk, dv: pairs and states rounded to bf16 (2^-8), the result too (2^-8), w_j z_j as two parts (2^-16), a product over d
    in fp32: 2^-7 + 2^-16 + f + d 2^-23;
  - dg is a sum, from an event to at most 8 chunks further, of terms of either sign that are right to f + d 2^-23 (three
    parts: no rounding to bf16).  With random inputs the terms' errors are independent: their sum over 576 events is 24 of
    them, and dg itself at least one of the terms: a norm of the error of 24 (f + d 2^-23) of that of dg.  For one decay a head,
    errors of the 128 events between two marks are alike: sqrt(128) (f + d 2^-23) 24 of the norm of the events' dg.
Inputs are bf16 values (g fp32), so both sides start from the same numbers.
"""
import zlib

import numpy as np
import pytest
import torch

from oracle import decay as oracle
from recommendation_model_sparse_amd import (binding, dlrm_seq_decay_bwd, dlrm_seq_decay_fwd, dlrm_seq_decay_step, synth)

from gpu_util import DEV, rel_err, say, to_dev

pytestmark = pytest.mark.gpu


def rng_of(*a):
    return np.random.default_rng(zlib.crc32("-".join(map(str, a)).encode()))


def bf16(rng, *shape):
    """(device bf16 tensor, host fp64 values)."""
    bits = synth.f32_to_bf16_bits(rng.standard_normal(shape).astype(np.float32))
    return to_dev(bits), synth.bf16_bits_to_f32(bits).astype(np.float64)


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def offsets(lens, dtype=np.int64):
    return np.cumsum([0] + list(lens)).astype(dtype)


def decays(rng, N, H, each):
    """By the time between events: mostly short, now and then a pause that ends what was before."""
    if not each:
        return (-rng.exponential(0.1, H)).astype(np.float32)
    g = -rng.exponential(0.1, (N, H))
    return np.where(rng.random((N, 1)) < 0.02, -20.0, g).astype(np.float32)


def gates(n, d):
    f = (n / 64 + 3) * 2.0 ** -21 + 80 * 2.0 ** -23
    return dict(state=f, bf16=2.0 ** -7 + 2.0 ** -16 + f + d * 2.0 ** -23, dg=24 * (f + d * 2.0 ** -23))


def problem(rng, lens, Hq, Hkv, d, each=True, itype=np.int64):
    off = offsets(lens, itype)
    N = int(off[-1])
    x = [bf16(rng, N, Hq, d), bf16(rng, N, Hkv, d), bf16(rng, N, Hkv, d)]
    g = decays(rng, N, Hkv, each)
    do = bf16(rng, N, Hq, d)
    return off, [a for a, _ in x], [b for _, b in x], g, do


def check_dg(got, ref, refs, gate, each):
    """refs: the events' dg.  Norm of the error over that of dg (for each head where there is one decay for it)."""
    if each:
        assert np.linalg.norm(got - ref) <= gate * np.linalg.norm(ref)
    else:
        assert (np.abs(got - ref) <= np.sqrt(128) * gate * np.linalg.norm(refs, axis=0)).all()


LENS = {
    "one": [1], "few": [3, 0, 1, 2, 0], "chunks": [63, 64, 65, 1, 15, 16, 17], "twos": [127, 128, 129, 31, 32, 33], "long": [700, 5, 391],
    "marks": [511, 512, 513, 576], "runs": [1500],
}
SHAPES = [
    # lens, Hq, Hkv, d, a decay for each event, the longest history as the call is told
    ("one", 1, 1, 8, True, 1), ("one", 4, 2, 64, False, None), ("few", 2, 1, 16, True, 3), ("few", 3, 3, 128, False, None), ("chunks", 2, 2, 32, True, 65),
    ("chunks", 4, 1, 64, True, None), ("chunks", 2, 1, 40, False, 65), ("chunks", 2, 2, 128, True, 65), ("twos", 6, 2, 64, True, 129),
    ("twos", 4, 2, 96, False, None), ("twos", 1, 1, 128, True, None), ("long", 2, 1, 64, True, None), ("long", 2, 2, 32, False, 700), ("long", 6, 2, 128, True, 700),
    ("long", 4, 4, 24, True, 1), ("long", 8, 1, 128, False, None), ("marks", 2, 1, 64, True, 1), ("marks", 1, 1, 32, False, 1), ("marks", 2, 2, 128, True, 1),
    ("runs", 2, 2, 32, True, None), ("runs", 4, 2, 64, False, None), ("runs", 3, 1, 128, True, None), ("runs", 1, 1, 64, True, 1)]


@pytest.mark.parametrize("lens,Hq,Hkv,d,each,longest", SHAPES)
@pytest.mark.parametrize("itype", [np.int64, np.int32])
def test_forward_backward(lens, Hq, Hkv, d, each, longest, itype):
    if itype is np.int32 and lens not in ("few", "runs"):
        pytest.skip("int32 offsets on two sets of lengths")
    rng = rng_of("decay", lens, Hq, Hkv, d, each)
    off, dev, (q, k, v), g, (do_d, do) = problem(rng, LENS[lens], Hq, Hkv, d, each, itype)
    scale = float(np.float32(d ** -0.5))
    full = oracle.decay(q, k, v, np.broadcast_to(g, (len(q), Hkv)).astype(np.float64), off, scale, do=do)
    gate = gates(max(LENS[lens]), d)
    off_d, g_d = to_dev(off), to_dev(g)
    say(f"[decay] {lens} Hq={Hq} Hkv={Hkv} d={d} each={each} longest={longest} {itype.__name__}")
    o = dlrm_seq_decay_fwd(*dev, g_d, off_d, max_len=longest)
    torch.cuda.synchronize()
    assert rel_err(host(o), full["o"], full["o_s"]) <= gate["bf16"]
    o2, state = dlrm_seq_decay_fwd(*dev, g_d, off_d, max_len=longest, want_state=True)
    torch.cuda.synchronize()
    assert rel_err(host(o2), full["o"], full["o_s"]) <= gate["bf16"]
    assert rel_err(state.cpu().numpy().astype(np.float64), full["state"], full["state_s"]) <= gate["state"]
    got = dlrm_seq_decay_bwd(do_d, *dev, g_d, off_d, max_len=longest)
    again = dlrm_seq_decay_bwd(do_d, *dev, g_d, off_d, max_len=longest)
    fixed = dlrm_seq_decay_bwd(do_d, *dev, g_d, off_d, max_len=longest, want_dg=False)
    torch.cuda.synchronize()
    assert fixed[3] is None
    for name, x, y, z in zip(("dq", "dk", "dv"), got, again, fixed):
        err = rel_err(host(x), full[name], full[name + "_s"])
        say(f"   {name} {err:.2e} (gate {gate['bf16']:.2e})")
        assert torch.equal(x, y) and err <= gate["bf16"] and rel_err(host(z), full[name], full[name + "_s"]) <= gate["bf16"], name
    assert torch.equal(got[3], again[3])
    want = full["dg"] if each else full["dg"].sum(0)
    check_dg(got[3].cpu().numpy().astype(np.float64), want, full["dg"], gate["dg"], each)


# sequences, their lengths, Hq, Hkv, d: cut into runs of one chunk to many (and a length a call is told that leaves them whole)
CUTS = [(26, 1100, 1500, 2, 2, 128), (8, 500, 2000, 4, 4, 128), (4, 2000, 4096, 8, 2, 128), (64, 500, 1500, 2, 2, 64), (200, 100, 2000, 4, 2, 64),
        (16, 300, 600, 4, 4, 32), (1, 8192, 8192, 4, 4, 64), (64, 200, 1500, 8, 2, 128), (3, 20000, 30000, 1, 1, 64), (100, 1000, 2000, 1, 1, 24)]


@pytest.mark.parametrize("B,lo,hi,Hq,Hkv,d", CUTS)
def test_runs_of_every_length(B, lo, hi, Hq, Hkv, d):
    """Cut and whole the results agree to twice the gates, in the norm of the values themselves (roundings of either sign add up
    as the terms do), and one decay a head has the events' gradients' sum."""
    rng = rng_of("cuts", B, lo, hi, d)
    lens = rng.integers(lo, hi + 1, B)
    off, dev, _, g, (do, _) = problem(rng, lens, Hq, Hkv, d, False)
    off, g, n = to_dev(off), to_dev(g), int(lens.max())
    each = g.expand(dev[0].shape[0], Hkv).contiguous()
    gate = gates(n, d)
    cut, whole = (dlrm_seq_decay_bwd(do, *dev, each, off, max_len=m) for m in (n, 1))
    head, head_whole = (dlrm_seq_decay_bwd(do, *dev, g, off, max_len=m) for m in (n, 1))
    o, o_whole = (dlrm_seq_decay_fwd(*dev, each, off, want_state=True, max_len=m) for m in (n, 1))
    torch.cuda.synchronize()
    far = lambda x, y: float((x.double() - y.double()).norm() / y.double().norm())  # noqa: E731
    say(f"[decay] {B} of {lo}..{hi} d={d}: dg {far(cut[3], whole[3]):.1e}, a head's {far(head[3], cut[3].double().sum(0)):.1e}")
    for x, y in zip(cut[:3] + head[:3] + o[:1], whole[:3] + head_whole[:3] + o_whole[:1]):
        assert far(x, y) <= 2 * gate["bf16"]
    assert far(o[1], o_whole[1]) <= 2 * gate["state"]
    assert far(cut[3], whole[3]) <= 2 * gate["dg"]
    want, room = cut[3].double().sum(0), 2 * np.sqrt(128) * gate["dg"] * cut[3].double().norm(dim=0)
    for x in (head[3], head_whole[3]):
        assert ((x.double() - want).abs() <= room).all()


def test_gradients_against_differences():
    """The loss <do, o> along a direction of each input: the kernels' gradients against central differences of the oracle's
    forward in fp64."""
    rng = rng_of("decay-diff")
    off, dev, at, g, (do_d, do) = problem(rng, [50, 130, 7], 2, 1, 32)
    g = np.maximum(g, -3.0)  # a pause's derivative is below the gate
    got = dlrm_seq_decay_bwd(do_d, *dev, to_dev(g), to_dev(off))
    torch.cuda.synchronize()
    at = at + [g.astype(np.float64)]
    scale, h, gate = float(np.float32(32 ** -0.5)), 2.0 ** -12, gates(130, 32)
    ref = oracle.decay(*at, off, scale, do=do)
    for i, name in enumerate(("dq", "dk", "dv", "dg")):
        step = rng.standard_normal(at[i].shape)
        ends = []
        for sign in (1, -1):
            x = list(at)
            x[i] = at[i] + sign * h * step if name != "dg" else np.minimum(at[i] + sign * h * step, 0.0)
            ends.append((oracle.decay(*x, off, scale)["o"] * do).sum())
        if name == "dg":  # (a decay next to 0 moves by less than the step: the step as it was taken)
            step = (np.minimum(at[i] + h * step, 0.0) - np.minimum(at[i] - h * step, 0.0)) / (2 * h)
        slope, want = (ends[0] - ends[1]) / (2 * h), (host(got[i]) * step).sum()
        room = gate["bf16"] * (ref[name + "_s"] * np.abs(step)).sum() if name != "dg" else 2.0 ** -10 * (np.abs(ref["dg"] * step)).sum()
        say(f"[decay] {name} slope {slope:.6f} gradient {want:.6f}")
        assert abs(slope - want) <= room, name


@pytest.mark.parametrize("lens,Hq,Hkv,d,longest", [("few", 2, 2, 64, None), ("twos", 4, 2, 32, 129), ("long", 4, 1, 128, None), ("long", 2, 2, 96, 700),
                                                   ("runs", 8, 2, 64, None)])
def test_states(lens, Hq, Hkv, d, longest):
    """From a state on; in place; and in two visits."""
    rng = rng_of("decay-state", lens, d)
    off, dev, (q, k, v), g, _ = problem(rng, LENS[lens], Hq, Hkv, d)
    B, scale = len(off) - 1, float(np.float32(d ** -0.5))
    first = rng.standard_normal((B, Hkv, d, d)).astype(np.float32)
    ref = oracle.decay(q, k, v, g.astype(np.float64), off, scale, first.astype(np.float64))
    gate = gates(max(LENS[lens]), d)
    say(f"[decay] states {lens} d={d}")
    o, last = dlrm_seq_decay_fwd(*dev, to_dev(g), to_dev(off), state=to_dev(first), want_state=True, max_len=longest)
    torch.cuda.synchronize()
    assert rel_err(host(o), ref["o"], ref["o_s"]) <= gate["bf16"]
    assert rel_err(last.cpu().numpy().astype(np.float64), ref["state"], ref["state_s"]) <= gate["state"]
    for b in range(B):
        if off[b] == off[b + 1]:
            assert np.array_equal(last[b].cpu().numpy(), first[b])
    own = to_dev(first)
    o2, same = dlrm_seq_decay_fwd(*dev, to_dev(g), to_dev(off), state=own, state_out=own, max_len=longest)
    torch.cuda.synchronize()
    assert same is own and torch.equal(own, last) and torch.equal(o2, o)
    # two visits: the first half of each sequence, then the rest
    half = [(int(off[b]), int(off[b] + off[b + 1]) // 2, int(off[b + 1])) for b in range(B)]
    state, outs = to_dev(first), {}
    for part in (0, 1):
        rows = np.concatenate([np.arange(h[part], h[part + 1]) for h in half]).astype(np.int64)
        cut = offsets([h[part + 1] - h[part] for h in half])
        at = to_dev(rows)
        out, _ = dlrm_seq_decay_fwd(*(x[at] for x in dev), to_dev(g)[at], to_dev(cut), state=state, state_out=state, max_len=longest)
        outs[part] = (rows, host(out))
    torch.cuda.synchronize()
    got = np.zeros(ref["o"].shape)
    for rows, out in outs.values():
        got[rows] = out
    assert rel_err(got, ref["o"], ref["o_s"]) <= gate["bf16"]
    assert rel_err(state.cpu().numpy().astype(np.float64), ref["state"], ref["state_s"]) <= 2 * gate["state"]


@pytest.mark.parametrize("B,Hq,Hkv,d,each", [(1, 4, 4, 32, True), (3, 2, 1, 8, True), (5, 8, 2, 64, False), (2, 12, 1, 128, True), (7, 10, 2, 40, True), (300, 2, 2, 96, False)])
def test_step_by_step(B, Hq, Hkv, d, each):
    """Four events of each user, one after the other, on the state of the one before."""
    rng = rng_of("decay-step", B, d)
    n = 4
    off, dev, (q, k, v), g, _ = problem(rng, [n] * B, Hq, Hkv, d, each)
    first = rng.standard_normal((B, Hkv, d, d)).astype(np.float32)
    scale = float(np.float32(d ** -0.5))
    ref = oracle.decay(q, k, v, g.astype(np.float64), off, scale, first.astype(np.float64))
    state = to_dev(first)
    say(f"[decay] step B={B} Hq={Hq} Hkv={Hkv} d={d}")
    for t in range(n):
        at = to_dev(off[:-1] + t)
        # expf and its product: 2^-22; d fp32 additions; the result rounded
        o = dlrm_seq_decay_step(*(x[at] for x in dev), to_dev(g)[at] if each else to_dev(g), state)
        torch.cuda.synchronize()
        rows = off[:-1] + t
        assert rel_err(host(o), ref["o"][rows], ref["o_s"][rows]) <= 2.0 ** -8 + (t + 1) * 2.0 ** -21 + d * 2.0 ** -23
    assert rel_err(state.cpu().numpy().astype(np.float64), ref["state"], ref["state_s"]) <= n * 2.0 ** -21


def test_strided_views_of_a_joint_projection():
    rng = rng_of("decay-strided")
    lens, Hq, Hkv, d = [40, 90, 3], 4, 2, 32
    off = to_dev(offsets(lens))
    N = sum(lens)
    joint, _ = bf16(rng, N, Hq + 2 * Hkv, d)
    qkv = [joint[:, :Hq], joint[:, Hq:Hq + Hkv], joint[:, Hq + Hkv:]]
    wide = to_dev(decays(rng, N, 5, True))
    g = wide[:, 1:1 + Hkv]  # rows of five
    do, _ = bf16(rng, N, Hq, d)
    packed = [t.contiguous() for t in qkv]
    heads_first = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in packed]  # head stride above the row stride
    state = to_dev(rng.standard_normal((3, Hkv, d, d)).astype(np.float32))
    results = []
    for x, y in ((qkv, g), (packed, g.contiguous()), (heads_first, g.contiguous())):
        results.append([dlrm_seq_decay_fwd(*x, y, off), *dlrm_seq_decay_fwd(*x, y, off, state=state, want_state=True), *dlrm_seq_decay_bwd(do, *x, y, off)])
        own = state[:1].clone()
        results[-1] += [dlrm_seq_decay_step(*(t[:1] for t in x), y[:1], own), own]
    torch.cuda.synchronize()
    for r in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], r))


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("which", ["q", "k", "v", "g"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_what_later_events_hold(d, which, bad):
    """An infinity or NaN changes nothing before it and nothing in other sequences; after it, what it reaches is not
    finite.  In dq neither, for those in k and v."""
    rng = rng_of("decay-hidden", d, which)
    n, at = 200, 137
    off = to_dev(offsets([n, n]))
    q, k, v, do = (bf16(rng, 2 * n, h, d)[0] for h in (2, 1, 1, 2))
    g = to_dev(np.maximum(decays(rng, 2 * n, 1, True), -0.5))
    clean = dlrm_seq_decay_fwd(q, k, v, g, off)
    grads = dlrm_seq_decay_bwd(do, q, k, v, g, off)
    x = dict(q=q.clone(), k=k.clone(), v=v.clone(), g=g.clone())
    if which == "g" and bad == float("inf"):
        pytest.skip("a decay above 0 counts as 0")
    if which == "g":
        x["g"][at] = bad
    else:
        x[which][at, 0, 3] = bad
    say(f"[decay] {which} holds {bad} d={d}")
    o = dlrm_seq_decay_fwd(x["q"], x["k"], x["v"], x["g"], off)
    torch.cuda.synchronize()
    assert torch.equal(o[:at], clean[:at]) and torch.equal(o[n:], clean[n:])
    if which == "q":
        assert torch.equal(o[at + 1:], clean[at + 1:]) and torch.equal(o[at, 1], clean[at, 1]) and not torch.isfinite(o[at, 0].float()).any()
    elif which == "v":
        assert not torch.isfinite(o[at:n, :, 3].float()).any() and torch.equal(o[at:n, :, 4:], clean[at:n, :, 4:])
    else:
        assert not torch.isfinite(o[at:n].float()).any()
    if which in "kv":
        dq = dlrm_seq_decay_bwd(do, x["q"], x["k"], x["v"], x["g"], off)
        torch.cuda.synchronize()
        assert torch.equal(dq[0][:at], grads[0][:at])
        assert all(torch.equal(a[n:], b[n:]) for a, b in zip(dq, grads))


def test_decays_at_the_ends():
    """-infinity and -1000 end what was before (e^g is 0), 0 keeps all, what is above counts as 0, with a gradient of 0."""
    rng = rng_of("decay-ends")
    off, dev, (q, k, v), _, (do_d, do) = problem(rng, [150, 70], 2, 2, 64)
    g = np.full((220, 2), -0.05, np.float32)
    g[20], g[90], g[100], g[64] = -np.inf, -1000.0, 0.0, 2.5
    g[0] = 7.0
    scale = float(np.float32(64 ** -0.5))
    with np.errstate(under="ignore"):
        ref = oracle.decay(q, k, v, g.astype(np.float64), off, scale, do=do)
    gate = gates(150, 64)
    say("[decay] the ends of the decays")
    o, state = dlrm_seq_decay_fwd(*dev, to_dev(g), to_dev(off), want_state=True)
    got = dlrm_seq_decay_bwd(do_d, *dev, to_dev(g), to_dev(off))
    torch.cuda.synchronize()
    assert rel_err(host(o), ref["o"], ref["o_s"]) <= gate["bf16"] and rel_err(state.cpu().numpy().astype(np.float64), ref["state"], ref["state_s"]) <= gate["state"]
    for name, x in zip(("dq", "dk", "dv"), got):
        assert rel_err(host(x), ref[name], ref[name + "_s"]) <= gate["bf16"], name
    check_dg(host(got[3]), ref["dg"], ref["dg"], gate["dg"], True)
    assert (got[3][64] == 0).all() and (got[3][0] == 0).all()
    head = dlrm_seq_decay_bwd(do_d, *dev, to_dev(np.array([0.5, -0.1], np.float32)), to_dev(off))[3]
    assert head[0] == 0 and head[1] != 0


def test_rows_outside_every_sequence_are_left():
    rng = rng_of("decay-outside")
    N, Hq, Hkv, d = 300, 2, 1, 40
    off = to_dev(np.array([30, 100, 100, 270], np.int64))
    (q, qh), (k, kh), (v, vh), (do, doh) = (bf16(rng, N, h, d) for h in (Hq, Hkv, Hkv, Hq))
    g = decays(rng, N, Hkv, True)
    bf = dict(dtype=torch.bfloat16, device=DEV)
    outs = [torch.full((N, Hq, d), 7.0, **bf), torch.full((N, Hq, d), 7.0, **bf), torch.full((N, Hkv, d), 7.0, **bf), torch.full((N, Hkv, d), 7.0, **bf),
            torch.full((N, Hkv), 7.0, device=DEV)]
    say("[decay] rows outside")
    dlrm_seq_decay_fwd(q, k, v, to_dev(g), off, out=outs[0])
    dlrm_seq_decay_bwd(do, q, k, v, to_dev(g), off, dq=outs[1], dk=outs[2], dv=outs[3], dg=outs[4])
    torch.cuda.synchronize()
    ref, gate = oracle.decay(qh, kh, vh, g.astype(np.float64), [30, 100, 100, 270], float(np.float32(d ** -0.5)), do=doh), gates(170, d)
    inside = slice(30, 270)
    for name, x in zip(("o", "dq", "dk", "dv", "dg"), outs):
        assert (x[:30] == 7).all() and (x[270:] == 7).all(), name
        if name != "dg":
            assert rel_err(host(x[inside]), ref[name][inside], ref[name + "_s"][inside]) <= gate["bf16"], name
    check_dg(host(outs[4][inside]), ref["dg"][inside], ref["dg"][inside], gate["dg"], True)


def test_nothing():
    say("[decay] nothing")
    bf = dict(dtype=torch.bfloat16, device=DEV)
    q, k = torch.zeros((0, 2, 32), **bf), torch.zeros((0, 1, 32), **bf)
    for B in (0, 3):
        off = torch.zeros(B + 1, dtype=torch.int64, device=DEV)
        state = torch.randn((B, 1, 32, 32), device=DEV)
        o, last = dlrm_seq_decay_fwd(q, k, k, torch.zeros((0, 1), device=DEV), off, state=state, want_state=True)
        got = dlrm_seq_decay_bwd(q, q, k, k, torch.zeros(1, device=DEV), off)
        torch.cuda.synchronize()
        assert o.shape == (0, 2, 32) and torch.equal(last, state) and (got[3] == 0).all()
    assert dlrm_seq_decay_step(q, k, k, torch.zeros(1, device=DEV), torch.zeros((0, 1, 32, 32), device=DEV)).shape == (0, 2, 32)


@pytest.mark.parametrize("d,Hq,Hkv", [(32, 2, 2), (64, 2, 1), (128, 1, 1)])
def test_many_sequences_of_every_length(d, Hq, Hkv):
    """More sequences than places (they go by their length): each as by itself, and one sum for a head's decay."""
    rng = rng_of("decay-many", d)
    B = 1700
    lens = rng.integers(0, 200, B)
    off = offsets(lens)
    N = int(off[-1])
    g1, g2 = torch.Generator(device=DEV).manual_seed(1), decays(rng, N, Hkv, True)
    q, k, v, do = (torch.randn((N, h, d), generator=g1, device=DEV).bfloat16() for h in (Hq, Hkv, Hkv, Hq))
    say(f"[decay] many d={d}")
    o, state = dlrm_seq_decay_fwd(q, k, v, to_dev(g2), to_dev(off), want_state=True, max_len=200)
    got = dlrm_seq_decay_bwd(do, q, k, v, to_dev(g2), to_dev(off), max_len=200)
    one = to_dev(np.full(Hkv, -0.03, np.float32))
    head = dlrm_seq_decay_bwd(do, q, k, v, one, to_dev(off), max_len=200)[3]
    spread = dlrm_seq_decay_bwd(do, q, k, v, one.expand(N, Hkv).contiguous(), to_dev(off), max_len=200)[3]
    torch.cuda.synchronize()
    for _ in range(3):
        assert torch.equal(dlrm_seq_decay_bwd(do, q, k, v, one, to_dev(off), max_len=200)[3], head)
    gate = gates(200, d)["dg"]
    check_dg(host(head), host(spread).sum(0), host(spread), 2 * gate, False)
    for b in list(range(0, B, 97)) + [int(lens.argmax()), int(lens.argmin())]:
        rows = slice(int(off[b]), int(off[b + 1]))
        alone = to_dev(offsets([lens[b]]))
        x = [t[rows] for t in (q, k, v)] + [to_dev(g2)[rows], alone]
        o1, s1 = dlrm_seq_decay_fwd(*x, want_state=True, max_len=1)
        assert torch.equal(o[rows], o1) and torch.equal(state[b], s1[0])
        *alone, dg = dlrm_seq_decay_bwd(do[rows], *x, max_len=1)
        assert all(torch.equal(a[rows], c) for a, c in zip(got, alone))
        # by itself a sequence's query heads go to two workgroups, whose terms are added in fp32 afterwards
        check_dg(host(got[3][rows]), host(dg), host(dg), gate, True)


def test_large_rows_and_strides():
    """Rows whose elements lie past 2^31."""
    rng = rng_of("decay-far")
    N, d, row = 260, 32, 1 << 23  # 260 * 2^23 elements: past 2^31
    wide = torch.zeros((N, row), dtype=torch.bfloat16, device=DEV)
    near = [bf16(rng, N, 1, d)[0] for _ in range(3)]
    far = []
    for i, t in enumerate(near):
        wide[:, i * d:(i + 1) * d] = t[:, 0]
        far.append(wide[:, i * d:(i + 1) * d].unflatten(1, (1, d)))
    g, off = to_dev(decays(rng, N, 1, True)), to_dev(offsets([200, 60]))
    do = bf16(rng, N, 1, d)[0]
    say("[decay] rows past 2^31 elements")
    a = [dlrm_seq_decay_fwd(*far, g, off), *dlrm_seq_decay_bwd(do, *far, g, off)]
    b = [dlrm_seq_decay_fwd(*near, g, off), *dlrm_seq_decay_bwd(do, *near, g, off)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_captured_and_replayed():
    """A training step and a single event, captured; other data and lengths in the same buffers; eager work between."""
    rng = rng_of("decay-graph")
    Hq, Hkv, d, lens = 4, 2, 64, [100, 300, 20]
    off, dev, _, g, (do, _) = problem(rng, lens, Hq, Hkv, d)
    off, g = to_dev(off), to_dev(g)
    state = torch.zeros((3, Hkv, d, d), device=DEV)

    def step():
        o, last = dlrm_seq_decay_fwd(*dev, g, off, state=state, want_state=True)
        return [o, last, *dlrm_seq_decay_bwd(do, *dev, g, off), dlrm_seq_decay_step(*(x[:3] for x in dev), g[:3], last)]

    say("[decay] captured")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for lens in ([100, 300, 20], [1, 0, 419], [140, 140, 140], [420, 0, 0]):
        off.copy_(to_dev(offsets(lens)))
        for t in dev:
            t.copy_(torch.randn(t.shape, device=DEV).bfloat16())
        state.normal_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs]
        for x, y in zip(got, step()):
            assert torch.equal(x, y)


def test_two_streams_at_once():
    """Two calls under way, each with its own workspace, on streams that are not the current one."""
    rng = rng_of("decay-streams")
    jobs = [problem(rng, lens, 2, 1, 64) for lens in ([900, 800], [70] * 30)]
    args = [(do[0], *dev, to_dev(g), to_dev(off)) for off, dev, _, g, do in jobs]
    want = [dlrm_seq_decay_bwd(*a) for a in args]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in jobs], [None, None]
    say("[decay] two streams")
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = dlrm_seq_decay_bwd(*args[i])
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_offsets_that_are_out_of_order():
    """Offsets below 0, past N and falling: no row outside is written, and nothing else is promised."""
    rng = rng_of("decay-offsets")
    N = 200
    q, k, v, do = (bf16(rng, N, 1, 32)[0] for _ in range(4))
    g = to_dev(decays(rng, N, 1, True))
    say("[decay] offsets out of order")
    for off in ([0, 300, 100, 200], [-5, 50, 1 << 40, 60], [200, 100, 0, 0], [10, 10, 10, -1]):
        guard = torch.full((N + 128, 1, 32), 3.0, dtype=torch.bfloat16, device=DEV)
        dlrm_seq_decay_fwd(q, k, v, g, to_dev(np.array(off, np.int64)), out=guard[64:N + 64])
        dlrm_seq_decay_bwd(do, q, k, v, g, to_dev(np.array(off, np.int64)))
        torch.cuda.synchronize()
        assert (guard[:64] == 3).all() and (guard[N + 64:] == 3).all()


def guarded(bytes_, fill):
    """(a buffer's bytes between 4096 of `fill` on either side, what says whether those are as they were); 256-byte aligned."""
    whole = torch.full((bytes_ + 2 * 4096,), fill, dtype=torch.uint8, device=DEV)
    return whole[4096:4096 + bytes_], lambda: bool((whole[:4096] == fill).all() and (whole[4096 + bytes_:] == fill).all())


@pytest.mark.parametrize("N,d,Hq,Hkv", [(200, 32, 1, 1), (200, 128, 4, 2), (3000, 32, 2, 1), (3000, 128, 2, 2)])
@pytest.mark.parametrize("each", [True, False])
def test_offsets_that_are_out_of_order_write_nothing_outside(N, d, Hq, Hkv, each):
    """Of outputs, gradients, states and workspaces, whole sequences and runs of several chunks: each lies between guards."""
    rng = rng_of("decay-guards", N, d)
    q, k, v, do = (bf16(rng, N, h, d)[0] for h in (Hq, Hkv, Hkv, Hq))
    g = to_dev(decays(rng, N, Hkv, each))
    first = to_dev(rng.standard_normal((3, Hkv, d, d)).astype(np.float32))
    say(f"[decay] guards N={N} d={d} each={each}")
    for off in ([0, N + 100, N // 2, N], [-5, N // 4, 1 << 40, N // 3], [N, N // 2, 0, 0], [10, 10, 10, -1], [N // 2, N, 0, N - 1]):
        off = to_dev(np.array(off, np.int64))
        for longest in (1, None):
            desc = binding._seq_decay(q, k, v, g, off, 3, None, longest)[0]
            sizes = [binding.lib().dlrm_seq_decay_fwd_workspace_size(desc), binding.lib().dlrm_seq_decay_bwd_workspace_size(desc)]
            assert (sizes[0] > 256) == (N > 200 and longest is None)  # cut into runs
            spaces = [guarded(n, 0x11) for n in sizes]
            outs = [guarded(2 * t.numel(), 0x22) for t in (q, q, k, v)] + [guarded(4 * g.numel(), 0x22), guarded(4 * first.numel(), 0x22)]
            o, dq, dk, dv = (x[0].view(torch.bfloat16).view(t.shape) for x, t in zip(outs, (q, q, k, v)))
            dg, state = outs[4][0].view(torch.float32).view(g.shape), outs[5][0].view(torch.float32).view(first.shape)
            state.copy_(first)
            dlrm_seq_decay_fwd(q, k, v, g, off, state=state, state_out=state, max_len=longest, out=o, workspace=spaces[0][0])
            dlrm_seq_decay_bwd(do, q, k, v, g, off, max_len=longest, dq=dq, dk=dk, dv=dv, dg=dg, workspace=spaces[1][0])
            torch.cuda.synchronize()
            assert all(left() for _, left in spaces + outs), longest


@pytest.mark.parametrize("lens,Hq,Hkv,d", [([0, 1500, 0, 5], 8, 2, 64), ([5, 0, 2000, 0, 700, 0], 2, 2, 128), ([0, 0, 4000], 4, 1, 32)])
def test_states_in_place_where_sequences_are_cut(lens, Hq, Hkv, d):
    """Empty ones among them keep their states; the rest as apart from the first states, bit by bit, and as in fp64."""
    rng = rng_of("decay-in-place", *lens)
    off, dev, (q, k, v), g, _ = problem(rng, lens, Hq, Hkv, d)
    first = rng.standard_normal((len(lens), Hkv, d, d)).astype(np.float32)
    ref = oracle.decay(q, k, v, g.astype(np.float64), off, float(np.float32(d ** -0.5)), first.astype(np.float64))
    gate, own, off_d = gates(max(lens), d), to_dev(first), to_dev(off)
    assert binding.lib().dlrm_seq_decay_fwd_workspace_size(binding._seq_decay(*dev, to_dev(g), off_d, len(lens), None, max(lens))[0]) > 4096
    say(f"[decay] in place, cut: {lens} d={d}")
    for _ in range(2):
        apart = dlrm_seq_decay_fwd(*dev, to_dev(g), off_d, state=to_dev(first), want_state=True, max_len=max(lens))
        own.copy_(to_dev(first))
        o, last = dlrm_seq_decay_fwd(*dev, to_dev(g), off_d, state=own, state_out=own, max_len=max(lens))
        torch.cuda.synchronize()
        assert last is own and torch.equal(o, apart[0]) and torch.equal(own, apart[1])
    assert rel_err(host(o), ref["o"], ref["o_s"]) <= gate["bf16"]
    assert rel_err(own.cpu().numpy().astype(np.float64), ref["state"], ref["state_s"]) <= gate["state"]
    for b, n in enumerate(lens):
        assert n or np.array_equal(own[b].cpu().numpy(), first[b])
