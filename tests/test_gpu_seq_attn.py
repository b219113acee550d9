"""GPU parity of attention over jagged histories (dlrm_seq.h; needs an MI355X) against oracle/seq.py.

Error measure: |gpu - oracle| over the sum of the absolute values of the terms (the oracle's scales).
Gates, from the arithmetic, with e = (d + 8) 2^-24 z_s a bound of a logit's error (fp32 products and
sums; z_s the largest sum of a logit's terms), which is a relative error of P:
  - o: P rounded to bf16 (8 significant bits: 2^-8), o too, and e twice (P and its sum):
    2^-7 + 2 e + 2^-16 for exp2 and the fp32 sums;
  - lse: an absolute error of e + 2^-21 z_s + 2^-20;
  - dq, dk: ds rounded to bf16, the result too: 2^-7, and P and dP - delta in fp32: 2^-14 + 4 e; without
    a bias delta comes from o as rounded: 2^-8 more;  dv: P and the result rounded: 2^-7 + 2^-14 + 4 e;
  - dbias: no rounding to bf16: 2^-14 + 4 e.
Inputs are bf16 values, so both sides start from the same numbers.
"""
import zlib

import numpy as np
import pytest
import torch

from oracle import seq
from recommendation_model_sparse_amd import binding
from recommendation_model_sparse_amd import (DlrmError, dlrm_seq_attn_bwd, dlrm_seq_attn_decode, dlrm_seq_attn_fwd,
                                             dlrm_seq_bucket_bounds, synth)

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


def e_of(d, ref):
    return (d + 8) * 2.0 ** -24 * ref["z_s"]


def check_lse(got, ref, e):
    dead = np.isinf(ref["lse"])
    assert np.array_equal(np.isinf(got), dead) and (got[dead] < 0).all()
    if (~dead).any():
        assert np.abs(got[~dead] - ref["lse"][~dead]).max() <= e + 2.0 ** -21 * ref["z_s"] + 2.0 ** -20


LENS = {
    "one": ([1], [1]),
    "few": ([3, 0, 1, 2, 0], [3, 0, 1, 2, 0]),
    "tiles": ([31, 32, 33, 63, 64, 65, 1], [31, 32, 33, 63, 64, 65, 1]),
    "blocks": ([127, 128, 129, 200], [127, 128, 129, 200]),
    "long": ([700, 5, 391], [700, 5, 391]),
    "later": ([3, 64, 130, 1, 40], [90, 200, 131, 77, 40]),     # the queries are the last events
    "blind": ([70, 5, 140, 3], [3, 0, 65, 3]),                  # more queries than keys: the first see none
}
SHAPES = [
    # lens, Hq, Hkv, d, window, sinks, buckets, reach
    ("one", 1, 1, 8, 0, 0, 0, 0), ("one", 4, 2, 64, 1, 1, 8, 20), ("few", 2, 1, 16, 0, 0, 1, 5), ("few", 3, 3, 128, 2, 1, 32, 128),
    ("tiles", 2, 2, 32, 0, 0, 32, 128), ("tiles", 4, 1, 64, 0, 0, 0, 0), ("tiles", 2, 1, 40, 10, 0, 8, 64),
    ("tiles", 2, 2, 128, 33, 3, 33, 40), ("blocks", 2, 2, 64, 0, 0, 32, 64), ("blocks", 4, 2, 96, 64, 70, 64, 150),
    ("blocks", 1, 1, 128, 0, 0, 128, 300), ("long", 2, 1, 64, 100, 4, 32, 128), ("long", 2, 2, 32, 0, 0, 8, 30),
    ("long", 6, 2, 128, 0, 0, 32, 4096), ("long", 1, 1, 64, 1, 0, 4, 4), ("long", 2, 2, 64, 130, 200, 16, 100),
    ("later", 4, 2, 64, 0, 0, 32, 128), ("later", 2, 1, 128, 50, 3, 16, 64), ("later", 2, 2, 32, 64, 64, 0, 0),
    ("blind", 2, 1, 64, 0, 0, 16, 64), ("blind", 4, 4, 32, 20, 2, 8, 16),
]


@pytest.mark.parametrize("lens,Hq,Hkv,d,window,sinks,buckets,reach", SHAPES)
@pytest.mark.parametrize("itype", [np.int64, np.int32])
def test_forward_backward(lens, Hq, Hkv, d, window, sinks, buckets, reach, itype):
    if itype is np.int32 and lens not in ("few", "later"):
        pytest.skip("int32 offsets on two sets of lengths")
    rng = rng_of("seq", lens, Hq, Hkv, d, window, sinks, buckets)
    q_lens, k_lens = LENS[lens]
    qo, ko = offsets(q_lens, itype), offsets(k_lens, itype)
    q_d, q = bf16(rng, qo[-1], Hq, d)
    k_d, k = bf16(rng, ko[-1], Hkv, d)
    v_d, v = bf16(rng, ko[-1], Hkv, d)
    g_d, g = bf16(rng, qo[-1], Hq, d)
    scale = float(np.float32(1.0 / np.sqrt(d)))
    bias = bounds = None
    how = dict(window=window, sinks=sinks, scale=scale)
    if buckets:
        bias, bounds = rng.standard_normal((Hq, buckets)).astype(np.float32), dlrm_seq_bucket_bounds(buckets, reach)
        how.update(bias=to_dev(bias), bounds=bounds)
        bias = bias.astype(np.float64)
    ref = seq.seq_attn(q, k, v, qo, ko[:-1], ko[1:], window, sinks, scale, bias, bounds, g)
    e = e_of(d, ref)
    qo_d, ko_d = to_dev(qo), to_dev(ko)
    say(f"[seq] {lens} Hq={Hq} Hkv={Hkv} d={d} window={window} sinks={sinks} buckets={buckets} {itype.__name__}")
    o1 = dlrm_seq_attn_fwd(q_d, k_d, v_d, qo_d, ko_d, **how)
    torch.cuda.synchronize()
    assert rel_err(host(o1), ref["o"], ref["o_s"]) <= 2.0 ** -7 + 2 * e + 2.0 ** -16
    o, tiles, lse = dlrm_seq_attn_fwd(q_d, k_d, v_d, qo_d, ko_d, for_backward=True, **how)
    torch.cuda.synchronize()
    assert torch.equal(o, o1)
    check_lse(lse.cpu().numpy().astype(np.float64), ref, e)
    got = dlrm_seq_attn_bwd(g_d, q_d, k_d, v_d, o, tiles, lse, qo_d, ko_d, **how)
    again = dlrm_seq_attn_bwd(g_d, q_d, k_d, v_d, o, tiles, lse, qo_d, ko_d, **how)
    torch.cuda.synchronize()
    for name, x, y in zip(("dq", "dk", "dv", "dbias"), got, again):
        if x is None:
            assert name == "dbias" and not buckets
            continue
        assert torch.equal(x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32),
                           y.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32)), name
        err, gate = rel_err(host(x), ref[name], ref[name + "_s"]), (2.0 ** -7 if name != "dbias" else 0) + 2.0 ** -14 + 4 * e
        gate += 2.0 ** -8 if not buckets and name in ("dq", "dk") else 0
        say(f"   {name} {err:.2e} (gate {gate:.2e})")
        assert err <= gate, name


# Biases that differ to where the backward takes another table (256 at heads of 64), and past every table (2048).
LENS["longer"] = ([2500, 3, 320], [2500, 3, 320])


@pytest.mark.parametrize("Hq,Hkv,d,window,sinks,buckets,reach", [
    (2, 1, 64, 0, 0, 64, 250), (2, 1, 64, 0, 0, 64, 300), (2, 2, 64, 0, 0, 64, 4096), (1, 1, 64, 2300, 4, 100, 4096),
    (2, 1, 64, 256, 4, 64, 4096), (2, 1, 64, 257, 4, 64, 4096), (1, 1, 32, 0, 0, 64, 4096), (2, 1, 128, 2300, 70, 64, 4096)])
def test_bias_past_the_table(Hq, Hkv, d, window, sinks, buckets, reach):
    test_forward_backward("longer", Hq, Hkv, d, window, sinks, buckets, reach, np.int64)


def test_gradients_against_differences():
    """The loss <do, o> along a direction of each input: the kernels' gradients against central
    differences of the oracle's forward in fp64 (step 2^-12: its own error is 2^-24 of the third
    derivatives)."""
    rng = rng_of("seq-diff")
    qo = offsets([50, 130, 7])
    q_d, q = bf16(rng, qo[-1], 2, 32)
    k_d, k = bf16(rng, qo[-1], 1, 32)
    v_d, v = bf16(rng, qo[-1], 1, 32)
    g_d, g = bf16(rng, qo[-1], 2, 32)
    bounds, scale = dlrm_seq_bucket_bounds(16, 64), float(np.float32(32 ** -0.5))
    bias = rng.standard_normal((2, 16)).astype(np.float32)
    how = dict(window=60, sinks=2, bias=to_dev(bias), bounds=bounds)
    got = dlrm_seq_attn_bwd(g_d, q_d, k_d, v_d, *dlrm_seq_attn_fwd(q_d, k_d, v_d, to_dev(qo), for_backward=True, **how), to_dev(qo), **how)
    torch.cuda.synchronize()
    at = [q, k, v, bias.astype(np.float64)]
    ref = seq.seq_attn(*at[:3], qo, qo[:-1], qo[1:], 60, 2, scale, at[3], bounds, g)
    e, h = e_of(32, ref), 2.0 ** -12
    for i, name in enumerate(("dq", "dk", "dv", "dbias")):
        step = rng.standard_normal(at[i].shape)
        ends = []
        for sign in (1, -1):
            x = list(at)
            x[i] = at[i] + sign * h * step
            ends.append((seq.seq_attn(*x[:3], qo, qo[:-1], qo[1:], 60, 2, scale, x[3], bounds)["o"] * g).sum())
        slope, want = (ends[0] - ends[1]) / (2 * h), (host(got[i]) * step).sum()
        gate = (2.0 ** -7 if name != "dbias" else 0) + 2.0 ** -14 + 4 * e
        say(f"[seq] {name} slope {slope:.6f} gradient {want:.6f}")
        assert abs(slope - want) <= gate * (ref[name + "_s"] * np.abs(step)).sum()


@pytest.mark.parametrize("lens,Hq,Hkv,d,window,sinks,buckets", [
    ([1500], 4, 1, 32, 0, 0, 8), ([1300, 40], 2, 1, 64, 100, 4, 16), ([900], 8, 2, 128, 64, 70, 32), ([2100], 1, 1, 64, 300, 1, 0),
    ([1100, 0, 700], 2, 2, 40, 256, 128, 8), ([800], 2, 1, 32, 50, 200, 8)])
def test_long_sequences(lens, Hq, Hkv, d, window, sinks, buckets):
    """Few long sequences: key blocks whose queries are split, first keys with a part of their own."""
    rng = rng_of("seq-far", lens, Hq, d, window, sinks)
    qo = offsets(lens)
    q_d, q = bf16(rng, qo[-1], Hq, d)
    k_d, k = bf16(rng, qo[-1], Hkv, d)
    v_d, v = bf16(rng, qo[-1], Hkv, d)
    g_d, g = bf16(rng, qo[-1], Hq, d)
    how, bias, bounds = dict(window=window, sinks=sinks), None, None
    if buckets:
        bias, bounds = rng.standard_normal((Hq, buckets)).astype(np.float32), dlrm_seq_bucket_bounds(buckets, 200)
        how.update(bias=to_dev(bias), bounds=bounds)
        bias = bias.astype(np.float64)
    ref = seq.seq_attn(q, k, v, qo, qo[:-1], qo[1:], window, sinks, float(np.float32(d ** -0.5)), bias, bounds, g)
    e = e_of(d, ref)
    o, tiles, lse = dlrm_seq_attn_fwd(q_d, k_d, v_d, to_dev(qo), for_backward=True, **how)
    got = dlrm_seq_attn_bwd(g_d, q_d, k_d, v_d, o, tiles, lse, to_dev(qo), **how)
    again = dlrm_seq_attn_bwd(g_d, q_d, k_d, v_d, o, tiles, lse, to_dev(qo), **how)
    torch.cuda.synchronize()
    assert rel_err(host(o), ref["o"], ref["o_s"]) <= 2.0 ** -7 + 2 * e + 2.0 ** -16
    for name, x, y in zip(("dq", "dk", "dv", "dbias"), got, again):
        if x is None:
            continue
        assert torch.equal(x, y)
        err, gate = rel_err(host(x), ref[name], ref[name + "_s"]), (2.0 ** -7 if name != "dbias" else 0) + 2.0 ** -14 + 4 * e
        gate += 2.0 ** -8 if not buckets and name in ("dq", "dk") else 0
        say(f"[seq] {lens} {name} {err:.2e} (gate {gate:.2e})")
        assert err <= gate, name


def test_strided_views_of_a_joint_projection():
    rng = rng_of("seq-strided")
    lens, Hq, Hkv, d = [40, 90, 3], 4, 2, 32
    qo = offsets(lens)
    joint_d, joint = bf16(rng, qo[-1], Hq + 2 * Hkv, d)
    qkv = joint_d[:, :Hq], joint_d[:, Hq:Hq + Hkv], joint_d[:, Hq + Hkv:]
    packed = [t.contiguous() for t in qkv]
    g_d, _ = bf16(rng, qo[-1], Hq, d)
    a = dlrm_seq_attn_fwd(*qkv, to_dev(qo), for_backward=True, window=30, sinks=2)
    b = dlrm_seq_attn_fwd(*packed, to_dev(qo), for_backward=True, window=30, sinks=2)
    c = dlrm_seq_attn_bwd(g_d, *qkv, *a, to_dev(qo), window=30, sinks=2)[:3]
    e = dlrm_seq_attn_bwd(g_d, *packed, *b, to_dev(qo), window=30, sinks=2)[:3]
    heads_first = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in packed]  # head stride above the row stride
    f = dlrm_seq_attn_fwd(*heads_first, to_dev(qo), for_backward=True, window=30, sinks=2)
    torch.cuda.synchronize()
    for x, y in list(zip(a, b)) + list(zip(c, e)) + list(zip(f, b)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("d", [32, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 0), (40, 3)])
def test_what_hidden_keys_hold(d, window, sinks):
    """NaN and infinities in a key change nothing for the queries that do not see it, and everything
    for those that do; in the gradient too for keys that no query sees."""
    rng = rng_of("seq-hidden", d, window, sinks)
    n = 150
    qo = to_dev(offsets([n]))
    q_d, _ = bf16(rng, n, 2, d)
    k_d, _ = bf16(rng, n, 1, d)
    v_d, _ = bf16(rng, n, 1, d)
    bias, bounds = to_dev(rng.standard_normal((2, 8)).astype(np.float32)), dlrm_seq_bucket_bounds(8, 32)
    how = dict(window=window, sinks=sinks, bias=bias, bounds=bounds)
    clean = dlrm_seq_attn_fwd(q_d, k_d, v_d, qo, for_backward=True, **how)
    for j, what in ((70, float("nan")), (100, float("inf")), (20, float("-inf")), (149, float("nan"))):
        for hurt_k in (False, True):
            k2, v2 = k_d.clone(), v_d.clone()
            (k2 if hurt_k else v2)[j, 0, 3] = what
            o, tiles, lse = dlrm_seq_attn_fwd(q_d, k2, v2, qo, for_backward=True, **how)
            o1 = dlrm_seq_attn_fwd(q_d, k2, v2, qo, **how)
            torch.cuda.synchronize()
            i = np.arange(n)
            sees = torch.from_numpy((i >= j) & ((window == 0) | (i - j < window) | (j < sinks)))
            assert torch.equal(o.cpu()[~sees], clean[0].cpu()[~sees]), (j, what, hurt_k)
            assert torch.isfinite(o1.cpu()[~sees].float()).all()
            if not hurt_k:
                col = o.cpu()[sees][:, :, 3].float()
                assert (torch.isnan(col) if what != what else col == what).all()
                assert torch.equal(lse.cpu(), clean[2].cpu())
            elif what != what:
                assert torch.isnan(o.cpu()[sees].float()).all()
    if window and not sinks:  # only the last 30 events ask: keys before the window are seen by none
        m = 30
        new = to_dev(offsets([m]))
        ko = to_dev(offsets([n]))
        k2, v2 = k_d.clone(), v_d.clone()
        k2[:n - m - window + 1] = float("nan")
        v2[:n - m - window + 1] = float("inf")
        g_d, _ = bf16(rng, m, 2, d)
        res = []
        for kk, vv in ((k_d, v_d), (k2, v2)):
            o, tiles, lse = dlrm_seq_attn_fwd(q_d[n - m:], kk, vv, new, ko, for_backward=True, **how)
            res.append((o, tiles, lse) + dlrm_seq_attn_bwd(g_d, q_d[n - m:], kk, vv, o, tiles, lse, new, ko, **how))
        torch.cuda.synchronize()
        for x, y in zip(*res):
            assert torch.equal(x, y)
        assert (res[0][4][:n - m - window + 1] == 0).all()


@pytest.mark.parametrize("low", [-1e9, float(torch.finfo(torch.float32).min), -float("inf")])
def test_bias_that_masks(low):
    """A bucket at a mask's usual values: no weight beside other keys; a query whose every key has it
    attends to them evenly (-infinity: to none)."""
    rng = rng_of("seq-mask")
    n, d = 100, 64
    qo = to_dev(offsets([n]))
    q_d, q = bf16(rng, n, 1, d)
    k_d, k = bf16(rng, n, 1, d)
    v_d, v = bf16(rng, n, 1, d)
    g_d, g = bf16(rng, n, 1, d)
    bounds = [0, 1, 20]  # a key's own event is masked: the first query sees nothing else
    bias = np.array([[low, 0.5, -0.25]], np.float32)
    o, tiles, lse = dlrm_seq_attn_fwd(q_d, k_d, v_d, qo, bias=to_dev(bias), bounds=bounds, for_backward=True)
    got = dlrm_seq_attn_bwd(g_d, q_d, k_d, v_d, o, tiles, lse, qo, bias=to_dev(bias), bounds=bounds)
    torch.cuda.synchronize()
    whole = host(o)
    ref = seq.seq_attn(q, k, v, [0, n], [0], [n], 0, 0, float(np.float32(d ** -0.5)), bias.astype(np.float64), bounds, g)
    e = (d + 8) * 2.0 ** -24 * 60  # the unmasked logits' terms
    if low == -float("inf"):
        assert (whole[0] == 0).all() and lse[0, 0].item() == low
    else:
        assert np.array_equal(whole[0], v[0]) and lse[0, 0].item() == np.float32(low)
    assert rel_err(whole[1:], ref["o"][1:], ref["o_s"][1:]) <= 2.0 ** -7 + 2 * e + 2.0 ** -16
    for name, x in zip(("dq", "dk", "dv"), got):
        assert rel_err(host(x), ref[name], ref[name + "_s"]) <= 2.0 ** -7 + 2.0 ** -14 + 4 * e, name


def test_cache_regions_with_gaps():
    """begin and end apart from each other: each user's keys fill the front of a region of its own, the
    rest of which holds NaN."""
    rng = rng_of("seq-gaps")
    lens, cap, d = [100, 0, 37, 64], 128, 64
    begin = np.arange(4) * cap
    end = begin + lens
    new = [5, 2, 37, 1]
    qo = offsets(new)
    q_d, q = bf16(rng, qo[-1], 4, d)
    k_d, k = bf16(rng, 4 * cap, 2, d)
    v_d, v = bf16(rng, 4 * cap, 2, d)
    for b in range(4):
        k_d[end[b]:begin[b] + cap] = float("nan")
        v_d[end[b]:begin[b] + cap] = float("nan")
    scale = float(np.float32(d ** -0.5))
    ref = seq.seq_attn(q, k, v, qo, begin, end, 20, 2, scale)
    o = dlrm_seq_attn_fwd(q_d, k_d, v_d, to_dev(qo), (to_dev(begin), to_dev(end)), window=20, sinks=2)
    last = torch.from_numpy(qo[1:] - 1).to(DEV)
    o1 = dlrm_seq_attn_decode(q_d[last], k_d, v_d, to_dev(begin), to_dev(end), window=20, sinks=2)
    torch.cuda.synchronize()
    gate = 2.0 ** -7 + 2 * e_of(d, ref) + 2.0 ** -16
    assert rel_err(host(o), ref["o"], ref["o_s"]) <= gate
    assert rel_err(host(o1), ref["o"][qo[1:] - 1], ref["o_s"][qo[1:] - 1]) <= gate


DECODE = [
    # lens, Hq, Hkv, d, window, sinks, buckets, reach
    ([1], 1, 1, 8, 0, 0, 0, 0), ([0, 1, 2, 31, 32, 33], 4, 4, 32, 0, 0, 32, 128), ([5, 0, 700], 8, 2, 64, 0, 0, 32, 128),
    ([3000], 4, 1, 128, 0, 0, 32, 512), ([127, 128, 129, 4000], 16, 1, 64, 0, 0, 8, 2000), ([900, 40], 20, 1, 40, 0, 0, 33, 300),
    ([2500, 90, 10], 8, 2, 128, 100, 4, 32, 64), ([2500, 300], 2, 2, 96, 513, 70, 16, 1000), ([600], 2, 1, 64, 1, 0, 4, 9),
    ([5000, 1], 33, 1, 16, 0, 0, 0, 0),
]


@pytest.mark.parametrize("lens,Hq,Hkv,d,window,sinks,buckets,reach", DECODE)
def test_decode(lens, Hq, Hkv, d, window, sinks, buckets, reach):
    rng = rng_of("dec", lens, Hq, Hkv, d, window)
    B, ko = len(lens), offsets(lens)
    q_d, q = bf16(rng, B, Hq, d)
    k_d, k = bf16(rng, ko[-1], Hkv, d)
    v_d, v = bf16(rng, ko[-1], Hkv, d)
    scale = float(np.float32(0.7 / np.sqrt(d)))
    bias = bounds = None
    how = dict(window=window, sinks=sinks, scale=scale)
    if buckets:
        bias, bounds = rng.standard_normal((Hq, buckets)).astype(np.float32), dlrm_seq_bucket_bounds(buckets, reach)
        how.update(bias=to_dev(bias), bounds=bounds)
        bias = bias.astype(np.float64)
    ref = seq.seq_attn(q, k, v, np.arange(B + 1), ko[:-1], ko[1:], window, sinks, scale, bias, bounds)
    gate = 2.0 ** -7 + 2 * e_of(d, ref) + 2.0 ** -16
    for itype in (np.int64, np.int32):
        off = to_dev(ko.astype(itype))
        for longest in (None, 1, max(lens)):  # the split changes; the answer does not, but for rounding
            say(f"[seq] decode {lens} Hq={Hq} Hkv={Hkv} d={d} window={window} longest={longest} {itype.__name__}")
            o = dlrm_seq_attn_decode(q_d, k_d, v_d, off[:-1], off[1:], max_kv_len=longest, **how)
            torch.cuda.synchronize()
            assert rel_err(host(o), ref["o"], ref["o_s"]) <= gate
    # the forward's one-query case is the same operator
    o = dlrm_seq_attn_fwd(q_d, k_d, v_d, to_dev(np.arange(B + 1)), to_dev(ko), **how)
    torch.cuda.synchronize()
    assert rel_err(host(o), ref["o"], ref["o_s"]) <= gate


def test_another_stream():
    rng = rng_of("seq-stream")
    lens = [300, 200]
    qo = to_dev(offsets(lens))
    q_d, _ = bf16(rng, 500, 2, 64)
    k_d, _ = bf16(rng, 500, 2, 64)
    v_d, _ = bf16(rng, 500, 2, 64)
    g_d, _ = bf16(rng, 500, 2, 64)
    bias, bounds = to_dev(rng.standard_normal((2, 8)).astype(np.float32)), dlrm_seq_bucket_bounds(8, 32)

    def both():
        o, tiles, lse = dlrm_seq_attn_fwd(q_d, k_d, v_d, qo, bias=bias, bounds=bounds, for_backward=True)
        return (o, tiles, lse) + dlrm_seq_attn_bwd(g_d, q_d, k_d, v_d, o, tiles, lse, qo, bias=bias, bounds=bounds)

    here = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        there = both()
    side.synchronize()
    for x, y in zip(here, there):
        assert torch.equal(x, y)


def test_nothing_to_do():
    q = torch.empty((0, 2, 32), dtype=torch.bfloat16, device=DEV)
    zero = torch.zeros(1, dtype=torch.int64, device=DEV)
    bias = torch.ones((2, 4), device=DEV)
    o, tiles, lse = dlrm_seq_attn_fwd(q, q, q, zero, bias=bias, bounds=[0, 1, 2, 3], for_backward=True)
    dq, dk, dv, db = dlrm_seq_attn_bwd(q, q, q, q, o, tiles, lse, zero, bias=bias, bounds=[0, 1, 2, 3])
    assert o.shape == q.shape and (db == 0).all()
    three = torch.zeros(4, dtype=torch.int64, device=DEV)  # three empty sequences
    o, tiles, lse = dlrm_seq_attn_fwd(q, q, q, three, bias=bias, bounds=[0, 1, 2, 3], for_backward=True)
    assert (dlrm_seq_attn_bwd(q, q, q, q, o, tiles, lse, three, bias=bias, bounds=[0, 1, 2, 3])[3] == 0).all()
    q1 = torch.ones((3, 2, 32), dtype=torch.bfloat16, device=DEV)
    assert (dlrm_seq_attn_decode(q1, q, q, three[:3], three[1:]) == 0).all()
    assert dlrm_seq_attn_decode(q, q, q, zero[:0], zero[:0]).shape == (0, 2, 32)


def test_refusals():
    rng = rng_of("seq-refuse")
    q, _ = bf16(rng, 10, 4, 32)
    k, _ = bf16(rng, 10, 2, 32)
    off = to_dev(offsets([4, 6]))
    bias = torch.zeros((4, 3), device=DEV)
    ok = dict(q=q, k=k, v=k, q_offsets=off)
    dlrm_seq_attn_fwd(**ok)
    wide, _ = bf16(rng, 10, 1, 136)
    odd, _ = bf16(rng, 10, 2, 12)
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(k=k[:9]), dict(k=k[:, :, :16]), dict(v=k[:, :1]),
                dict(q=q[:, :3]), dict(q_offsets=off.float()), dict(q_offsets=off.cpu()), dict(kv_offsets=off[:2]),
                dict(kv_offsets=off.int()), dict(window=-1), dict(sinks=-2), dict(bias=bias), dict(bounds=[0, 1, 2]),
                dict(bias=bias, bounds=[0, 2, 2]), dict(bias=bias, bounds=[1, 2, 3]), dict(bias=bias, bounds=[0, 1]),
                dict(bias=bias[:2], bounds=[0, 1, 2]), dict(out=q[:5]), dict(out=q.float()), dict(q=wide, k=wide, v=wide),
                dict(q=odd, k=odd, v=odd), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), dict(lse=bias)):
        with pytest.raises(ValueError):
            dlrm_seq_attn_fwd(**{**ok, **bad})
    flat = torch.zeros(10 * 4 * 32 + 8, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(DlrmError):  # 8-byte aligned rows
        dlrm_seq_attn_fwd(**{**ok, "q": flat[4:4 + 1280].view(10, 4, 32)})
    o, tiles, lse = dlrm_seq_attn_fwd(**ok, for_backward=True)
    good = dict(dout=q, **ok, o=o, tiles=tiles, lse=lse)
    dlrm_seq_attn_bwd(**good)
    for bad in (dict(dout=q[:5]), dict(o=o.float()), dict(lse=lse[:, :2]), dict(dbias=bias), dict(dk=q), dict(dq=k), dict(tiles=tiles[1:]), dict(tiles=tiles.long()),
                dict(kv_offsets=(off[:-1], off[1:])), dict(workspace=torch.zeros(4, device=DEV))):
        with pytest.raises(ValueError):
            dlrm_seq_attn_bwd(**{**good, **bad})
    one = dict(q=q[:2], k=k, v=k, kv_begin=off[:-1], kv_end=off[1:])
    dlrm_seq_attn_decode(**one)
    for bad in (dict(q=q[:3]), dict(kv_begin=off), dict(kv_end=off[1:].int()), dict(max_kv_len=-1), dict(out=q)):
        with pytest.raises(ValueError):
            dlrm_seq_attn_decode(**{**one, **bad})


@pytest.mark.parametrize("Hq,Hkv,d,window,sinks,buckets", [(1, 1, 32, 0, 0, 0), (4, 1, 64, 0, 0, 8), (2, 2, 128, 100, 4, 8)])
def test_no_keys_at_all(Hq, Hkv, d, window, sinks, buckets):
    """Queries over k and v of no rows, as many as have a key block's queries split: o and every gradient are 0."""
    rng = rng_of("seq-keyless", Hq, d)
    n = 1200
    qo, ko = to_dev(offsets([n])), to_dev(offsets([0]))
    q_d, _ = bf16(rng, n, Hq, d)
    g_d, _ = bf16(rng, n, Hq, d)
    k = torch.empty((0, Hkv, d), dtype=torch.bfloat16, device=DEV)
    how = dict(window=window, sinks=sinks)
    if buckets:
        how.update(bias=to_dev(rng.standard_normal((Hq, buckets)).astype(np.float32)), bounds=dlrm_seq_bucket_bounds(buckets, 64))
    say(f"[seq] no keys, Hq={Hq} d={d}")
    o, tiles, lse = dlrm_seq_attn_fwd(q_d, k, k, qo, ko, for_backward=True, **how)
    dq, dk, dv, dbias = dlrm_seq_attn_bwd(g_d, q_d, k, k, o, tiles, lse, qo, ko, **how)
    torch.cuda.synchronize()
    assert (o == 0).all() and (lse == -float("inf")).all() and (dq == 0).all()
    assert dk.shape == k.shape and dv.shape == k.shape and (dbias is None or (dbias == 0).all())


@pytest.mark.parametrize("buckets", [0, 4])
def test_keys_that_nobody_asks(buckets):
    """Keys without any query: gradients of 0.  The C call takes no tiles then, as the forward writes none."""
    n, Hkv, d = 200, 2, 64
    q = torch.empty((0, 4, d), dtype=torch.bfloat16, device=DEV)
    k = torch.ones((n, Hkv, d), dtype=torch.bfloat16, device=DEV)
    none, ko = torch.zeros(3, dtype=torch.int64, device=DEV), to_dev(offsets([70, 130]))
    bias = torch.ones((4, 4), device=DEV) if buckets else None
    a, edges, dev, _, _ = binding._seq_attn(q, k, k, none, ko[:-1], ko[1:], 2, 50, 3, None, bias, [0, 1, 2, 3] if buckets else None)
    L = binding.lib()
    dk, dv = torch.full_like(k, 7), torch.full_like(k, 7)
    dbias = torch.full((4, 4), 7.0, device=DEV) if buckets else None
    ws = torch.empty(L.dlrm_seq_attn_bwd_workspace_size(a), dtype=torch.uint8, device=DEV)
    at = binding._ptr
    say(f"[seq] no queries, buckets={buckets}")
    assert L.dlrm_seq_attn_bwd(a, None, None, None, None, None, at(dk), at(dv), at(dbias), at(ws), ws.numel(), binding._stream(dev)) == 0
    torch.cuda.synchronize()
    assert (dk == 0).all() and (dv == 0).all() and (dbias is None or (dbias == 0).all())


@pytest.mark.parametrize("lens,Hq,Hkv,d", [([1500], 4, 1, 32), ([900], 8, 2, 128), ([40, 90], 2, 2, 64)])
def test_rows_outside_every_sequence(lens, Hq, Hkv, d):
    """Rows before the first offset and from the last on keep what the outputs held, whether a key block's
    queries are split (the first two) or not; the others are those of tensors without such rows."""
    rng = rng_of("seq-padding", lens, Hq, d)
    n, lead, trail = sum(lens), 37, 50
    inner = slice(lead, lead + n)
    qo = to_dev(offsets(lens))
    q_d, _ = bf16(rng, lead + n + trail, Hq, d)
    k_d, _ = bf16(rng, lead + n + trail, Hkv, d)
    v_d, _ = bf16(rng, lead + n + trail, Hkv, d)
    g_d, _ = bf16(rng, lead + n + trail, Hq, d)
    say(f"[seq] padding {lens} Hq={Hq} d={d}")
    ws = torch.full((64 << 20,), 0x7f, dtype=torch.uint8, device=DEV)  # what an earlier call may have left there
    out = [torch.full_like(t, 7.0) for t in (q_d, q_d, k_d, v_d)]
    o, tiles, lse = dlrm_seq_attn_fwd(q_d, k_d, v_d, qo + lead, for_backward=True, out=out[0])
    dlrm_seq_attn_bwd(g_d, q_d, k_d, v_d, o, tiles, lse, qo + lead, dq=out[1], dk=out[2], dv=out[3], workspace=ws)
    packed = [t[inner].contiguous() for t in (q_d, k_d, v_d)]
    kept = dlrm_seq_attn_fwd(*packed, qo, for_backward=True)
    want = (kept[0],) + dlrm_seq_attn_bwd(g_d[inner].contiguous(), *packed, *kept, qo)[:3]
    torch.cuda.synchronize()
    for name, x, y in zip(("o", "dq", "dk", "dv"), out, want):
        assert torch.equal(x[inner], y), name
        assert (x[:lead] == 7).all() and (x[lead + n:] == 7).all(), name


@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("j", [0, 20, 32, 70, 149])
def test_lse_of_what_sees_nan(d, j):
    """A NaN in a key is in the lse of the queries that see it, at either half of a tile, and in no other's."""
    rng = rng_of("seq-lse", d, j)
    n = 150
    qo = to_dev(offsets([n]))
    q_d, _ = bf16(rng, n, 2, d)
    k_d, _ = bf16(rng, n, 1, d)
    v_d, _ = bf16(rng, n, 1, d)
    clean = dlrm_seq_attn_fwd(q_d, k_d, v_d, qo, for_backward=True)
    k_d[j, 0, 3] = float("nan")
    say(f"[seq] lse d={d} j={j}")
    o, _, lse = dlrm_seq_attn_fwd(q_d, k_d, v_d, qo, for_backward=True)
    torch.cuda.synchronize()
    assert torch.isnan(lse[j:]).all() and torch.isnan(o[j:].float()).all()
    assert torch.equal(lse[:j], clean[2][:j]) and torch.equal(o[:j], clean[0][:j])


@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
@pytest.mark.parametrize("hurt", [False, True])
def test_values_near_the_largest(d, window, sinks, hurt):
    """An output is a mean of its values: finite however large they are, though their sum before the
    division is not; with a NaN in a key beside them (hurt), for the queries that do not see it."""
    rng = rng_of("seq-big", d, window)
    n, j = 150, 100
    qo = offsets([n])
    q_d, q = bf16(rng, n, 2, d)
    k_d, k = bf16(rng, n, 1, d)
    v_d, _ = bf16(rng, n, 1, d)
    bits = synth.f32_to_bf16_bits((3e38 * rng.uniform(-1, 1, (n, 1, d))).astype(np.float32))
    b_d, b = to_dev(bits), synth.bf16_bits_to_f32(bits).astype(np.float64)
    scale = float(np.float32(2.0 / np.sqrt(d)))  # maxima that move: the reference starts up to 8 below
    how = dict(window=window, sinks=sinks, scale=scale)
    ref = seq.seq_attn(q, k, b, qo, qo[:-1], qo[1:], window, sinks, scale)
    if hurt:
        k_d[j, 0, 3] = float("nan")
    say(f"[seq] large values d={d} window={window} hurt={hurt}")
    o, _, lse = dlrm_seq_attn_fwd(q_d, k_d, b_d, to_dev(qo), for_backward=True, **how)
    _, _, lse0 = dlrm_seq_attn_fwd(q_d, k_d, v_d, to_dev(qo), for_backward=True, **how)
    torch.cuda.synchronize()
    i = np.arange(n)
    free = ~((i >= j) & ((window == 0) | (i - j < window))) if hurt else np.ones(n, bool)
    gate = 2.0 ** -7 + 2 * e_of(d, ref) + 2.0 ** -16
    assert rel_err(host(o)[free], ref["o"][free], ref["o_s"][free]) <= gate
    assert torch.equal(lse.cpu()[torch.from_numpy(free)], lse0.cpu()[torch.from_numpy(free)])  # the values are not in it


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("longest", [1, 5000])
def test_decode_of_values_near_the_largest(d, longest):
    """As above for one event, unsplit and split."""
    rng = rng_of("dec-big", d)
    ko = offsets([1, 40, 5000])
    q_d, q = bf16(rng, 3, 4, d)
    k_d, k = bf16(rng, ko[-1], 2, d)
    bits = synth.f32_to_bf16_bits((3e38 * rng.uniform(0.5, 1, (ko[-1], 2, d))).astype(np.float32))
    v_d, v = to_dev(bits), synth.bf16_bits_to_f32(bits).astype(np.float64)
    ref = seq.seq_attn(q, k, v, np.arange(4), ko[:-1], ko[1:], 0, 0, float(np.float32(1 / np.sqrt(d))))
    say(f"[seq] decode of large values d={d} longest={longest}")
    o = dlrm_seq_attn_decode(q_d, k_d, v_d, to_dev(ko[:-1]), to_dev(ko[1:]), max_kv_len=longest)
    torch.cuda.synchronize()
    assert rel_err(host(o), ref["o"], ref["o_s"]) <= 2.0 ** -7 + 2 * e_of(d, ref) + 2.0 ** -16


def test_decode_past_one_launch_of_the_join():
    """2^24 rows of a head are 2^32 work-items in the join of a sequence's runs, and so more than one launch.
    max_kv_len only chooses the split: unsplit, the same sequences give the same, but for the output's rounding
    (2^-7 of it) and that of sums near 0."""
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("8 GiB of free memory")
    rng = rng_of("dec-join")
    B, Hq, d = (1 << 21) + 3, 8, 8
    few, _ = bf16(rng, 1021, Hq, d)
    q = few.repeat(B // 1021 + 1, 1, 1)[:B]
    k, _ = bf16(rng, 64, 1, d)
    v, _ = bf16(rng, 64, 1, d)
    begin = torch.arange(B, device=DEV) % 50
    end = begin + 1 + torch.arange(B, device=DEV) % 7
    say(f"[seq] decode B={B} Hq={Hq}")
    got = dlrm_seq_attn_decode(q, k, v, begin, end, max_kv_len=(1 << 20) + 1)
    torch.cuda.synchronize()
    want = dlrm_seq_attn_decode(q, k, v, begin, end, max_kv_len=10)
    torch.cuda.synchronize()
    most = float(v.abs().max())
    for a, b in zip(got.split(1 << 18), want.split(1 << 18)):
        assert ((a.float() - b.float()).abs() <= 2.0 ** -7 * b.float().abs() + 2.0 ** -16 * most).all()


def test_one_row_of_heads_far_apart():
    """A tensor of one row has no row stride to refuse: heads 2^22 elements apart, forward and for one event."""
    rng = rng_of("seq-one-row")
    H, d = 4, 64
    far = torch.zeros((H, (1 << 22) // d, d), dtype=torch.bfloat16, device=DEV)
    q_d, _ = bf16(rng, 1, H, d)
    k_d, _ = bf16(rng, 1, H, d)
    v_d, _ = bf16(rng, 90, H, d)
    far[:, :1] = q_d.transpose(0, 1)
    q2 = far.transpose(0, 1)[:1]
    one, off = to_dev(offsets([1])), to_dev(offsets([90]))
    say("[seq] one row of far heads")
    a = dlrm_seq_attn_fwd(q2, v_d, v_d, one, off), dlrm_seq_attn_decode(q2, v_d, v_d, off[:1], off[1:])
    b = dlrm_seq_attn_fwd(q_d, v_d, v_d, one, off), dlrm_seq_attn_decode(q_d, v_d, v_d, off[:1], off[1:])
    far[:, :1] = k_d.transpose(0, 1)
    c, e = dlrm_seq_attn_fwd(q_d, q2, q2, one), dlrm_seq_attn_fwd(q_d, k_d, k_d, one)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(c, e)


@pytest.mark.parametrize("d,buckets", [(32, 8), (64, 0), (64, 8), (96, 8), (128, 0), (128, 8)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
def test_gradients_beside_hidden_keys(d, buckets, window, sinks):
    """NaN and infinities in a key change nothing in dq of the queries that do not see it."""
    rng = rng_of("seq-hidden-grad", d, buckets, window)
    n = 200
    qo = to_dev(offsets([n]))
    q_d, _ = bf16(rng, n, 2, d)
    k_d, _ = bf16(rng, n, 1, d)
    v_d, _ = bf16(rng, n, 1, d)
    g_d, _ = bf16(rng, n, 2, d)
    how = dict(window=window, sinks=sinks)
    if buckets:
        how.update(bias=to_dev(rng.standard_normal((2, buckets)).astype(np.float32)), bounds=dlrm_seq_bucket_bounds(buckets, 32))
    clean = dlrm_seq_attn_fwd(q_d, k_d, v_d, qo, for_backward=True, **how)
    dq0 = dlrm_seq_attn_bwd(g_d, q_d, k_d, v_d, *clean, qo, **how)[0]
    i = np.arange(n)
    for j, what in ((130, float("nan")), (70, float("inf")), (32, float("-inf")), (199, float("nan"))):
        for hurt_k in (False, True):
            k2, v2 = k_d.clone(), v_d.clone()
            (k2 if hurt_k else v2)[j, 0, 3] = what
            say(f"[seq] hidden gradients d={d} buckets={buckets} window={window} j={j} {what} k={hurt_k}")
            kept = dlrm_seq_attn_fwd(q_d, k2, v2, qo, for_backward=True, **how)
            dq = dlrm_seq_attn_bwd(g_d, q_d, k2, v2, *kept, qo, **how)[0]
            torch.cuda.synchronize()
            free = torch.from_numpy(~((i >= j) & ((window == 0) | (i - j < window) | (j < sinks))))
            assert torch.equal(dq.cpu()[free], dq0.cpu()[free]), (j, what, hurt_k)


def test_rows_past_32_bits():
    """Keys and queries past 2^31 elements of their tensors."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("60 GiB of free memory")
    rng = rng_of("seq-far-rows")
    Hq, Hkv, d, n = 2, 2, 64, 300
    rows = (1 << 31) // (Hkv * d) + 1000
    k = torch.zeros((rows, Hkv, d), dtype=torch.bfloat16, device=DEV)
    v = torch.zeros((rows, Hkv, d), dtype=torch.bfloat16, device=DEV)
    q_d, q = bf16(rng, n, Hq, d)
    k_d, kh = bf16(rng, n, Hkv, d)
    v_d, vh = bf16(rng, n, Hkv, d)
    g_d, g = bf16(rng, n, Hq, d)
    k[rows - n:], v[rows - n:] = k_d, v_d
    ref = seq.seq_attn(q, kh, vh, [0, n], [0], [n], 50, 3, float(np.float32(d ** -0.5)), do=g)
    e = e_of(d, ref)

    def check(o, dq, dk, dv):
        torch.cuda.synchronize()
        assert rel_err(host(o), ref["o"], ref["o_s"]) <= 2.0 ** -7 + 2 * e + 2.0 ** -16
        for name, x in (("dq", dq), ("dk", dk), ("dv", dv)):
            gate = 2.0 ** -7 + 2.0 ** -14 + 4 * e + (2.0 ** -8 if name != "dv" else 0)
            assert rel_err(host(x), ref[name], ref[name + "_s"]) <= gate, name

    say(f"[seq] rows past 32 bits: {rows}")
    how = dict(window=50, sinks=3)
    qo, one = to_dev(offsets([n])), to_dev(np.array([rows - n, rows]))
    kept = dlrm_seq_attn_fwd(q_d, k, v, qo, one, for_backward=True, **how)
    dq, dk, dv, _ = dlrm_seq_attn_bwd(g_d, q_d, k, v, *kept, qo, one, **how)
    check(kept[0], dq, dk[rows - n:], dv[rows - n:])
    last = dlrm_seq_attn_decode(q_d[-1:], k, v, one[:1], one[1:], max_kv_len=n, **how)
    torch.cuda.synchronize()
    assert rel_err(host(last), ref["o"][-1:], ref["o_s"][-1:]) <= 2.0 ** -7 + 2 * e + 2.0 ** -16
    del dk, dv
    wide = torch.zeros((rows, Hq, d), dtype=torch.bfloat16, device=DEV)
    grad = torch.zeros_like(wide)
    wide[rows - n:], grad[rows - n:] = q_d, g_d
    kept = dlrm_seq_attn_fwd(wide, k_d, v_d, one, qo, for_backward=True, **how)
    dq, dk, dv, _ = dlrm_seq_attn_bwd(grad, wide, k_d, v_d, *kept, one, qo, **how)
    check(kept[0][rows - n:], dq[rows - n:], dk, dv)


def test_graph_replays():
    """A training pass and a step of serving, captured; every replay is the eager result for the inputs as they
    are then, with eager work and other lengths between the replays."""
    rng = rng_of("seq-graph")
    total, H, d = 500, 4, 64
    q, k, v, g = (bf16(rng, total, H, d)[0] for _ in range(4))
    bias, bounds = to_dev(rng.standard_normal((H, 8)).astype(np.float32)), dlrm_seq_bucket_bounds(8, 64)
    off = to_dev(offsets([300, 120, 80]))
    how = dict(window=100, sinks=2, bias=bias, bounds=bounds)

    def train():
        kept = dlrm_seq_attn_fwd(q, k, v, off, for_backward=True, **how)
        return kept + dlrm_seq_attn_bwd(g, q, k, v, *kept, off, **how) + (
            dlrm_seq_attn_decode(q[:3], k, v, off[:-1], off[1:], max_kv_len=total, **how),)

    train()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = train()
    for lens in ([300, 120, 80], [10, 490, 0], [1, 2, 497], [300, 120, 80]):
        off.copy_(to_dev(offsets(lens)))
        say(f"[seq] replay {lens}")
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = train()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
