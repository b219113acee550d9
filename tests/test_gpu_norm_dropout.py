"""GPU parity of the residual norm and of dropout (dlrm_seq.h; needs an MI355X) against oracle/seq.py.

Gates, from the arithmetic (u = 2^-24): s in fp32 has two roundings (the scaling and the sum), 2 u of
its terms; in bf16 (8 significant bits) one more, 2^-8.  rstd: a sum of D squares, at most (64 + 8) u in runs of at most
64 values and 8 joins, and the root's and quotient's u: 2^-17 with room.  y, dx and dresidual: 2^-16 of
their terms in fp32, and 2^-8 more in bf16.  dw: each lane sums M / blocks rows, then the
blocks' sums are added in 32 runs: at most (M / 16 + 64 + 64) u, and its terms' 2^-16.  8-bit: the
value and its scale to 2^-16, rounded to 4 significant bits: 2^-4 of the value, and 2^-10 of the row's
scale below the smallest normal.  Dropout alone is compared bit for bit.
"""
import zlib

import numpy as np
import pytest
import torch

from oracle import seq
from recommendation_model_sparse_amd import (DlrmError, dlrm_add_rmsnorm_bwd, dlrm_add_rmsnorm_fwd, dlrm_dropout, synth)

from gpu_util import DEV, rel_err, say, to_dev

pytestmark = pytest.mark.gpu


def rng_of(*a):
    return np.random.default_rng(zlib.crc32("-".join(map(str, a)).encode()))


def draw(rng, dtype, *shape):
    x = rng.standard_normal(shape).astype(np.float32)
    if dtype == torch.float32:
        return to_dev(x), x.astype(np.float64)
    bits = synth.f32_to_bf16_bits(x)
    return to_dev(bits), synth.bf16_bits_to_f32(bits).astype(np.float64)


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def rounder(dtype):
    if dtype == torch.float32:
        return lambda a: a.astype(np.float32).astype(np.float64)
    return lambda a: synth.bf16_bits_to_f32(synth.f32_to_bf16_bits(a.astype(np.float32))).astype(np.float64)


F, H, E = torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.mark.parametrize("n", [1, 7, 8, 9, 2047, 4096, 10001])
@pytest.mark.parametrize("dtype", [F, H])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_dropout(n, dtype, p):
    rng = rng_of("drop", n, dtype, p)
    x_d, x = draw(rng, dtype, n)
    seed, offset = int(rng.integers(0, 1 << 63)) * 2 + 1, int(rng.integers(0, 1 << 40))
    f = seq.drop_factors(n, p, seed, offset)
    say(f"[drop] n={n} {dtype} p={p}")
    y = dlrm_dropout(x_d, p, seed, offset)
    dev = torch.tensor([offset - 5], dtype=torch.int64, device=DEV)
    y2 = dlrm_dropout(x_d, p, seed, 5, offset_dev=dev)
    same = x_d.clone()
    dlrm_dropout(same, p, seed, offset, out=same)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(y, same)
    # one fp32 product, rounded once more to bf16: the same bits
    assert np.array_equal(host(y), rounder(dtype)(rounder(F)(seq.dropout(x, f))))


def test_dropout_gradient_and_dropped_values():
    """The derivative is the same call on the gradient, and a dropped NaN is 0."""
    rng = rng_of("drop-grad")
    x_d, x = draw(rng, F, 1000)
    g_d, g = draw(rng, F, 1000)
    f = seq.drop_factors(1000, 0.3, 5, 0)
    y, dx = dlrm_dropout(x_d, 0.3, 5), dlrm_dropout(g_d, 0.3, 5)
    step = 0.5 * rng.standard_normal(1000).astype(np.float32)
    moved = (host(dlrm_dropout(to_dev((x + step).astype(np.float32)), 0.3, 5)) - host(y)) * g
    assert abs(moved.sum() - (host(dx) * step).sum()) <= 2.0 ** -20 * np.abs(x * g * f).sum() + 2.0 ** -20 * np.abs(step * g * f).sum()
    x_d[:] = float("nan")
    y = host(dlrm_dropout(x_d, 0.3, 5))
    assert np.array_equal(np.isnan(y), f != 0) and (y[f == 0] == 0).all()


WIDTHS = [1, 7, 8, 100, 128, 129, 136, 250, 256, 479, 512, 520, 1000, 1001, 1024, 1500, 2048, 4095, 4096, 8192, 16384]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("xt,rt,yt,p", [(H, F, H, 0.1), (F, F, F, 0.2), (H, H, H, 0.0), (F, H, H, 0.3), (H, F, F, 0.0)])
@pytest.mark.parametrize("M", [1, 37])
def test_norm(M, D, xt, rt, yt, p):
    rng = rng_of("norm", M, D, xt, rt, yt, p)
    x_d, x = draw(rng, xt, M, D)
    r_d, r = draw(rng, rt, M, D)
    w_d, w = draw(rng, F, D)
    dy_d, dy = draw(rng, yt, M, D)
    ds_d, ds = draw(rng, rt, M, D)
    eps = float(np.float32(1e-5))
    seed, offset = 1234567 + D, 17
    f = seq.drop_factors(M * D, p, seed, offset).reshape(M, D) if p else None
    how = dict(p=p, seed=seed, offset=offset)
    say(f"[norm] M={M} D={D} x={xt} res={rt} y={yt} p={p}")
    s, y, rstd, _ = dlrm_add_rmsnorm_fwd(x_d, r_d, w_d, eps, y_dtype=yt, **how)
    torch.cuda.synchronize()
    exact, _, _, _ = seq.add_rmsnorm(x, r, w, eps, f, rounder(rt))
    terms = np.abs(r) + np.abs(x if f is None else seq.dropout(x, f))
    assert rel_err(host(s), exact, terms) <= 2.0 ** -22 + (2.0 ** -8 if rt == H else 0)
    h = host(s)  # from here on the kept sum is the input
    inv = 1 / np.sqrt((h * h).mean(1) + eps)
    assert rel_err(host(rstd), inv, inv) <= 2.0 ** -17
    ref = h * inv[:, None] * w
    gate = 2.0 ** -16 + (2.0 ** -8 if yt == H else 0)
    assert rel_err(host(y), ref, np.abs(ref)) <= gate
    dx, dres, dw = dlrm_add_rmsnorm_bwd(dy_d, ds_d, s, w_d, rstd, x_dtype=xt, **how)
    torch.cuda.synchronize()
    rdx, rdres, rdw, sc, scw = seq.add_rmsnorm_bwd(dy, ds, h, w, eps, f)
    assert rel_err(host(dres), rdres, sc) <= 2.0 ** -16 + (2.0 ** -8 if rt == H else 0)
    assert np.array_equal(host(dx)[rdx == 0], rdx[rdx == 0]) if f is not None else True
    scale_x = sc if f is None else seq.dropout(sc, f)
    assert rel_err(host(dx), rdx, scale_x) <= 2.0 ** -16 + (2.0 ** -8 if xt == H else 0)
    assert rel_err(host(dw), rdw, scw) <= 2.0 ** -16 + (M / 16 + 128) * 2.0 ** -24
    again = dlrm_add_rmsnorm_bwd(dy_d, ds_d, s, w_d, rstd, x_dtype=xt, **how)
    for a, b in zip((dx, dres, dw), again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("D", [8, 100, 128, 479, 1024, 2048, 4096])
@pytest.mark.parametrize("M", [1, 33])
@pytest.mark.parametrize("xt,rt,p", [(H, H, 0.0), (F, F, 0.1)])
def test_norm_8bit(M, D, xt, rt, p):
    rng = rng_of("norm8", M, D, xt, p)
    x_d, _ = draw(rng, xt, M, D)
    r_d, _ = draw(rng, rt, M, D)
    w_d, w = draw(rng, F, D)
    if M > 1:
        x_d[3] = 0
        r_d[3] = 0  # a row of zeros
    say(f"[norm8] M={M} D={D} {xt} p={p}")
    s, y, rstd, scale = dlrm_add_rmsnorm_fwd(x_d, r_d, w_d, 1e-5, y_dtype=E, p=p, seed=3)
    _, y32, _, none = dlrm_add_rmsnorm_fwd(x_d, r_d, w_d, 1e-5, y_dtype=F, p=p, seed=3)
    torch.cuda.synchronize()
    assert y.dtype == E and none is None
    ref, sc = host(y32), host(scale)
    most = np.abs(ref).max(1)
    assert rel_err(sc, np.where(most == 0, 1.0, most / 448), np.where(most == 0, 1.0, most / 448)) <= 2.0 ** -22
    got = host(y) * sc[:, None]
    assert (np.abs(got - ref) <= 2.0 ** -4 * np.abs(ref) + 2.0 ** -10 * sc[:, None]).all()
    q = host(y)
    assert np.isfinite(q).all() and (np.abs(q).max(1)[most > 0] == 448).all()


def test_norm_without_residual_in_place_and_empty():
    rng = rng_of("norm-none")
    x_d, x = draw(rng, H, 9, 64)
    w_d, w = draw(rng, F, 64)
    s, y, rstd, _ = dlrm_add_rmsnorm_fwd(x_d, None, w_d, 1e-5, res_dtype=F)
    assert torch.equal(s, x_d.float())
    r_d, r = draw(rng, F, 9, 64)
    keep = r_d.clone()
    s2, y2, _, _ = dlrm_add_rmsnorm_fwd(x_d, r_d, w_d, 1e-5, s=r_d)
    s3, y3, rstd3, _ = dlrm_add_rmsnorm_fwd(x_d, keep, w_d, 1e-5)
    assert s2 is r_d and torch.equal(r_d, s3) and torch.equal(y2, y3)
    dy_d, _ = draw(rng, H, 9, 64)
    ds_d, _ = draw(rng, F, 9, 64)
    a = dlrm_add_rmsnorm_bwd(dy_d, ds_d.clone(), s3, w_d, rstd3)
    b = dlrm_add_rmsnorm_bwd(dy_d, ds_d, s3, w_d, rstd3, dresidual=ds_d)
    zero = dlrm_add_rmsnorm_bwd(dy_d, torch.zeros_like(ds_d), s3, w_d, rstd3)
    none = dlrm_add_rmsnorm_bwd(dy_d, None, s3, w_d, rstd3)
    torch.cuda.synchronize()
    for x, y in list(zip(a, b)) + list(zip(zero, none)):
        assert torch.equal(x, y)
    e = torch.empty((0, 64), dtype=H, device=DEV)
    s, y, rstd, _ = dlrm_add_rmsnorm_fwd(e, None, w_d)
    assert s.shape == (0, 64)
    dx, dr, dw = dlrm_add_rmsnorm_bwd(e, None, e, w_d, rstd)
    assert (dw == 0).all()


def test_fused_and_plain_dropout_agree():
    rng = rng_of("norm-drop")
    x_d, _ = draw(rng, F, 13, 479)
    w_d = torch.ones(479, device=DEV)
    s, _, _, _ = dlrm_add_rmsnorm_fwd(x_d, None, w_d, p=0.4, seed=99, offset=7)
    assert torch.equal(s, dlrm_dropout(x_d, 0.4, 99, 7))


def test_many_rows():
    """Rows past what one pass of the backward's workgroups takes."""
    rng = rng_of("norm-many")
    M, D = 70001, 16
    x_d, x = draw(rng, H, M, D)
    w_d, w = draw(rng, F, D)
    dy_d, dy = draw(rng, H, M, D)
    s, y, rstd, _ = dlrm_add_rmsnorm_fwd(x_d, None, w_d, 1e-5, res_dtype=F)
    dx, dres, dw = dlrm_add_rmsnorm_bwd(dy_d, None, s, w_d, rstd, x_dtype=F)
    torch.cuda.synchronize()
    rdx, _, rdw, sc, scw = seq.add_rmsnorm_bwd(dy, np.zeros_like(x), x, w, float(np.float32(1e-5)), None)
    assert rel_err(host(dx), rdx, sc) <= 2.0 ** -16
    assert rel_err(host(dw), rdw, scw) <= 2.0 ** -16 + (M / 16 + 128) * 2.0 ** -24


def test_graph_replay_moves_with_the_offset():
    x = torch.ones(4096, device=DEV)
    at = torch.zeros(1, dtype=torch.int64, device=DEV)
    y = torch.empty_like(x)
    dlrm_dropout(x, 0.5, 11, offset_dev=at, out=y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dlrm_dropout(x, 0.5, 11, offset_dev=at, out=y)
    for step in range(4):
        at.fill_(512 * step)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, dlrm_dropout(x, 0.5, 11, 512 * step))


def test_refusals():
    x = torch.ones((4, 16), device=DEV)
    w = torch.ones(16, device=DEV)
    for bad in (dict(p=-0.1), dict(p=1.5), dict(seed=-1), dict(offset=1 << 64), dict(x=x.half()), dict(x=x.cpu()),
                dict(out=x[:2]), dict(x=x.t()), dict(offset_dev=torch.zeros(1, device=DEV))):
        with pytest.raises(ValueError):
            dlrm_dropout(**{**dict(x=x, p=0.1, seed=1), **bad})
    with pytest.raises(DlrmError):
        dlrm_dropout(torch.ones(64, device=DEV)[1:], 0.1, 1)
    for bad in (dict(x=x[0]), dict(residual=x[:2]), dict(w=w[:8]), dict(w=w.bfloat16()), dict(y_dtype=torch.float16),
                dict(p=2.0), dict(s=x[:2]), dict(residual=x.cpu()), dict(rstd=w)):
        with pytest.raises(ValueError):
            dlrm_add_rmsnorm_fwd(**{**dict(x=x, residual=x, w=w), **bad})
    with pytest.raises(DlrmError):
        dlrm_add_rmsnorm_fwd(x, x, w, -1.0)
    with pytest.raises(DlrmError):
        dlrm_add_rmsnorm_fwd(torch.ones((2, 4097), device=DEV), None, torch.ones(4097, device=DEV))
    s, y, rstd, _ = dlrm_add_rmsnorm_fwd(x, x, w)
    for bad in (dict(dy=x[:2]), dict(ds=x.bfloat16()), dict(rstd=rstd[:2]), dict(x_dtype=torch.float16), dict(dw=w[:2]),
                dict(dx=x[:1])):
        with pytest.raises(ValueError):
            dlrm_add_rmsnorm_bwd(**{**dict(dy=x, ds=x, s=s, w=w, rstd=rstd), **bad})


@pytest.mark.parametrize("D", [8, 100, 128, 4096])
@pytest.mark.parametrize("size", [1e-36, 1e-37])
def test_norm_8bit_rows_near_the_smallest_numbers(D, size):
    """448 / max|y| is past the largest fp32 here; the row's zeros stay zeros.  The scale itself, below the
    smallest normal number, has 2^-17 of room at 1e-37 / 448."""
    rng = rng_of("tiny", D, size)
    x = rng.standard_normal((5, D)).astype(np.float32)
    x[:, ::3] = 0
    w = np.full(D, size, np.float32)
    say(f"[norm8 tiny] D={D} size={size}")
    _, y, _, scale = dlrm_add_rmsnorm_fwd(to_dev(x), None, to_dev(w), 1e-6, y_dtype=E)
    x64 = x.astype(np.float64)
    ref = x64 / np.sqrt((x64 ** 2).mean(1, keepdims=True) + 1e-6) * w.astype(np.float64)
    got, sc = host(y) * host(scale).reshape(-1, 1), np.abs(ref).max(1, keepdims=True) / 448
    assert np.isfinite(got).all() and (got[:, ::3] == 0).all()
    assert (np.abs(got - ref) <= (2.0 ** -4 + 2.0 ** -15) * np.abs(ref) + 2.0 ** -10 * sc).all()


def need(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"{gib} GiB of free memory")


def test_dropout_past_one_launch():
    """2^35 elements are 2^32 work-items: the last ones equal a call on them alone, moved by their offset."""
    need(140)
    n, tail = (1 << 35) + 40005, 1 << 13
    say(f"[drop] n={n}")
    x = torch.empty(n, dtype=H, device=DEV).fill_(1)
    y = dlrm_dropout(x, 0.25, 77, 5, out=x)
    first = n // 8 * 8 - tail
    want = dlrm_dropout(torch.ones(n - first, dtype=H, device=DEV), 0.25, 77, 5 + first // 8)
    assert torch.equal(y[first:], want) and torch.equal(y[:tail], dlrm_dropout(torch.ones(tail, dtype=H, device=DEV), 0.25, 77, 5))
    across = ((1 << 24) - 1) * 256 * 8
    want = dlrm_dropout(torch.ones(2 * tail, dtype=H, device=DEV), 0.25, 77, 5 + (across - tail) // 8)
    seam = y[across - tail:across + tail].clone()
    del x, y
    torch.cuda.empty_cache()
    assert seam.shape == want.shape and torch.equal(seam, want)


def test_norm_past_one_launch():
    """2^28 rows by 16 lanes each are 2^32 work-items."""
    need(40)
    M, D = (1 << 28) + 1037, 8
    say(f"[norm] M={M} D={D}")
    rng = rng_of("norm-launch")
    w_d, _ = draw(rng, F, D)
    x = torch.empty(M, D, dtype=H, device=DEV).fill_(0.5)
    some, _ = draw(rng, H, 400, D)
    x[-400:] = some
    at = ((1 << 24) - 1) * 16 - 200  # the first launch's end
    x[at:at + 400] = some
    _, y, rstd, _ = dlrm_add_rmsnorm_fwd(x, None, w_d, 1e-5)
    _, y1, rstd1, _ = dlrm_add_rmsnorm_fwd(some, None, w_d, 1e-5)
    for a in (at, M - 400):
        assert torch.equal(y[a:a + 400], y1) and torch.equal(rstd[a:a + 400], rstd1)


@pytest.mark.parametrize("M,D,xt", [(4096, 4096, H), (16384, 1024, F), (4096, 2001, F)])
def test_norm_8bit_is_the_quotient(M, D, xt):
    """The 8-bit values are y / y_scale in fp32, rounded once: bit for bit, with the fp32 y that the same
    call gives and the scale as stored."""
    rng = rng_of("norm8-quotient", M, D)
    x_d, _ = draw(rng, xt, M, D)
    w_d, _ = draw(rng, F, D)
    say(f"[norm8] quotient M={M} D={D} {xt}")
    _, q, _, scale = dlrm_add_rmsnorm_fwd(x_d, None, w_d, 1e-5, y_dtype=E)
    _, y, _, _ = dlrm_add_rmsnorm_fwd(x_d, None, w_d, 1e-5, y_dtype=F)
    torch.cuda.synchronize()
    want = (y.cpu() / scale.cpu()[:, None]).to(E)
    off = (q.cpu().view(torch.uint8) != want.view(torch.uint8)).sum().item()
    say(f"   {off} of {M * D} differ")
    assert off == 0


@pytest.mark.parametrize("size", [1e-40, 1e-42, 1e-44])
def test_norm_8bit_rows_below_the_normal_numbers(size):
    """Scales that are a few times the smallest number, or would round to 0: every value is within half of
    448 such steps (the scale's rounding) and an 8-bit step."""
    rng = rng_of("tiny8", size)
    x = rng.standard_normal((5, 256)).astype(np.float32)
    w = np.full(256, size, np.float32)
    say(f"[norm8 below normal] size={size}")
    _, y, _, scale = dlrm_add_rmsnorm_fwd(to_dev(x), None, to_dev(w), 1e-6, y_dtype=E)
    _, y32, _, _ = dlrm_add_rmsnorm_fwd(to_dev(x), None, to_dev(w), 1e-6, y_dtype=F)
    torch.cuda.synchronize()
    sc, ref = scale.cpu().numpy().astype(np.float64), host(y32)
    assert (sc >= 2.0 ** -149).all() and np.isfinite(host(y)).all()
    assert (np.abs(host(y) * sc[:, None] - ref) <= 2.0 ** -4 * np.abs(ref) + 225 * 2.0 ** -149).all()
