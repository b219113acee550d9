"""The fp64 oracle of the user-history operators against torch autograd in fp64, central differences
and published values (CPU)."""
import numpy as np
import pytest
import torch

from oracle import seq
from recommendation_model_sparse_amd import dlrm_seq_bucket_bounds


def jagged(rng, q_lens, k_lens, Hq, Hkv, d):
    qo, ko = np.cumsum([0] + q_lens), np.cumsum([0] + k_lens)
    return (rng.standard_normal((qo[-1], Hq, d)), rng.standard_normal((ko[-1], Hkv, d)), rng.standard_normal((ko[-1], Hkv, d)),
            qo, ko)


@pytest.mark.parametrize("window,sinks", [(0, 0), (3, 0), (3, 2), (1, 1)])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 2)])
def test_attention_against_autograd(window, sinks, Hq, Hkv):
    rng = np.random.default_rng(11)
    q_lens, k_lens, d = [5, 1, 4, 9], [5, 7, 4, 9], 8
    q, k, v, qo, ko = jagged(rng, q_lens, k_lens, Hq, Hkv, d)
    bounds = [0, 1, 2, 5]
    bias, do = rng.standard_normal((Hq, 4)), rng.standard_normal(q.shape)
    r = seq.seq_attn(q, k, v, qo, ko[:-1], ko[1:], window, sinks, 0.4, bias, bounds, do)
    tq, tk, tv, tb = (torch.tensor(x, requires_grad=True) for x in (q, k, v, bias))
    outs = []
    for b in range(len(q_lens)):
        for i in range(q_lens[b]):
            p = k_lens[b] - q_lens[b] + i
            keys = [j for j in range(p + 1) if not window or p - j < window or j < sinks]
            rows = []
            for h in range(Hq):
                g = h * Hkv // Hq
                z = torch.stack([0.4 * (tq[qo[b] + i, h] * tk[ko[b] + j, g]).sum()
                                 + tb[h, max(u for u in range(4) if bounds[u] <= p - j)] for j in keys])
                a = torch.softmax(z, 0)
                rows.append(sum(a[m] * tv[ko[b] + j, g] for m, j in enumerate(keys)))
                assert abs(torch.logsumexp(z, 0).item() - r["lse"][qo[b] + i, h]) < 1e-12
            outs.append(torch.stack(rows))
    o = torch.stack(outs)
    assert np.allclose(o.detach().numpy(), r["o"], rtol=0, atol=1e-12)
    for name, got in zip(("dq", "dk", "dv", "dbias"), torch.autograd.grad(o, (tq, tk, tv, tb), torch.tensor(do))):
        assert np.allclose(got.numpy(), r[name], rtol=0, atol=1e-11), name
        assert (np.abs(r[name]) <= r[name + "_s"] + 1e-12).all()


def test_attention_against_differences():
    rng = np.random.default_rng(5)
    q, k, v, qo, ko = jagged(rng, [6, 3], [6, 8], 2, 1, 8)
    bias, bounds, do = rng.standard_normal((2, 3)), [0, 2, 4], rng.standard_normal(q.shape)
    args = dict(q=q, k=k, v=v, bias=bias)

    def f(**over):
        a = {**args, **over}
        return float((seq.seq_attn(a["q"], a["k"], a["v"], qo, ko[:-1], ko[1:], 4, 1, 0.3, a["bias"], bounds)["o"] * do).sum())

    r = seq.seq_attn(q, k, v, qo, ko[:-1], ko[1:], 4, 1, 0.3, bias, bounds, do)
    for name in args:
        step = rng.standard_normal(args[name].shape)
        e = 1e-5
        slope = (f(**{name: args[name] + e * step}) - f(**{name: args[name] - e * step})) / (2 * e)
        assert abs(slope - float((r["d" + name] * step).sum())) < 1e-7, name


def test_rows_that_see_nothing():
    rng = np.random.default_rng(3)
    q, k, v, qo, ko = jagged(rng, [4, 2, 0], [2, 0, 3], 1, 1, 8)
    r = seq.seq_attn(q, k, v, qo, ko[:-1], ko[1:], do=np.ones_like(q))
    assert (r["o"][:2] == 0).all() and np.isinf(r["lse"][:2]).all() and (r["o"][4:] == 0).all()
    assert np.allclose(r["o"][2, 0], v[0, 0]) and (r["dk"][2:] == 0).all() and (r["dq"][:2] == 0).all()


def test_bucket_bounds():
    for buckets, reach in ((1, 5), (2, 2), (8, 20), (32, 128), (33, 128), (128, 100000), (64, 3)):
        b = dlrm_seq_bucket_bounds(buckets, reach)
        assert len(b) == buckets and b[0] == 0 and all(y > x for x, y in zip(b, b[1:]))
    assert dlrm_seq_bucket_bounds(8, 32) == [0, 1, 2, 3, 4, 8, 16, 32]
    assert seq.bucket_of([0, 1, 2, 3, 4, 8, 16, 32], np.array([0, 3, 4, 7, 8, 31, 32, 99])).tolist() == [0, 3, 4, 4, 5, 6, 7, 7]


def test_philox_known_answers():
    """The known-answer vectors published with the generator."""
    assert seq.philox4x32([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert seq.philox4x32([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert seq.philox4x32([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0]) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_drop_factors():
    f = seq.drop_factors(20000, 0.25, 7, 3)
    assert set(np.unique(f)) == {0.0, float(np.float32(65536 / 49152))}
    assert abs((f == 0).mean() - 0.25) < 5 * np.sqrt(0.25 * 0.75 / 20000)
    assert np.array_equal(seq.drop_factors(100, 0.25, 7, 4), f[8:108])  # the counter moves by 8 elements
    assert (seq.drop_factors(50, 1.0, 1, 0) == 0).all() and (seq.drop_factors(50, 0.0, 1, 0) == 1).all()


def test_norm_against_autograd_and_differences():
    rng = np.random.default_rng(2)
    x, res, w = rng.standard_normal((5, 12)), rng.standard_normal((5, 12)), rng.standard_normal(12)
    dy, ds = rng.standard_normal((5, 12)), rng.standard_normal((5, 12))
    f = seq.drop_factors(60, 0.3, 9, 1).reshape(5, 12)
    s, h, rstd, y = seq.add_rmsnorm(x, res, w, 1e-3, f, lambda a: a)
    dx, dres, dw, _, _ = seq.add_rmsnorm_bwd(dy, ds, h, w, 1e-3, f)
    tx, tr, tw = (torch.tensor(a, requires_grad=True) for a in (x, res, w))
    ts = tr + tx * torch.tensor(f)
    ty = ts * torch.rsqrt((ts * ts).mean(1, keepdim=True) + 1e-3) * tw
    assert np.allclose(ty.detach().numpy(), y, atol=1e-13) and np.allclose(ts.detach().numpy(), s)
    got = torch.autograd.grad((ty * torch.tensor(dy)).sum() + (ts * torch.tensor(ds)).sum(), (tx, tr, tw))
    for a, b in zip(got, (dx, dres, dw)):
        assert np.allclose(a.numpy(), b, atol=1e-12)

    def loss(x, res, w):
        s, _, _, y = seq.add_rmsnorm(x, res, w, 1e-3, f, lambda a: a)
        return float((y * dy).sum() + (s * ds).sum())

    for i, grad in enumerate((dx, dres, dw)):
        a = [x, res, w]
        step = rng.standard_normal(a[i].shape)
        up, down = list(a), list(a)
        up[i], down[i] = a[i] + 1e-5 * step, a[i] - 1e-5 * step
        assert abs((loss(*up) - loss(*down)) / 2e-5 - float((grad * step).sum())) < 1e-7
