"""The history encoder (history.py; needs an MI355X): its forward and gradients against the same model
in fp64 through torch autograd on the CPU, serving against training, and a run that learns.

Gates.  An activation is rounded to bf16 seven times a layer (relative 2^-9 in the mean square each):
over two layers and the final norm sqrt(15) 2^-9 = 0.8 %, and a norm or softmax between them may pass an
error on enlarged, up to fourfold is allowed: 3 % of the output's norm.  Backward has as many roundings
again on top of the forward's: 6 %; the ReLU's mask is a decision taken in floating point, which the
reference takes from the encoder's own forward.  Serving and training do the same roundings in another order of
sums: 3 %.  8-bit vectors: 2^-5 in the mean square (4 significant bits), 4 % more.
"""
import numpy as np
import pytest
import torch

from recommendation_model_sparse_amd.history import HistoryEncoder, Shape, main
from recommendation_model_sparse_amd import dlrm_dropout

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


def far(a, b):
    return float((a.double().cpu() - b.double().cpu()).norm() / b.double().cpu().norm())


def batch(rng, lens, events):
    off = np.concatenate([[0], np.cumsum(lens)])
    return torch.from_numpy(rng.integers(0, events, off[-1])).to(DEV), torch.from_numpy(off).to(DEV)


def reference(enc, ids, off, masks, on):
    """The model in fp64: (leaves by name, users)."""
    c, d = enc.c, enc.d
    leaf = lambda t: t.detach().double().cpu().requires_grad_(True)  # noqa: E731
    p = dict(rows=leaf(enc.table[ids]), w=leaf(enc.w))
    for i, layer in enumerate(enc.layers):
        for name in ("qkv", "out", "up", "down"):
            p[f"{name}{i}"], p[f"{name}_b{i}"] = leaf(layer[name].W16.float()), leaf(layer[name].b)
        for name in ("w1", "w2", "bias"):
            p[f"{name}{i}"] = leaf(layer[name])
    masks = iter(m.double().cpu() for m in masks)
    edge = torch.tensor(enc.bounds[1:])
    norm = lambda s, w: s * torch.rsqrt((s * s).mean(1, keepdim=True) + 1e-6) * w  # noqa: E731
    s = p["rows"] * next(masks)
    for i in range(c.layers):
        if i:
            s = s + x * next(masks)
        qkv = (norm(s, p[f"w1{i}"]) @ p[f"qkv{i}"].T + p[f"qkv_b{i}"]).view(-1, c.Hq + 2 * c.Hkv, d)
        outs = []
        for b in range(len(off) - 1):
            t = qkv[off[b]:off[b + 1]]
            n = torch.arange(len(t))[:, None] - torch.arange(len(t))[None]
            j = torch.arange(len(t))[None].expand_as(n)
            see = (n >= 0) & ((n < c.window) | (j < c.sinks) if c.window else n >= 0)
            o = []
            for h in range(c.Hq):
                g = h * c.Hkv // c.Hq
                z = t[:, h] @ t[:, c.Hq + g].T / d ** 0.5 + p[f"bias{i}"][h][torch.bucketize(n, edge, right=True)]
                o.append(torch.softmax(z.masked_fill(~see, -torch.inf), 1) @ t[:, c.Hq + c.Hkv + g])
            outs.append(torch.cat(o, 1))
        s = s + (torch.cat(outs) @ p[f"out{i}"].T + p[f"out_b{i}"]) * next(masks)
        x = ((norm(s, p[f"w2{i}"]) @ p[f"up{i}"].T + p[f"up_b{i}"]) * on[i]) @ p[f"down{i}"].T + p[f"down_b{i}"]
    s = s + x * next(masks)
    return p, norm(s, p["w"])[off[1:] - 1]


@pytest.mark.parametrize("window,sinks,p", [(0, 0, 0.0), (20, 3, 0.2)])
def test_forward_and_gradients(window, sinks, p):
    rng = np.random.default_rng(7)
    enc = HistoryEncoder(Shape(events=300, D=64, layers=2, Hq=4, Hkv=2, hidden=96, buckets=16, reach=64, window=window,
                               sinks=sinks, p=p), DEV, 3)
    for layer in enc.layers:
        layer["bias"].copy_(torch.from_numpy(rng.standard_normal((4, 16)).astype(np.float32)))
        layer["w1"].copy_(torch.from_numpy(1 + 0.2 * rng.standard_normal(64).astype(np.float32)))
    ids, off = batch(rng, [1, 70, 33, 64, 5], 300)
    users, kept = enc.forward(ids, off)
    g = torch.from_numpy(rng.standard_normal((5, 64)).astype(np.float32)).to(DEV)
    rows, grads, dw = enc.backward(g, kept)
    torch.cuda.synchronize()
    N, masks, at = ids.numel(), [], 0
    for _ in range(5):  # the same numbers, as factors
        masks.append(dlrm_dropout(torch.ones((N, 64), device=DEV), p, 3, at))
        at += N * 64 // 8
    ref, want = reference(enc, ids.cpu(), off.cpu(), masks, [(x[-1] > 0).double().cpu() for x in kept[3]])
    say(f"[history] window={window} p={p}: users {far(users, want.detach()):.2e}")
    assert far(users, want.detach()) <= 0.03
    names = list(ref)
    got = dict(rows=rows, w=dw)
    for i, layer in enumerate(enc.layers):
        for name in ("qkv", "out", "up", "down"):
            got[f"{name}{i}"], got[f"{name}_b{i}"] = layer[name].dW, layer[name].db
        got.update({f"{name}{i}": grads[i][name] for name in ("w1", "w2", "bias")})
    for name, x in zip(names, torch.autograd.grad((want * g.double().cpu()).sum(), [ref[n] for n in names])):
        say(f"   {name} {far(got[name], x):.2e}")
        assert far(got[name], x) <= 0.06, name


def test_serving_agrees_with_training():
    rng = np.random.default_rng(9)
    enc = HistoryEncoder(Shape(events=500, D=128, layers=2, window=40, sinks=2), DEV, 5)
    lens = np.array([30, 1, 100, 64])
    ids, off = batch(rng, lens + 3, 500)
    want, _ = enc.forward(ids, off, drop=False)
    cache = enc.cache(4, 120)
    o = off.cpu().numpy()
    first = np.concatenate([np.arange(a, a + n - n // 2) for a, n in zip(o[:-1], lens)])  # two visits, then single events
    second = np.concatenate([np.arange(a + n - n // 2, a + n) for a, n in zip(o[:-1], lens)])
    for part, counts in ((first, lens - lens // 2), (second, lens // 2)):
        cache.prefill(ids[torch.from_numpy(part).to(DEV)], torch.from_numpy(np.concatenate([[0], np.cumsum(counts)])).to(DEV), int(counts.max()))
    for i in range(3):
        at = torch.from_numpy(o[:-1] + lens + i).to(DEV)
        if i == 2:
            keep = cache.end.clone(), cache.longest
            q, scale = cache.append(ids[at], eight_bit=True)
            cache.end, cache.longest = keep
        got = cache.append(ids[at])
    torch.cuda.synchronize()
    assert got.shape == want.shape and far(got, want) <= 0.03
    assert far(q.float() * scale[:, None], got) <= 0.04
    with pytest.raises(ValueError):
        cache.prefill(ids, off, 100)


def test_it_learns():
    """Guessing the base rate gives the clicks' entropy (0.69 at most); a model that finds the event goes below."""
    first, last = main()
    assert last < 0.75 * first


def serving(rng, users, capacity, **over):
    enc = HistoryEncoder(Shape(events=500, D=64, layers=2, **over), DEV, 5)
    return enc, enc.cache(users, capacity)


def visit(rng, counts, dtype=np.int64):
    off = np.concatenate([[0], np.cumsum(counts)]).astype(dtype)
    return torch.from_numpy(rng.integers(0, 500, off[-1])).to(DEV), torch.from_numpy(off).to(DEV)


def test_prefill_refuses_what_would_leave_a_region():
    """More new events than longest_new says, or than a user's region holds: refused, and no other
    user's keys are touched."""
    rng = np.random.default_rng(11)
    enc, cache = serving(rng, 3, 64)
    cache.prefill(*visit(rng, [10, 20, 30]), 30)
    held = lambda: [t.view(torch.int16).clone() for t in cache.k + cache.v] + [cache.end]  # noqa: E731
    before = held()
    say("[history] prefill past a region")
    for counts, longest in (([60, 1, 1], 1), ([1, 50, 1], 49), ([1, 50, 1], 50)):
        with pytest.raises(ValueError):
            cache.prefill(*visit(rng, counts), longest)
    torch.cuda.synchronize()
    for x, y in zip(before, held()):
        assert torch.equal(x, y)


def test_prefill_refuses_offsets_that_are_not_the_events():
    rng = np.random.default_rng(15)
    enc, cache = serving(rng, 3, 64)
    ids, off = visit(rng, [10, 20, 30])
    say("[history] prefill refusals")
    for i, o in ((ids[:-1], off), (ids, off + 1), (ids, off[:-1]), (ids, off[[0, 2, 1, 3]])):
        with pytest.raises(ValueError):
            cache.prefill(i, o, 30)
    assert torch.equal(cache.end, cache.begin)


def test_prefill_takes_what_fits():
    """The longest history is that of a user, not the sum of the visits' longest."""
    rng = np.random.default_rng(12)
    enc, cache = serving(rng, 2, 64)
    say("[history] prefill of what fits")
    cache.prefill(*visit(rng, [50, 5]), 50)
    cache.prefill(*visit(rng, [5, 50]), 50)
    assert cache.longest == 55
    for _ in range(9):
        cache.append(torch.from_numpy(rng.integers(0, 500, 2)).to(DEV))
    with pytest.raises(ValueError):
        cache.append(torch.from_numpy(rng.integers(0, 500, 2)).to(DEV))


def test_users_without_a_new_event():
    """Their vectors are 0, not another user's; the others' are as without them."""
    rng = np.random.default_rng(13)
    enc, cache = serving(rng, 4, 64)
    first = visit(rng, [10, 20, 30, 5])
    cache.prefill(*first, 30)
    ids, off = visit(rng, [0, 7, 0, 3])
    say("[history] users without a new event")
    got = cache.prefill(ids, off, 7)
    assert (got[[0, 2]] == 0).all() and (got[[1, 3]] != 0).any(1).all()
    assert torch.equal((cache.end - cache.begin).cpu(), torch.tensor([10, 27, 30, 8]))


def test_no_new_event_at_all():
    rng = np.random.default_rng(14)
    enc, cache = serving(rng, 3, 64)
    cache.prefill(*visit(rng, [10, 20, 30]), 30)
    end = cache.end.clone()
    say("[history] no new event at all")
    got = cache.prefill(*visit(rng, [0, 0, 0]), 0)
    assert got.shape == (3, 64) and got.dtype == torch.bfloat16 and (got == 0).all() and torch.equal(cache.end, end)


def test_serving_keeps_no_activations():
    """Twelve layers need no more room for a visit than two: nothing reads a layer's activations again."""
    rng = np.random.default_rng(16)
    room = []
    for layers in (2, 12):
        enc = HistoryEncoder(Shape(events=500, D=128, layers=layers), DEV, 5)
        cache = enc.cache(16, 512)
        ids, off = visit(rng, [256] * 16)
        say(f"[history] room of {layers} layers")
        cache.prefill(ids, off, 256)
        torch.cuda.synchronize()
        held = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        cache.prefill(ids, off, 256)
        torch.cuda.synchronize()
        room.append(torch.cuda.max_memory_allocated() - held)
    say(f"   {room}")
    assert room[1] <= 1.1 * room[0]


def test_prefill_takes_int32_offsets():
    """As training does; the same vectors."""
    rng = np.random.default_rng(17)
    enc, cache = serving(rng, 3, 64)
    ids, off = visit(rng, [10, 20, 30])
    say("[history] int32 offsets")
    want = cache.prefill(ids, off, 30)
    got = enc.cache(3, 64).prefill(ids, off.int(), 30)
    assert torch.equal(got, want)
