"""The history encoder's pages and linear layers (history.py; needs an MI355X): a paged cache against one with a
region for each user; the encoder with linear layers against the same model in fp64 through torch
autograd, and its serving against its training.

Gates: those of test_gpu_history.py.  A linear layer rounds its state's part of an output to bf16 once more and
its heads' norm twice: two roundings a layer on top of seven, sqrt(19) 2^-9 = 0.85 %, within the same fourfold.
Two caches do the same roundings; a visit's sums over keys may be taken in parts, another order: 3 %, as serving has against
training there.
"""
import numpy as np
import pytest
import torch

from recommendation_model_sparse_amd import binding, dlrm_bce_head, dlrm_dropout
from recommendation_model_sparse_amd.history import HistoryEncoder, Shape

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


def far(a, b):
    return float((a.double().cpu() - b.double().cpu()).norm() / b.double().cpu().norm())


def put(a):
    return torch.from_numpy(np.asarray(a)).to(DEV)


def visit(rng, counts, dtype=np.int64):
    off = np.concatenate([[0], np.cumsum(counts)]).astype(dtype)
    return put(rng.integers(0, 500, off[-1])), put(off)


def encoder(**over):
    return HistoryEncoder(Shape(**dict(dict(events=500, D=64, layers=2), **over)), DEV, 5)


def leaves(enc, ids):
    """The encoder's weights and event rows in fp64, by name."""
    leaf = lambda t: t.detach().double().cpu().requires_grad_(True)  # noqa: E731
    p = dict(rows=leaf(enc.table[ids]), w=leaf(enc.w))
    for i, layer in enumerate(enc.layers):
        for name in ("qkv", "out", "up", "down"):
            p[f"{name}{i}"], p[f"{name}_b{i}"] = leaf(layer[name].W16.float()), leaf(layer[name].b)
        for name in ("w1", "w2") + (("g", "wo") if "g" in layer else ("bias",)):
            p[f"{name}{i}"] = leaf(layer[name])
    return p


def norm(s, w, eps=1e-6):
    return s * torch.rsqrt((s * s).mean(-1, keepdim=True) + eps) * w


def reference(enc, p, off, masks, on):
    """The users' vectors in fp64, from the definition: pairs of events with their weights."""
    c, d = enc.c, enc.d
    masks, edge, s = iter(masks), torch.tensor(enc.bounds[1:]), None
    x = p["rows"]
    for i in range(c.layers):
        s = x * next(masks) if s is None else s + x * next(masks)
        qkv = (norm(s, p[f"w1{i}"]) @ p[f"qkv{i}"].T + p[f"qkv_b{i}"]).view(-1, c.Hq + 2 * c.Hkv, d)
        outs = []
        for a, e in zip(off[:-1], off[1:]):
            t = qkv[a:e]
            n = torch.arange(len(t))[:, None] - torch.arange(len(t))[None]
            o = []
            for h in range(c.Hq):
                g = h * c.Hkv // c.Hq
                q, k, v = t[:, h], t[:, c.Hq + g], t[:, c.Hq + c.Hkv + g]
                if i < c.linear:
                    weight = torch.exp(p[f"g{i}"][g] * n.clamp(min=0)) * (n >= 0)
                    o.append(norm((q @ k.T * weight) @ v / d ** 0.5, p[f"wo{i}"], 1e-3))
                else:
                    z = q @ k.T / d ** 0.5 + p[f"bias{i}"][h][torch.bucketize(n, edge, right=True)]
                    o.append(torch.softmax(z.masked_fill(n < 0, -torch.inf), 1) @ v)
            outs.append(torch.cat(o, 1))
        s = s + (torch.cat(outs) @ p[f"out{i}"].T + p[f"out_b{i}"]) * next(masks)
        x = ((norm(s, p[f"w2{i}"]) @ p[f"up{i}"].T + p[f"up_b{i}"]) * on[i]) @ p[f"down{i}"].T + p[f"down_b{i}"]
    s = s + x * next(masks)
    return norm(s, p["w"])[off[1:] - 1]


@pytest.mark.parametrize("linear,layers,p,longest", [(1, 2, 0.0, None), (2, 2, 0.2, 200), (1, 1, 0.0, 200)])
def test_forward_and_gradients_of_linear_layers(linear, layers, p, longest):
    rng = np.random.default_rng(21)
    enc = encoder(layers=layers, linear=linear, hidden=96, buckets=16, reach=64, p=p)
    for layer in enc.layers:
        layer["w1"].copy_(put(1 + 0.2 * rng.standard_normal(64).astype(np.float32)))
        if "g" in layer:
            layer["wo"].copy_(put(1 + 0.2 * rng.standard_normal(16).astype(np.float32)))
    ids, off = visit(rng, [1, 70, 33, 64, 5, 200])
    users, kept = enc.forward(ids, off, longest=longest)
    g = put(rng.standard_normal((6, 64)).astype(np.float32))
    rows, grads, dw = enc.backward(g, kept)
    torch.cuda.synchronize()
    masks, at = [], 0
    for _ in range(2 * layers + 1):
        masks.append(dlrm_dropout(torch.ones((len(ids), 64), device=DEV), p, 5, at).double().cpu())
        at += len(ids) * 64 // 8
    ref = leaves(enc, ids)
    want = reference(enc, ref, off.cpu(), masks, [(x[-1] > 0).double().cpu() for x in kept[3]])
    say(f"[history] {linear} linear of {layers}, p={p}: users {far(users, want.detach()):.2e}")
    assert far(users, want.detach()) <= 0.03
    got = dict(rows=rows, w=dw)
    for i, layer in enumerate(enc.layers):
        for name in ("qkv", "out", "up", "down"):
            got[f"{name}{i}"], got[f"{name}_b{i}"] = layer[name].dW, layer[name].db
        got.update({f"{name}{i}": x for name, x in grads[i].items()})
    assert set(got) == set(ref)
    for name, x in zip(ref, torch.autograd.grad((want * g.double().cpu()).sum(), list(ref.values()))):
        say(f"   {name} {far(got[name], x):.2e}")
        assert far(got[name], x) <= 0.06, name


def test_a_step_moves_every_weight():
    rng = np.random.default_rng(22)
    enc = encoder(linear=1)
    before = [(name, i, layer[name].clone()) for i, layer in enumerate(enc.layers) for name in layer if torch.is_tensor(layer[name])]
    ids, off = visit(rng, [3, 40, 64, 65])
    loss = enc.step(ids, off, put(np.array([0, 1, 1, 0], np.float32)), longest=65)
    assert torch.isfinite(loss).all()
    assert {name for name, _, _ in before} == {"w1", "w2", "bias", "g", "wo"}
    for name, i, x in before:
        assert torch.isfinite(enc.layers[i][name]).all() and not torch.equal(enc.layers[i][name], x), (name, i)


def test_a_decay_pushed_against_0_learns_again():
    """A step that would take decays past 0 leaves them at 0; there they have a gradient, and the next step goes by it.
    (A step is w - lr dw in fp32: lr's rounding, the product's and the sum's, 2^-22 of both terms.)"""
    rng = np.random.default_rng(29)
    enc = encoder(linear=2, Hkv=4, p=0.0)
    ids, off = visit(rng, [30, 40, 64, 65, 10, 100])
    clicks = np.array([0, 1, 1, 0, 1, 0], np.float32)
    decays = lambda: torch.cat([layer["g"].clone() for layer in enc.layers])  # noqa: E731
    for layer in enc.layers:
        layer["g"].fill_(-1e-7)
    enc.step(ids, off, put(clicks))
    first = decays()
    say(f"[history] decays after a step past 0: {first.tolist()}")
    assert (first <= 0).all() and (first == 0).any() and (first < -1e-7).any()
    users, kept = enc.forward(ids, off)
    dx = dlrm_bce_head(users, enc.head.W16.view(-1), enc.head.b, put(1 - clicks))["dx"]
    dg = torch.cat([grads["g"] for grads in enc.backward(dx, kept)[1]])
    assert (dg != 0).all() and (dg[first == 0] > 0).any()
    enc.step(ids, off, put(1 - clicks))
    second = decays()
    say(f"[history] and after the opposite one: {second.tolist()}")
    assert ((second - (first - enc.lr * dg).clamp(max=0)).abs() <= 2.0 ** -22 * (first.abs() + enc.lr * dg.abs())).all()


@pytest.mark.parametrize("page", [8, 64])
@pytest.mark.parametrize("over", [dict(), dict(window=20, sinks=3), dict(linear=1), dict(linear=2), dict(Hq=8, Hkv=1, linear=1),
                                  dict(D=512), dict(D=384, window=20, sinks=3, linear=1)])
def test_pages_give_the_regions_vectors(page, over):
    """Visits with users that come, stay away and come again, then single events, 8-bit ones too."""
    rng = np.random.default_rng(23)
    enc = encoder(**over)
    one, other = enc.cache(5, 160), enc.paged_cache(5, 160, -(-160 // page) * 5, page)
    say(f"[history] pages of {page}, {over}")
    alike = lambda x, y: far(x, y) <= 0.03 and torch.equal((x != 0).any(1), (y != 0).any(1))  # noqa: E731
    for counts in ([30, 1, 0, 64, 100], [0, 7, 65, 1, 0], [0, 0, 0, 0, 0], [1, 0, 8, 0, 9]):
        v = visit(rng, counts, np.int32 if counts[0] else np.int64)
        x, y = one.prefill(*v, 100), other.prefill(*v, 100)
        assert alike(x, y) or not y.any() and torch.equal(x, y), counts
    for i in range(9):
        ids = put(rng.integers(0, 500, 5))
        a, b = one.append(ids, eight_bit=i == 4), other.append(ids, eight_bit=i == 4)
        if i == 4:  # 8 bits: 2^-5 in the mean square, of two rounded values
            (x, s), (y, t) = a, b
            assert far(x.float() * s[:, None], y.float() * t[:, None]) <= 0.08
        else:
            assert alike(a, b), i
    assert torch.equal((one.end - one.begin).cpu(), other.lengths.cpu().long())
    assert (other.held == other.lengths.cpu().numpy()).all()


@pytest.mark.parametrize("linear", [0, 1, 2])
def test_serving_agrees_with_training(linear):
    rng = np.random.default_rng(24)
    enc = encoder(D=128, linear=linear)
    lens = np.array([30, 1, 100, 64, 131])
    ids, off = visit(rng, lens + 3)
    want, _ = enc.forward(ids, off, drop=False)
    cache, o = enc.paged_cache(5, 140, 30, 16), off.cpu().numpy()
    parts = (o[:-1], o[:-1] + lens - lens // 2, o[:-1] + lens)
    for first, end in zip(parts[:-1], parts[1:]):
        at = np.concatenate([np.arange(a, e) for a, e in zip(first, end)])
        cache.prefill(ids[put(at)], put(np.concatenate([[0], np.cumsum(end - first)])), int((end - first).max()))
    for i in range(3):
        got = cache.append(ids[put(o[:-1] + lens + i)])
    say(f"[history] served from pages, {linear} linear layers: {far(got, want):.2e}")
    assert far(got, want) <= 0.03


@pytest.mark.parametrize("linear", [0, 1])
def test_a_user_that_leaves_begins_anew(linear):
    """Its pages go to others, and its next events are encoded as a first visit."""
    rng = np.random.default_rng(25)
    enc = encoder(linear=linear)
    cache, fresh = enc.paged_cache(3, 64, 8, 16), enc.paged_cache(3, 64, 8, 16)
    cache.prefill(*visit(rng, [48, 10, 33]), 48)  # 3 + 1 + 3 pages
    cache.release([0, 2])
    assert int(cache.free_count) == 7 and cache.lengths.tolist() == [0, 10, 0]
    ids, off = visit(rng, [20, 0, 60])
    got, want = cache.prefill(ids, off, 60), fresh.prefill(ids, off, 60)
    assert torch.equal(got, want)
    ids = put(rng.integers(0, 500, 3))
    got, want = cache.append(ids), fresh.append(ids)
    assert torch.equal(got[[0, 2]], want[[0, 2]]) and not torch.equal(got[1], want[1])
    cache.release([])
    assert cache.lengths.tolist() == [21, 11, 61]


def test_what_does_not_fit_is_refused_before_anything_changes():
    rng = np.random.default_rng(26)
    enc = encoder(linear=1)
    cache = enc.paged_cache(3, 64, 6, 16)
    cache.prefill(*visit(rng, [10, 32, 30]), 32)  # 1 + 2 + 2 pages
    held = lambda: [t.clone().view(torch.uint8) for t in (cache.k[1], cache.v[1], cache.state[0], cache.table, cache.lengths, cache.free, cache.free_count)]  # noqa: E731
    before = held()
    ids, off = visit(rng, [1, 2, 3])
    for call in (lambda: cache.prefill(*visit(rng, [55, 0, 0]), 55),      # past the longest
                 lambda: cache.prefill(*visit(rng, [7, 1, 0]), 7),        # past the pool: 2 + 3 + 2
                 lambda: cache.prefill(ids, off, 2),                      # past longest_new
                 lambda: cache.prefill(ids[:-1], off, 3),
                 lambda: cache.prefill(ids, off[:-1], 3),
                 lambda: cache.append(ids[:2]),
                 lambda: cache.release([3]),
                 lambda: cache.release([-1])):
        with pytest.raises(ValueError):
            call()
    for x, y in zip(before, held()):
        assert torch.equal(x, y)
    cache.append(ids[:3])  # 1 + 3 + 2 pages
    assert int(cache.free_count) == 0
    for n in range(15):
        cache.append(ids[:3])
        if cache.held[2] == 32:
            break
    with pytest.raises(ValueError):
        cache.append(ids[:3])
    with pytest.raises(ValueError):
        HistoryEncoder(Shape(events=5, D=64, layers=1, linear=2), DEV)


@pytest.mark.parametrize("call", ["prefill", "append"])
@pytest.mark.parametrize("linear", [0, 1])
@pytest.mark.parametrize("paged", [True, False])
def test_a_visit_that_ends_half_way(monkeypatch, paged, linear, call):
    """A layer that cannot go on: what has come to be part of a history is not served.  Over pages, users leave and begin anew, the
    others go on; regions without linear layers hold what they held, and the visit can be made again."""
    rng = np.random.default_rng(28)
    enc = encoder(linear=linear)
    make = lambda: enc.paged_cache(3, 64, 12, 16) if paged else enc.cache(3, 64)  # noqa: E731
    cache, fresh = make(), make()
    for c in (cache, fresh):
        c.prefill(*visit(np.random.default_rng(1), [20, 0, 33]), 33)
    counts = [5, 0, 7] if call == "prefill" else [1, 1, 1]
    ids, off = visit(rng, counts)
    go = (lambda c: c.prefill(ids, off, 7)) if call == "prefill" else (lambda c: c.append(ids))
    calls = 0

    def fails(*a, real=binding.dlrm_linear_fwd, **k):
        nonlocal calls
        calls += 1
        if calls == 7:  # in the second layer, past its attention
            raise MemoryError("of a test")
        return real(*a, **k)

    with monkeypatch.context() as m:
        m.setattr(binding, "dlrm_linear_fwd", fails)
        with pytest.raises(MemoryError):
            go(cache)
    say(f"[history] half way: paged {paged} linear {linear} {call}")
    if not paged and not linear:
        assert torch.equal(go(cache), go(fresh)) and torch.equal(cache.end, fresh.end)
        return
    for again in (go, lambda c: c.append(ids[:1].expand(3).contiguous()), lambda c: c.prefill(*visit(rng, [0, 0, 0]), 1)):
        with pytest.raises(RuntimeError):
            again(cache)
    if not paged:
        return
    left = [i for i in range(3) if counts[i]]
    cache.release(left[:-1])
    with pytest.raises(RuntimeError):
        go(cache)
    cache.release(left[-1:])
    fresh.release(left)
    for c in (cache, fresh):
        assert c.lengths.tolist() == [0 if n else h for n, h in zip(counts, [20, 0, 33])]
    assert torch.equal(go(cache), go(fresh)) and torch.equal(cache.lengths, fresh.lengths) and cache.held.tolist() == fresh.held.tolist()


@pytest.mark.parametrize("linear", [0, 1])
@pytest.mark.parametrize("paged", [True, False])
def test_what_is_refused_leaves_the_cache_as_it_is(paged, linear):
    """Ids that cannot be, and too few of them: no history changes, and the next visit is served."""
    enc, rng = encoder(linear=linear), np.random.default_rng(30)
    cache = enc.paged_cache(3, 64, 12, 16) if paged else enc.cache(3, 64)
    ids, off = visit(rng, [4, 2, 9])
    for call in (lambda: cache.append(ids[:2]), lambda: cache.append(ids[:3].float()), lambda: cache.prefill(ids.float(), off, 9), lambda: cache.prefill(ids, off, 8)):
        with pytest.raises((ValueError, TypeError)):
            call()
    other = enc.paged_cache(3, 64, 12, 16) if paged else enc.cache(3, 64)
    assert torch.equal(cache.prefill(ids, off, 9), other.prefill(ids, off, 9)) and torch.equal(cache.append(ids[:3]), other.append(ids[:3]))


def test_linear_layers_alone_keep_no_rows():
    """The state of a history longer than any page: no keys, no values, and the vectors of the whole history."""
    rng = np.random.default_rng(27)
    enc = encoder(layers=1, linear=1)
    cache = enc.cache(2, 1000)
    assert cache.k == [None] and cache.state[0].shape == (2, 2, 16, 16)
    ids, off = visit(rng, [700, 131])
    want, _ = enc.forward(ids, off, drop=False)
    cut = np.concatenate([np.arange(0, 699), np.arange(700, 830)])
    cache.prefill(ids[put(cut)], put(np.array([0, 699, 829])), 699)
    assert far(cache.append(ids[put(np.array([699, 830]))]), want) <= 0.03
