"""An encoder of user histories, trained and served on one GPU, as a sequence of the library's calls.

A bag pools a user's ids without their order; this module encodes the events in their order.  Each
event's row is looked up (one-hot bags of one table), a stack of pre-norm layers follows -- RMS norm,
causal attention over the user's own history with a learned bias by distance buckets, RMS norm, two
fully connected layers -- and the last event's vector, after a final norm, is the user's: input of a
sigmoid head here, or one more row of the dot-product interaction.

    s = dropout(event rows)
    s = s + dropout(Wo attn(Wqkv norm(s)));  s = s + dropout(W2 relu(W1 norm(s)))      per layer
    user = norm(s)[last event]

Like dlrm_step, it only orders the calls and owns the weights: every step runs in the library's
kernels, but for what moves data: torch indexes rows, and in the backward joins dq, dk and dv and
casts them.  The residual stream is fp32, activations and the dense layers' weights bf16 with fp32
masters (SGD), the table is updated by row-wise Adagrad.  Histories are jagged: event rows laid end
to end, with offsets [B + 1].

Serving keeps each layer's keys and values in a region of `capacity` rows a user: `prefill` encodes the
events since the last visit against them, `append` one new event a user, and `append(eight_bit=True)`
gives the users' vectors as 8-bit rows with scales for a store of candidates.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Dict, List, Optional, Tuple

import numpy as np
import torch

from . import binding as L


class _Dense:
    """W [N][K] (fp32 master, bf16 copy) and b [N], and their gradients."""

    def __init__(self, rng, N: int, K: int, dev):
        a = 1.0 / np.sqrt(K)
        self.W32 = torch.from_numpy(rng.uniform(-a, a, (N, K)).astype(np.float32)).to(dev)
        self.W16 = self.W32.to(torch.bfloat16)
        self.b = torch.zeros(N, device=dev)
        self.dW, self.db = torch.empty_like(self.W32), torch.empty_like(self.b)

    def fwd(self, x, act=L.DLRM_ACT_NONE):
        return L.dlrm_linear_fwd(x, self.W16, self.b, act)

    def bwd(self, dy, x, y=None, act=L.DLRM_ACT_NONE):
        return L.dlrm_linear_bwd(dy, y, act, x, self.W16, dW=self.dW, db=self.db)[0]

    def params(self):
        return [(self.W32, self.W16, self.dW), (self.b, None, self.db)]


@dataclass
class Shape:
    events: int          # rows of the event table
    D: int = 128         # width of the events and the encoder
    layers: int = 2
    Hq: int = 4
    Hkv: int = 2
    hidden: int = 256
    buckets: int = 32    # distance buckets of the attention bias, up to `reach`
    reach: int = 128
    window: int = 0      # 0: the whole history
    sinks: int = 0
    p: float = 0.1       # dropout


class HistoryEncoder:
    def __init__(self, shape: Shape, dev, seed: int = 0, lr: float = 0.1, lr_emb: float = 0.05, eps_emb: float = 1e-8):
        self.c, self.dev, self.lr, self.lr_emb, self.eps_emb, self.seed = shape, dev, lr, lr_emb, eps_emb, seed
        c = shape
        if c.D % c.Hq or c.D // c.Hq % 8:
            raise ValueError(f"D must be {c.Hq} heads of a multiple of 8 columns, got {c.D}")
        self.d = c.D // c.Hq
        self.bounds = L.dlrm_seq_bucket_bounds(c.buckets, c.reach)
        rng = np.random.default_rng(seed)
        self.table = torch.from_numpy(rng.standard_normal((c.events, c.D)).astype(np.float32)).to(dev)
        self.state = torch.zeros(c.events, device=dev)
        wide = (c.Hq + 2 * c.Hkv) * self.d
        self.layers: List[Dict] = [dict(qkv=_Dense(rng, wide, c.D, dev), out=_Dense(rng, c.D, c.D, dev),
                                        up=_Dense(rng, c.hidden, c.D, dev), down=_Dense(rng, c.D, c.hidden, dev),
                                        w1=torch.ones(c.D, device=dev), w2=torch.ones(c.D, device=dev),
                                        bias=torch.zeros((c.Hq, c.buckets), device=dev)) for _ in range(c.layers)]
        self.w = torch.ones(c.D, device=dev)
        self.head = _Dense(rng, 1, c.D, dev)
        self.counter = 0  # groups of 8 random numbers used so far

    # ------------------------------------------------------------------ the parts

    def _events(self, ids: torch.Tensor) -> torch.Tensor:
        one = torch.arange(ids.numel() + 1, dtype=torch.int64, device=self.dev)
        return L.emb_bag_fwd([self.table], ids, one).view(-1, self.c.D)

    def _norm(self, x, s, w, drop, **how):
        """The next sum and its norm, with fresh dropout numbers when training; the numbers are noted."""
        spec = dict(p=0.0)
        if drop and self.c.p:
            spec = dict(p=self.c.p, seed=self.seed, offset=self.counter)
            self.counter += (x.numel() + 7) // 8
        s, y, rstd, scale = L.dlrm_add_rmsnorm_fwd(x, s, w, res_dtype=torch.float32, **spec, **how)
        return s, y, (s, rstd, spec), scale

    def _how(self, layer):
        return dict(window=self.c.window, sinks=self.c.sinks, bias=layer["bias"], bounds=self.bounds)

    def _split(self, qkv):
        x = qkv.view(-1, self.c.Hq + 2 * self.c.Hkv, self.d)
        return x[:, :self.c.Hq], x[:, self.c.Hq:self.c.Hq + self.c.Hkv], x[:, self.c.Hq + self.c.Hkv:]

    def _layers(self, x, attend, drop=False, keep=False):
        """The layers over event rows x; attend(i, layer, q, k, v) gives the attention's output and what
        its backward wants.  Returns the last sum's branch, the sum, and (keep) what each layer's backward wants."""
        s, saved = None, []
        for i, layer in enumerate(self.layers):
            s, y1, n1, _ = self._norm(x, s, layer["w1"], drop)
            qkv = layer["qkv"].fwd(y1)
            o, kept = attend(i, layer, *self._split(qkv))
            o = o.view(-1, self.c.D)
            s, y2, n2, _ = self._norm(layer["out"].fwd(o), s, layer["w2"], drop)
            h = layer["up"].fwd(y2, L.DLRM_ACT_RELU)
            x = layer["down"].fwd(h)
            if keep:
                saved.append((y1, n1, qkv, o, kept, y2, n2, h))
        return x, s, saved

    # ------------------------------------------------------------------ training

    def forward(self, ids: torch.Tensor, offsets: torch.Tensor, drop: bool = True):
        """(users [B, D] bf16, what backward wants); every history holds an event."""

        def attend(i, layer, q, k, v):
            o, tiles, lse = L.dlrm_seq_attn_fwd(q, k, v, offsets, for_backward=True, **self._how(layer))
            return o, (o, tiles, lse)

        x, s, saved = self._layers(self._events(ids), attend, drop, keep=True)
        _, y, n, _ = self._norm(x, s, self.w, drop)
        last = offsets[1:] - 1
        return y[last], (ids, offsets, last, saved, n)

    def backward(self, dusers: torch.Tensor, kept) -> Tuple[torch.Tensor, List[Dict], torch.Tensor]:
        """From the users' gradients [B, D] fp32: (the event rows' [N, D] fp32, per layer its bias's and
        norms', the final norm's); the dense layers keep their own."""
        ids, offsets, last, saved, n = kept
        N, D = ids.numel(), self.c.D
        f32 = dict(x_dtype=torch.float32)
        dy = torch.zeros((N, D), device=self.dev)
        dy[last] = dusers
        dx, ds, dw = L.dlrm_add_rmsnorm_bwd(dy, None, n[0], self.w, n[1], **f32, **n[2])
        grads = []
        for layer, (y1, n1, qkv, o, (oh, tiles, lse), y2, n2, h) in reversed(list(zip(self.layers, saved))):
            dh = layer["down"].bwd(dx, h)
            dy = layer["up"].bwd(dh, y2, h, L.DLRM_ACT_RELU)
            dx, ds, dw2 = L.dlrm_add_rmsnorm_bwd(dy, ds, n2[0], layer["w2"], n2[1], **f32, **n2[2])
            do = L.dlrm_cast_rows(layer["out"].bwd(dx, o), D, D, torch.bfloat16).view(N, self.c.Hq, self.d)
            dq, dk, dv, dbias = L.dlrm_seq_attn_bwd(do, *self._split(qkv), oh, tiles, lse, offsets, **self._how(layer))
            dqkv = torch.cat((dq, dk, dv), 1).view(N, -1)
            dy = layer["qkv"].bwd(dqkv.float(), y1)
            dx, ds, dw1 = L.dlrm_add_rmsnorm_bwd(dy, ds, n1[0], layer["w1"], n1[1], **f32, **n1[2])
            grads.append(dict(bias=dbias, w1=dw1, w2=dw2))
        return dx, grads[::-1], dw

    def step(self, ids: torch.Tensor, offsets: torch.Tensor, clicks: torch.Tensor) -> torch.Tensor:
        """One training step on B histories and their clicks [B] (0 or 1); returns the loss [1]."""
        users, kept = self.forward(ids, offsets)
        head = L.dlrm_bce_head(users, self.head.W16.view(-1), self.head.b, clicks)
        rows, grads, dw = self.backward(head["dx"], kept)
        params = [(self.w, None, dw), (self.head.W32.view(-1), self.head.W16.view(-1), head["dw"]), (self.head.b, None, head["db"])]
        for layer, g in zip(self.layers, grads):
            for name in ("qkv", "out", "up", "down"):
                params += layer[name].params()
            params += [(layer[name], None, g[name]) for name in ("w1", "w2", "bias")]
        for i in range(0, len(params), 64):
            L.dlrm_sgd_dense_multi(params[i:i + 64], self.lr)
        one = torch.arange(ids.numel() + 1, dtype=torch.int64, device=self.dev)
        L.emb_bag_bwd_adagrad([self.table], [self.state], ids, one, None, rows.view(-1, 1, self.c.D), self.lr_emb, self.eps_emb)
        return head["loss"]

    # ------------------------------------------------------------------ serving

    def cache(self, users: int, capacity: int) -> "HistoryCache":
        return HistoryCache(self, users, capacity)


class HistoryCache:
    """Keys and values of `users` histories of up to `capacity` events, for every layer."""

    def __init__(self, enc: HistoryEncoder, users: int, capacity: int):
        c = enc.c
        self.enc, self.users, self.capacity = enc, users, capacity
        kv = dict(dtype=torch.bfloat16, device=enc.dev)
        self.k = [torch.empty((users * capacity, c.Hkv, enc.d), **kv) for _ in range(c.layers)]
        self.v = [torch.empty((users * capacity, c.Hkv, enc.d), **kv) for _ in range(c.layers)]
        self.begin = torch.arange(users, dtype=torch.int64, device=enc.dev) * capacity
        self.end = self.begin.clone()
        self.longest = 0  # the longest history, as the host knows it

    def prefill(self, ids: torch.Tensor, offsets: torch.Tensor, longest_new: int) -> torch.Tensor:
        """Encodes the users' new events (jagged, offsets [users + 1], at most longest_new each) against
        what the cache holds; returns each user's vector [users, D] (zeros for a user with no new event).
        The lengths are checked on the host, which waits for the device once: a count past longest_new or a
        region's end would be written into the next user's."""
        if offsets.shape != (self.users + 1,):
            raise ValueError(f"offsets must have {self.users + 1} entries, got {tuple(offsets.shape)}")
        offsets = offsets.to(torch.int64)  # the type of the regions'
        host = torch.cat((self.end - self.begin, offsets)).cpu().numpy()
        held, off = host[:self.users], host[self.users:]
        count = np.diff(off)
        if off[0] != 0 or off[-1] != ids.numel() or (count < 0).any():
            raise ValueError(f"offsets must rise from 0 to the number of events, {ids.numel()}")
        if count.max(initial=0) > longest_new:
            raise ValueError(f"longest_new is {longest_new}, but a user has {count.max()} new events")
        longest = int((held + count).max(initial=0))
        if longest > self.capacity:
            raise ValueError(f"a history of {longest} events does not fit a capacity of {self.capacity}")
        if ids.numel() == 0:
            return torch.zeros((self.users, self.enc.c.D), dtype=torch.bfloat16, device=self.enc.dev)
        enc, count = self.enc, offsets.diff()
        at = torch.arange(ids.numel(), device=enc.dev) + torch.repeat_interleave(self.end - offsets[:-1], count, output_size=ids.numel())
        end = self.end + count

        def attend(i, layer, q, k, v):
            self.k[i][at], self.v[i][at] = k, v
            return L.dlrm_seq_attn_fwd(q, self.k[i], self.v[i], offsets, (self.begin, end), **enc._how(layer)), None

        x, s, _ = enc._layers(enc._events(ids), attend)
        self.end, self.longest = end, longest
        last = (offsets[1:] - 1).clamp(min=0)
        y = enc._norm(x[last], s[last], enc.w, False)[1]
        return torch.where(count[:, None] > 0, y, 0)

    def append(self, ids: torch.Tensor, eight_bit: bool = False):
        """One new event of every user; returns their vectors [users, D] bf16, or with eight_bit 8-bit
        rows and their scales [users]."""
        if self.longest + 1 > self.capacity:
            raise ValueError(f"the cache holds {self.capacity} events a user")
        enc, at = self.enc, self.end
        end = at + 1

        def attend(i, layer, q, k, v):
            self.k[i][at], self.v[i][at] = k, v
            return L.dlrm_seq_attn_decode(q, self.k[i], self.v[i], self.begin, end, max_kv_len=self.longest + 1,
                                          **enc._how(layer)), None

        x, s, _ = enc._layers(enc._events(ids), attend)
        self.end, self.longest = end, self.longest + 1
        _, y, _, scale = enc._norm(x, s, enc.w, False, y_dtype=torch.float8_e4m3fn if eight_bit else torch.bfloat16)
        return (y, scale) if eight_bit else y


def main(steps: int = 800, users: int = 256, seed: int = 0) -> Tuple[float, float]:
    """Trains on synthetic histories (a click follows when one of a few event types is among the last
    four), then serves: the histories go into a cache, one new event each is appended, and the vectors
    are compared with the training forward's.  Returns the mean loss of the first and last steps."""
    dev = torch.device("cuda:0")
    enc = HistoryEncoder(Shape(events=1000, window=64, sinks=2), dev, seed, lr=0.3)
    rng = np.random.default_rng(seed + 1)
    losses = []
    for step in range(steps):
        lens = rng.integers(4, 120, users)
        off = np.concatenate([[0], np.cumsum(lens)])
        ids = rng.integers(0, 1000, off[-1])
        ids[rng.random(off[-1]) < 0.15] = 7
        clicks = np.array([(ids[e - 4:e] == 7).any() for e in off[1:]], np.float32)
        put = lambda a: torch.from_numpy(a).to(dev)  # noqa: E731
        losses.append(enc.step(put(ids), put(off), put(clicks)))
    first, last = (float(torch.cat(x).mean()) for x in (losses[:5], losses[-5:]))
    print(f"history: loss {first:.4f} -> {last:.4f} in {steps} steps of {users} histories", flush=True)
    cache = enc.cache(users, 128)
    cut = np.concatenate([np.arange(a, b - 1) for a, b in zip(off[:-1], off[1:])])
    cache.prefill(put(ids[cut]), put(off - np.arange(users + 1)), int(lens.max()))
    got = cache.append(put(ids[off[1:] - 1]))
    want, _ = enc.forward(put(ids), put(off), drop=False)
    err = float((got.float() - want.float()).norm() / want.float().norm())
    print(f"history: served vectors against the training forward's: relative difference {err:.2e}", flush=True)
    return first, last


if __name__ == "__main__":
    main()
