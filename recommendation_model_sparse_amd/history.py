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
kernels, but for what moves data: torch indexes rows, in the backward joins dq, dk and dv and
casts them, and keeps the learned decays at 0 or below.  The residual stream is fp32, activations and
the dense layers' weights bf16 with fp32 masters (SGD), the table is updated by row-wise Adagrad.
Histories are jagged: event rows laid end to end, with offsets [B + 1].

Serving keeps each layer's keys and values in a region of `capacity` rows a user (`cache`), or in pages of
a pool that all users share (`paged_cache`): `prefill` encodes the events since the last visit against them,
`append` one new event a user, and `append(eight_bit=True)` gives the users' vectors as 8-bit rows with scales
for a store of candidates.

The first `linear` layers have linear attention with a learned decay for each key head instead, and an RMS norm
of each head's output: what they keep of a user is one d x d state a key head, however long the history.
"""
from __future__ import annotations

import contextlib
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
    linear: int = 0      # of the layers, the first ones with linear attention


class HistoryEncoder:
    def __init__(self, shape: Shape, dev, seed: int = 0, lr: float = 0.1, lr_emb: float = 0.05, eps_emb: float = 1e-8):
        self.c, self.dev, self.lr, self.lr_emb, self.eps_emb, self.seed = shape, dev, lr, lr_emb, eps_emb, seed
        c = shape
        if c.D % c.Hq or c.D // c.Hq % 8:
            raise ValueError(f"D must be {c.Hq} heads of a multiple of 8 columns, got {c.D}")
        if not 0 <= c.linear <= c.layers:
            raise ValueError(f"linear must be 0 to {c.layers} layers, got {c.linear}")
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
        for layer in self.layers[:c.linear]:  # half of what a state holds is gone after 2, 5, 11, 22 .. events
            del layer["bias"]
            layer.update(g=-torch.exp2(-2.0 - torch.arange(c.Hkv)).to(dev), wo=torch.ones(self.d, device=dev))
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

    def _heads_norm(self, o, layer):
        """The norm of a linear layer's heads, and what its backward wants.  eps: a head's output is as small as q . k
        of a first event may be, and the norm passes an error on enlarged up to 1 / sqrt(eps) times.  q . k / sqrt(d)
        of bf16 values of about 0.6 is off by 1e-3: times v and 1 / sqrt(1e-3) 2 % of a normed head at most, where
        1e-6 would leave a gradient of any size."""
        s, y, rstd, _ = L.dlrm_add_rmsnorm_fwd(o.view(-1, self.d), None, layer["wo"], eps=1e-3, res_dtype=torch.bfloat16)
        return y, (s, rstd)

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

    def forward(self, ids: torch.Tensor, offsets: torch.Tensor, drop: bool = True, longest: Optional[int] = None):
        """(users [B, D] bf16, what backward wants); every history holds an event.  longest: the longest history
        where the host knows it, for the linear layers' choice of how they work (1024 histories of up to 512 events, heads of 64:
        a layer's forward 63 us and 91 without it, its backward 253 and 346)."""

        def attend(i, layer, q, k, v):
            if "g" in layer:
                return self._heads_norm(L.dlrm_seq_decay_fwd(q, k, v, layer["g"], offsets, max_len=longest), layer)
            o, tiles, lse = L.dlrm_seq_attn_fwd(q, k, v, offsets, for_backward=True, **self._how(layer))
            return o, (o, tiles, lse)

        x, s, saved = self._layers(self._events(ids), attend, drop, keep=True)
        _, y, n, _ = self._norm(x, s, self.w, drop)
        last = offsets[1:] - 1
        return y[last], (ids, offsets, last, saved, n, longest)

    def backward(self, dusers: torch.Tensor, kept) -> Tuple[torch.Tensor, List[Dict], torch.Tensor]:
        """From the users' gradients [B, D] fp32: (the event rows' [N, D] fp32, per layer its bias's or decays' and
        norms', the final norm's); the dense layers keep their own."""
        ids, offsets, last, saved, n, longest = kept
        N, D = ids.numel(), self.c.D
        f32 = dict(x_dtype=torch.float32)
        dy = torch.zeros((N, D), device=self.dev)
        dy[last] = dusers
        dx, ds, dw = L.dlrm_add_rmsnorm_bwd(dy, None, n[0], self.w, n[1], **f32, **n[2])
        grads = []
        for layer, (y1, n1, qkv, o, seen, y2, n2, h) in reversed(list(zip(self.layers, saved))):
            dh = layer["down"].bwd(dx, h)
            dy = layer["up"].bwd(dh, y2, h, L.DLRM_ACT_RELU)
            dx, ds, dw2 = L.dlrm_add_rmsnorm_bwd(dy, ds, n2[0], layer["w2"], n2[1], **f32, **n2[2])
            do = L.dlrm_cast_rows(layer["out"].bwd(dx, o), D, D, torch.bfloat16).view(N, self.c.Hq, self.d)
            if "g" in layer:
                do, _, dwo = L.dlrm_add_rmsnorm_bwd(do.view(-1, self.d), None, seen[0], layer["wo"], seen[1])
                dq, dk, dv, dg = L.dlrm_seq_decay_bwd(do.view(N, self.c.Hq, self.d), *self._split(qkv), layer["g"], offsets, max_len=longest)
                own = dict(g=dg, wo=dwo)
            else:
                oh, tiles, lse = seen
                dq, dk, dv, dbias = L.dlrm_seq_attn_bwd(do, *self._split(qkv), oh, tiles, lse, offsets, **self._how(layer))
                own = dict(bias=dbias)
            dqkv = torch.cat((dq, dk, dv), 1).view(N, -1)
            dy = layer["qkv"].bwd(dqkv.float(), y1)
            dx, ds, dw1 = L.dlrm_add_rmsnorm_bwd(dy, ds, n1[0], layer["w1"], n1[1], **f32, **n1[2])
            grads.append(dict(own, w1=dw1, w2=dw2))
        return dx, grads[::-1], dw

    def step(self, ids: torch.Tensor, offsets: torch.Tensor, clicks: torch.Tensor, longest: Optional[int] = None) -> torch.Tensor:
        """One training step on B histories and their clicks [B] (0 or 1); returns the loss [1].  A linear layer's decays
        stay at 0 or below: a step past 0 ends there."""
        users, kept = self.forward(ids, offsets, longest=longest)
        head = L.dlrm_bce_head(users, self.head.W16.view(-1), self.head.b, clicks)
        rows, grads, dw = self.backward(head["dx"], kept)
        params = [(self.w, None, dw), (self.head.W32.view(-1), self.head.W16.view(-1), head["dw"]), (self.head.b, None, head["db"])]
        for layer, g in zip(self.layers, grads):
            for name in ("qkv", "out", "up", "down"):
                params += layer[name].params()
            params += [(layer[name], None, g[name]) for name in g]
        for i in range(0, len(params), 64):
            L.dlrm_sgd_dense_multi(params[i:i + 64], self.lr)
        for layer in self.layers[:self.c.linear]:  # above 0 a decay counts as 0 without a gradient, and would stay there; at 0 it has one
            layer["g"].clamp_(max=0)
        one = torch.arange(ids.numel() + 1, dtype=torch.int64, device=self.dev)
        L.emb_bag_bwd_adagrad([self.table], [self.state], ids, one, None, rows.view(-1, 1, self.c.D), self.lr_emb, self.eps_emb)
        return head["loss"]

    # ------------------------------------------------------------------ serving

    def cache(self, users: int, capacity: int) -> "HistoryCache":
        return HistoryCache(self, users, capacity)

    def paged_cache(self, users: int, longest: int, pages: int, page: int = 64) -> "PagedHistoryCache":
        return PagedHistoryCache(self, users, longest, pages, page)


class _States:
    """The states of `users` histories in the linear layers, and what both caches do with them.

    A visit updates states layer by layer, in place.  Where it ends half way (no memory for a layer, for instance), its
    users' histories are neither with its events nor without: `torn` says whose, and until they have left every visit is refused."""

    def __init__(self, enc: HistoryEncoder, users: int):
        self.enc, self.users = enc, users
        self.torn = np.zeros(users, bool)
        self.state = [torch.zeros((users, enc.c.Hkv, enc.d, enc.d), device=enc.dev) for _ in range(enc.c.linear)]

    def _whole(self):
        if self.torn.any():
            raise RuntimeError(f"a visit of users {np.flatnonzero(self.torn).tolist()} ended half way: their histories cannot be used")

    @contextlib.contextmanager
    def _half_way(self, users):
        """What changes the histories of `users` (a mask) bit by bit."""
        try:
            yield
        except BaseException:
            self.torn |= users
            raise

    def _linear(self, i, layer, q, k, v, offsets, longest_new):
        """New events (offsets None: one of each user) through linear layer i."""
        if offsets is None:
            o = L.dlrm_seq_decay_step(q, k, v, layer["g"], self.state[i])
        else:
            o, _ = L.dlrm_seq_decay_fwd(q, k, v, layer["g"], offsets, state=self.state[i], state_out=self.state[i], max_len=longest_new)
        return self.enc._heads_norm(o, layer)[0], None

    def _offsets(self, ids, offsets, longest_new, *others):
        """Offsets as int64, each user's new events on the host, and the others' values there: one wait for the device."""
        if offsets.shape != (self.users + 1,):
            raise ValueError(f"offsets must have {self.users + 1} entries, got {tuple(offsets.shape)}")
        offsets = offsets.to(torch.int64)
        off, *values = torch.cat((offsets,) + others).cpu().split([self.users + 1] + [x.numel() for x in others])
        off = off.numpy()
        count = np.diff(off)
        if off[0] != 0 or off[-1] != ids.numel() or (count < 0).any():
            raise ValueError(f"offsets must rise from 0 to the number of events, {ids.numel()}")
        if count.max(initial=0) > longest_new:
            raise ValueError(f"longest_new is {longest_new}, but a user has {count.max()} new events")
        return offsets, count, [x.numpy() for x in values]

    def _users(self, x, s, offsets):
        """Each user's vector, its last event's [users, D] (zeros for a user with no new event)."""
        last = (offsets[1:] - 1).clamp(min=0)
        y = self.enc._norm(x[last], s[last], self.enc.w, False)[1]
        return torch.where(offsets.diff()[:, None] > 0, y, 0)

    def _appended(self, x, s, eight_bit):
        _, y, _, scale = self.enc._norm(x, s, self.enc.w, False, y_dtype=torch.float8_e4m3fn if eight_bit else torch.bfloat16)
        return (y, scale) if eight_bit else y


class HistoryCache(_States):
    """Keys and values of `users` histories of up to `capacity` events, for every layer that has them."""

    def __init__(self, enc: HistoryEncoder, users: int, capacity: int):
        super().__init__(enc, users)
        c = enc.c
        self.capacity = capacity
        kv = dict(dtype=torch.bfloat16, device=enc.dev)
        self.k = [torch.empty((users * capacity, c.Hkv, enc.d), **kv) if i >= c.linear else None for i in range(c.layers)]
        self.v = [torch.empty((users * capacity, c.Hkv, enc.d), **kv) if i >= c.linear else None for i in range(c.layers)]
        self.begin = torch.arange(users, dtype=torch.int64, device=enc.dev) * capacity
        self.end = self.begin.clone()
        self.longest = 0  # the longest history, as the host knows it

    def prefill(self, ids: torch.Tensor, offsets: torch.Tensor, longest_new: int) -> torch.Tensor:
        """Encodes the users' new events (jagged, offsets [users + 1], at most longest_new each) against
        what the cache holds; returns each user's vector [users, D] (zeros for a user with no new event).
        The lengths are checked on the host, which waits for the device once: a count past longest_new or a
        region's end would be written into the next user's.  (A visit that ends half way can be made again, but with linear
        layers: then the cache refuses any further one.)"""
        self._whole()
        offsets, count, (held,) = self._offsets(ids, offsets, longest_new, self.end - self.begin)
        longest = int((held + count).max(initial=0))
        if longest > self.capacity:
            raise ValueError(f"a history of {longest} events does not fit a capacity of {self.capacity}")
        if ids.numel() == 0:
            return torch.zeros((self.users, self.enc.c.D), dtype=torch.bfloat16, device=self.enc.dev)
        enc, fresh, count = self.enc, count > 0, offsets.diff()
        at = torch.arange(ids.numel(), device=enc.dev) + torch.repeat_interleave(self.end - offsets[:-1], count, output_size=ids.numel())
        end, events = self.end + count, enc._events(ids)

        def attend(i, layer, q, k, v):
            if "g" in layer:
                return self._linear(i, layer, q, k, v, offsets, longest_new)
            self.k[i][at], self.v[i][at] = k, v
            return L.dlrm_seq_attn_fwd(q, self.k[i], self.v[i], offsets, (self.begin, end), **enc._how(layer)), None

        with self._half_way(fresh & bool(self.state)):
            x, s, _ = enc._layers(events, attend)
            users = self._users(x, s, offsets)
        self.end, self.longest = end, longest
        return users

    def append(self, ids: torch.Tensor, eight_bit: bool = False):
        """One new event of every user; returns their vectors [users, D] bf16, or with eight_bit 8-bit
        rows and their scales [users]."""
        self._whole()
        if self.longest + 1 > self.capacity:
            raise ValueError(f"the cache holds {self.capacity} events a user")
        if ids.shape != (self.users,):
            raise ValueError(f"ids must be one event of each of {self.users} users, got {tuple(ids.shape)}")
        enc, at = self.enc, self.end
        end, events = at + 1, enc._events(ids)

        def attend(i, layer, q, k, v):
            if "g" in layer:
                return self._linear(i, layer, q, k, v, None, 1)
            self.k[i][at], self.v[i][at] = k, v
            return L.dlrm_seq_attn_decode(q, self.k[i], self.v[i], self.begin, end, max_kv_len=self.longest + 1,
                                          **enc._how(layer)), None

        with self._half_way(np.full(self.users, bool(self.state))):
            x, s, _ = enc._layers(events, attend)
            users = self._appended(x, s, eight_bit)
        self.end, self.longest = end, self.longest + 1
        return users


class PagedHistoryCache(_States):
    """Keys and values of `users` histories of up to `longest` events in a pool of `pages` pages of `page` events each,
    which the users share: a history takes the pages that it fills, and gives them back when its user leaves.
    The host knows the histories' lengths, so that a call that does not fit is refused before anything changes.  Events are
    counted before the layers write their rows: users whose visit ends half way have to leave (`release`)."""

    def __init__(self, enc: HistoryEncoder, users: int, longest: int, pages: int, page: int = 64):
        super().__init__(enc, users)
        c, dev = enc.c, enc.dev
        self.longest, self.page, self.pages = longest, page, pages
        kv = dict(dtype=torch.bfloat16, device=dev)
        self.k = [torch.empty((pages * page, c.Hkv, enc.d), **kv) if i >= c.linear else None for i in range(c.layers)]
        self.v = [torch.empty((pages * page, c.Hkv, enc.d), **kv) if i >= c.linear else None for i in range(c.layers)]
        i32 = dict(dtype=torch.int32, device=dev)
        self.table = torch.full((users, -(-longest // page)), -1, **i32)
        self.lengths, self.free = torch.zeros(users, **i32), torch.arange(pages, **i32)
        self.free_count = torch.full((1,), pages, **i32)
        self.held = np.zeros(users, np.int64)  # the lengths, as the host knows them

    def _update(self, count, offsets, n, leave=None):
        """The new events' slots, and the lengths with them; `count` and `leave` on the host."""
        held = self.held if leave is None else np.where(leave, 0, self.held)
        new = held + count
        if new.max(initial=0) > self.longest:
            raise ValueError(f"a history of {int(new.max())} events does not fit the longest, {self.longest}")
        want = int((-(-new // self.page)).sum())
        if want > self.pages:
            raise ValueError(f"the histories need {want} pages of {self.pages}")
        gone = None if leave is None else torch.from_numpy(leave).to(self.enc.dev)
        slots, _ = L.dlrm_seq_pages_update(self.table, self.lengths, self.free, self.free_count, self.page, offsets, n, gone)
        self.held = new
        return slots

    def release(self, users) -> None:
        """Users (their numbers) leave: their pages go back, and they are without a history, also those whose last visit
        ended half way."""
        leave, users = np.zeros(self.users, bool), np.asarray(users, np.int64)
        if ((users < 0) | (users >= self.users)).any():
            raise ValueError(f"users must be 0 to {self.users - 1}, got {users}")
        leave[users] = True
        none = torch.zeros(self.users + 1, dtype=torch.int64, device=self.enc.dev)
        with self._half_way(leave):
            self._update(np.zeros(self.users, np.int64), none, 0, leave)
            for state in self.state:
                state[torch.from_numpy(leave).to(self.enc.dev)] = 0
        self.torn &= ~leave

    def prefill(self, ids: torch.Tensor, offsets: torch.Tensor, longest_new: int) -> torch.Tensor:
        """HistoryCache.prefill, over the pages."""
        self._whole()
        enc = self.enc
        offsets, count, _ = self._offsets(ids, offsets, longest_new)
        if ids.numel() == 0:
            return torch.zeros((self.users, enc.c.D), dtype=torch.bfloat16, device=enc.dev)
        events, slots = enc._events(ids), self._update(count, offsets, ids.numel())

        def attend(i, layer, q, k, v):
            if "g" in layer:
                return self._linear(i, layer, q, k, v, offsets, longest_new)
            L.dlrm_seq_pages_write(k, v, slots, self.k[i], self.v[i])
            return L.dlrm_seq_attn_paged_fwd(q, self.k[i], self.v[i], offsets, self.table, self.lengths, self.page, **enc._how(layer)), None

        with self._half_way(count > 0):
            x, s, _ = enc._layers(events, attend)
            return self._users(x, s, offsets)

    def append(self, ids: torch.Tensor, eight_bit: bool = False):
        """HistoryCache.append, over the pages."""
        self._whole()
        enc = self.enc
        if ids.shape != (self.users,):
            raise ValueError(f"ids must be one event of each of {self.users} users, got {tuple(ids.shape)}")
        one = torch.arange(self.users + 1, dtype=torch.int64, device=enc.dev)
        events, slots = enc._events(ids), self._update(np.ones(self.users, np.int64), one, self.users)
        longest = int(self.held.max(initial=0))

        def attend(i, layer, q, k, v):
            if "g" in layer:
                return self._linear(i, layer, q, k, v, None, 1)
            L.dlrm_seq_pages_write(k, v, slots, self.k[i], self.v[i])
            return L.dlrm_seq_attn_paged_decode(q, self.k[i], self.v[i], self.table, self.lengths, self.page, max_kv_len=longest,
                                                **enc._how(layer)), None

        with self._half_way(np.ones(self.users, bool)):
            x, s, _ = enc._layers(events, attend)
            return self._appended(x, s, eight_bit)


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
        losses.append(enc.step(put(ids), put(off), put(clicks), int(lens.max())))
    first, last = (float(torch.cat(x).mean()) for x in (losses[:5], losses[-5:]))
    print(f"history: loss {first:.4f} -> {last:.4f} in {steps} steps of {users} histories", flush=True)
    cache = enc.cache(users, 128)
    cut = np.concatenate([np.arange(a, b - 1) for a, b in zip(off[:-1], off[1:])])
    cache.prefill(put(ids[cut]), put(off - np.arange(users + 1)), int(lens.max()))
    got = cache.append(put(ids[off[1:] - 1]))
    want, _ = enc.forward(put(ids), put(off), drop=False)
    err = float((got.float() - want.float()).norm() / want.float().norm())
    print(f"history: served vectors against the training forward's: relative difference {err:.2e}", flush=True)
    paged = enc.paged_cache(users, 128, 5 * users, 32)
    paged.prefill(put(ids[cut]), put(off - np.arange(users + 1)), int(lens.max()))
    err = float((paged.append(put(ids[off[1:] - 1])).float() - got.float()).norm() / got.float().norm())
    print(f"history: served from pages: relative difference {err:.2e}", flush=True)
    return first, last


if __name__ == "__main__":
    main()
