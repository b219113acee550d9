"""Plain fp64 definition of linear attention with a decay (dlrm_seq_decay.h), event by event: test
infrastructure only.  Each value comes with its error scale, the sum of the absolute values of the
terms that it adds."""
from __future__ import annotations

import numpy as np


def decay(q, k, v, g, off, scale=1.0, state=None, do=None):
    """Forward and, with do, backward of sequences off[b] .. off[b+1].  q [N,Hq,d], k, v [N,Hkv,d], g [N,Hkv] (or
    [Hkv]) in fp64, state [B,Hkv,d,d] or None.  A dict: o, state (after the last events), with do also dq, dk, dv, dg; and
    their scales (o_s ...; dg_s: of all terms <q, dq> and <k, dk> of the sequence)."""
    N, Hq, d = q.shape
    Hkv = k.shape[1]
    B, group = len(off) - 1, Hq // Hkv
    each = np.ndim(g) == 2
    g = g if each else np.broadcast_to(g, (N, Hkv))
    lam = np.exp(np.minimum(g, 0.0))
    first = np.zeros((B, Hkv, d, d)) if state is None else state
    r = dict(state=first.copy(), state_s=np.abs(first))
    names = [("o", q)] + ([("dq", q), ("dk", k), ("dv", v)] if do is not None else [])
    for name, like in names:
        r[name], r[name + "_s"] = np.zeros(like.shape), np.zeros(like.shape)
    if do is not None:
        r["dg"], r["dg_s"] = np.zeros((N, Hkv)), np.zeros((N, Hkv))
    heads = lambda x: x.reshape(x.shape[0], Hkv, group, d)  # noqa: E731
    for b in range(B):
        t0, t1 = int(off[b]), int(off[b + 1])
        for sign in ("", "_s"):
            f = np.abs if sign else (lambda x: x)
            Q, K, V = heads(f(q[t0:t1])), f(k[t0:t1]), f(v[t0:t1])
            S = f(first[b]).copy()
            before = []
            for t in range(t1 - t0):
                before.append(S)
                S = lam[t0 + t][:, None, None] * S + K[t][:, :, None] * V[t][:, None, :]
                r["o" + sign][t0 + t] = scale * np.einsum("hgc,hce->hge", Q[t], S).reshape(Hq, d)
                if do is not None:
                    r["dq" + sign][t0 + t] = scale * np.einsum("hge,hce->hgc", heads(f(do[t0:t1]))[t], S).reshape(Hq, d)
            r["state" + sign][b] = S
            if do is None:
                continue
            G, R = heads(f(do[t0:t1])), np.zeros((Hkv, d, d))
            for t in range(t1 - t0 - 1, -1, -1):
                R = (R if t == t1 - t0 - 1 else lam[t0 + t + 1][:, None, None] * R) + np.einsum("hgc,hge->hce", Q[t], G[t])
                r["dk" + sign][t0 + t] = scale * np.einsum("hce,he->hc", R, V[t])
                r["dv" + sign][t0 + t] = scale * np.einsum("hce,hc->he", R, K[t])
                if not sign:
                    r["dg"][t0 + t] = np.where(g[t0 + t] > 0, 0.0, scale * lam[t0 + t] * np.einsum("hce,hce->h", before[t], R))
        if do is not None and t1 > t0:
            terms = (np.abs(q[t0:t1]) * r["dq_s"][t0:t1]).reshape(t1 - t0, Hkv, -1).sum((0, 2)) + \
                    (np.abs(k[t0:t1]) * r["dk_s"][t0:t1]).sum((0, 2))
            r["dg_s"][t0:t1] = terms
    if do is not None and not each:  # each event's sum is of up to all terms of its sequence
        r["dg"], r["dg_s"] = r["dg"].sum(0), r["dg_s"].sum(0)
    return r
