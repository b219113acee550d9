"""Plain fp64 definitions of the user-history operators (dlrm_seq.h): test infrastructure only.

Every function also returns error scales: the sums of the absolute values of the terms that an
output adds, against which its error is measured.
"""
from __future__ import annotations

import numpy as np


def bucket_of(bounds, n):
    """The last bucket whose first distance is at most n, for an array of distances n >= 0."""
    out = np.zeros(n.shape, np.int64)
    for t, first in enumerate(bounds):
        out[n >= first] = t
    return out


def visible(n, j, window, sinks):
    see = n >= 0
    if window:
        see &= (n < window) | (j < sinks)
    return see


def seq_attn(q, k, v, q_off, kv_begin, kv_end, window=0, sinks=0, scale=1.0, bias=None, bounds=None, do=None):
    """Forward and, with do, backward.  q [Nq,Hq,d], k, v [Nkv,Hkv,d] in fp64.  A dict: o, lse and
    their scales (o_s; z_s, the largest sum of a logit's terms), with do also dq, dk, dv, dbias and
    theirs."""
    Nq, Hq, d = q.shape
    Hkv = k.shape[1]
    r = dict(o=np.zeros((Nq, Hq, d)), o_s=np.zeros((Nq, Hq, d)), lse=np.full((Nq, Hq), -np.inf), z_s=0.0)
    if do is not None:
        for name, like in (("dq", q), ("dk", k), ("dv", v)):
            r[name], r[name + "_s"] = np.zeros(like.shape), np.zeros(like.shape)
        if bias is not None:
            r["dbias"], r["dbias_s"] = np.zeros(bias.shape), np.zeros(bias.shape)
    for b in range(len(q_off) - 1):
        q0, q1, k0, k1 = int(q_off[b]), int(q_off[b + 1]), int(kv_begin[b]), int(kv_end[b])
        nq, nk = q1 - q0, k1 - k0
        if nq == 0 or nk == 0:
            continue
        j = np.arange(nk)[None, :]
        n = (nk - nq + np.arange(nq))[:, None] - j
        see = visible(n, j, window, sinks)
        t = bucket_of(bounds, np.maximum(n, 0)) if bias is not None else None
        for h in range(Hq):
            g = h // (Hq // Hkv)
            Q, K, V = q[q0:q1, h], k[k0:k1, g], v[k0:k1, g]
            with np.errstate(all="ignore"):
                z = scale * (Q @ K.T)
                zs = abs(scale) * (np.abs(Q) @ np.abs(K).T)
                if bias is not None:
                    z = z + bias[h][t]
                    zs = zs + np.abs(bias[h][t])
                z = np.where(see, z, -np.inf)
                if see.any():
                    r["z_s"] = max(r["z_s"], float(np.max(np.where(see & np.isfinite(zs), zs, 0.0))))
                top = z.max(1, keepdims=True)
                ref = np.where(np.isinf(top), 0.0, top)
                e = np.where(z == -np.inf, 0.0, np.exp(z - ref))
                total = e.sum(1, keepdims=True)
                P = e / np.where(total == 0, 1.0, total)
                lse = np.where(total == 0, -np.inf, ref + np.log(np.where(total == 0, 1.0, total)))
            hide = ~see.any(0)  # keys that nobody sees may hold anything
            V0 = np.where(hide[:, None], 0.0, V)
            if np.isfinite(V0).all():
                o, o_s = P @ V0, P @ np.abs(V0)
            else:
                o = np.stack([(P[i, see[i]][:, None] * V[see[i]]).sum(0) for i in range(nq)])
                o_s = np.abs(o)
            r["o"][q0:q1, h], r["o_s"][q0:q1, h], r["lse"][q0:q1, h] = o, o_s, lse[:, 0]
            if do is None:
                continue
            G = do[q0:q1, h]
            K0 = np.where(hide[:, None], 0.0, K)
            dP, dP_s = G @ V0.T, np.abs(G) @ np.abs(V0).T
            delta, delta_s = (G * o).sum(1, keepdims=True), (np.abs(G) * o_s).sum(1, keepdims=True)
            ds, ds_s = P * (dP - delta), P * (dP_s + delta_s)
            r["dq"][q0:q1, h], r["dq_s"][q0:q1, h] = scale * (ds @ K0), abs(scale) * (ds_s @ np.abs(K0))
            r["dk"][k0:k1, g] += scale * (ds.T @ Q)
            r["dk_s"][k0:k1, g] += abs(scale) * (ds_s.T @ np.abs(Q))
            r["dv"][k0:k1, g] += P.T @ G
            r["dv_s"][k0:k1, g] += P.T @ np.abs(G)
            if bias is not None:
                for u in range(bias.shape[1]):
                    pick = see & (t == u)
                    r["dbias"][h, u] += ds[pick].sum()
                    r["dbias_s"][h, u] += ds_s[pick].sum()
    return r


def philox4x32(counter, key):
    """Ten rounds of Philox4x32 (Salmon, Moraes, Dror and Shaw, 2011) in Python's integers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def drop_factors(n, p, seed, offset):
    """What each of n elements is multiplied by: 0, or one number that is kept in fp32."""
    limit = int(np.floor(float(np.float32(p)) * 65536 + 0.5))
    scale = float(np.float32(65536 / (65536 - limit))) if limit < 65536 else 0.0
    out = np.zeros(n)
    words = None
    for e in range(n):
        if e % 8 == 0:
            c = (offset + e // 8) % (1 << 64)
            words = philox4x32([c & 0xFFFFFFFF, c >> 32, 0, 0], [seed & 0xFFFFFFFF, seed >> 32])
        u = words[e % 8 // 2] >> (16 * (e % 2)) & 0xFFFF
        out[e] = scale if u >= limit else 0.0
    return out


def dropout(x, f):
    return np.where(f == 0, 0.0, x * np.where(f == 0, 1.0, f))


def add_rmsnorm(x, residual, w, eps, f, s_round):
    """(s exact, s rounded by s_round, rstd, y) with dropout factors f (of x's shape, or None)."""
    s = residual + (x if f is None else dropout(x, f))
    h = s_round(s)
    rstd = 1.0 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    return s, h, rstd[:, 0], h * rstd * w


def add_rmsnorm_bwd(dy, ds, h, w, eps, f):
    """(dx, dresidual, dw) and the scales of the last two, from the kept sum h."""
    rstd = 1.0 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    hat, g = h * rstd, dy * w
    dh = ds + rstd * (g - hat * (g * hat).mean(1, keepdims=True))
    dh_s = np.abs(ds) + rstd * (np.abs(g) + np.abs(hat) * np.abs(g * hat).mean(1, keepdims=True))
    return (dh if f is None else dropout(dh, f)), dh, (dy * hat).sum(0), dh_s, np.abs(dy * hat).sum(0)
