"""The cases that serving many user histories is measured on: block tables and slots built on the GPU
from the lengths of a visit, attention over a paged cache for one new event and for several, and
linear attention with a decay for each event and head, trained, run over new events from a state,
and for one event.

`run` computes a case in its plain form (elementary torch operations in fp32), or, where `own` is
true, through the package's entry points.  `exact` gives the same outputs from the definitions in
64 bits, one sequence at a time.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # a serving step of a batch: one new event of each user; users at the longest history start over
        dict(name="pages-append", op="pages", B=256, lo=1, hi=511, new=1, page=16, cap=512, share=1.0),
        # many users come back at once, with up to 300 events each since their last visit
        dict(name="pages-visit", op="pages", B=20000, lo=1, hi=700, new=300, page=64, cap=1024, share=1.0),
        # one user, one new event: latency
        dict(name="paged-one", op="decode", B=1, lo=150, hi=200, page=64, Hq=4, Hkv=4, d=32, window=0, sinks=0, buckets=32,
             reach=128),
        # a batch of users with histories of every length, small pages
        dict(name="paged-batch", op="decode", B=256, lo=64, hi=8192, page=16, Hq=8, Hkv=2, d=64, window=0, sinks=0,
             buckets=32, reach=1024),
        # very long histories, one shared key/value head: the pages are read from HBM
        dict(name="paged-long", op="decode", B=32, lo=32768, hi=65536, page=256, Hq=8, Hkv=1, d=128, window=0, sinks=0,
             buckets=64, reach=4096),
        # the events since the last visit (up to 300) against the whole paged history
        dict(name="paged-prefill", op="prefill", B=16, lo=100, hi=2048, new=300, page=64, Hq=8, Hkv=2, d=128, window=512,
             sinks=4, buckets=32, reach=512),
        # a batch of new users in training: a few events each, some with none, one decay for a head
        dict(name="decay-short", op="train", B=256, lo=1, hi=64, empty=0.05, Hq=4, Hkv=4, d=32, each=False),
        # the ordinary training batch: 1024 users of up to 512 events, decays by the time between events
        dict(name="decay-users", op="train", B=1024, lo=16, hi=512, empty=0.0, Hq=2, Hkv=2, d=64, each=True),
        # few users with long histories, shared key/value heads
        dict(name="decay-long", op="train", B=4, lo=2000, hi=4096, empty=0.0, Hq=8, Hkv=2, d=128, each=True),
        # the events since the last visit, from the state that it left to a new one
        dict(name="decay-prefill", op="state", B=64, lo=1, hi=1500, empty=0.0, Hq=8, Hkv=2, d=128, each=True),
        # one event of one user: latency
        dict(name="step-one", op="step", B=1, Hq=4, Hkv=4, d=32, each=True),
        # one event of every user of a large batch: the states are read and written in HBM
        dict(name="step-batch", op="step", B=512, Hq=8, Hkv=4, d=128, each=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pages", "decode", "decode", "prefill", "train", "train", "state", "step"])
    if op == "pages":
        page, cap = rng.choice([8, 16, 64, 256]), _log(rng, 64, 2048)
        new = rng.choice([1, _log(rng, 2, max(3, cap // 2))])
        return dict(op=op, B=_log(rng, 1, 20000), lo=1, hi=cap, new=new, page=page, cap=cap + new, share=rng.choice([1.0, 0.5]))
    d = rng.choice([32, 64, 128, 40, 96])
    Hkv = rng.choice([1, 2, 4])
    c = dict(op=op, Hq=Hkv * rng.choice([1, 1, 2, 4]), Hkv=Hkv, d=d)
    if op == "step":
        return dict(c, B=_log(rng, 1, max(2, (1 << 27) // (4 * Hkv * d * d))), each=rng.choice([True, False]))
    if op in ("train", "state"):
        hi = _log(rng, 16, 4096)
        most = max(1, min(1024, (1 << 27) // (hi * hi * c["Hq"]), (1 << 27) // (4 * Hkv * d * d)))
        return dict(c, B=_log(rng, 1, most), lo=max(1, hi // rng.choice([2, 30])), hi=hi, empty=rng.choice([0.0, 0.1]),
                    each=rng.choice([True, True, False]))
    window = rng.choice([0, 0, _log(rng, 16, 1024)])
    c.update(window=window, sinks=rng.choice([0, 1, 4, 7]) if window else 0, buckets=rng.choice([8, 32, 33, 64]),
             reach=_log(rng, 128, 4096), page=rng.choice([8, 16, 32, 64, 128, 512]))
    if op == "decode":
        hi = _log(rng, 16, 65536)
        most = max(1, min(1024, (1 << 30) // (hi * Hkv * d * 4)))
        return dict(c, B=_log(rng, 1, most), lo=max(1, hi // rng.choice([2, 50])), hi=hi)
    hi = _log(rng, 16, 4096)
    most = max(1, min(512, (1 << 27) // (hi * hi * c["Hq"])))
    return dict(c, B=_log(rng, 1, most), lo=max(1, hi // rng.choice([2, 30])), hi=hi, new=_log(rng, 1, hi))


# ------------------------------------------------------------------------------------- the inputs

def _lens(case, seed):
    """(events, new events) of each history: lengths log-uniform over [lo, hi], a share of them empty.
    The lengths are the case's own, in an order that the seed gives."""
    r = random.Random(case["B"] * 7919 + case["hi"])
    kv = [max(case["lo"], min(case["hi"], _log(r, case["lo"], case["hi"]))) for _ in range(case["B"])]
    some = [0 if r.random() < case.get("empty", 0.0) else n for n in kv]
    kv = some if any(some) else kv
    if case["op"] in ("train", "state"):
        new = kv
    elif case["op"] == "pages":
        new = [_log(r, 1, case["new"]) for _ in kv]
    else:
        new = [min(n, r.randint(1, case.get("new", 1))) for n in kv]
    both = list(zip(kv, new))
    random.Random(seed).shuffle(both)
    return [n for n, _ in both], [m for _, m in both]


def _starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _bounds(buckets, reach):
    """First distance of each bucket: one distance a bucket for the first half, then growing
    geometrically up to `reach`; the last bucket is open."""
    half = max(1, buckets // 2)
    out = list(range(half))
    for i in range(half, buckets):
        f = (i - half) / max(1, buckets - 1 - half)
        out.append(max(out[-1] + 1, int(round(half * (max(reach, half + 1) / half) ** f))))
    return out


def _normal(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _dev(values, dtype):
    return torch.tensor(values, dtype=dtype, device=DEV)


def _tables(lens, page, width, spare, g):
    """Histories as a service has them after a while: every page of the pool in some user's hands or on
    the stack of free ones, in no order.  (table, free pages, how many of them are free, pages)."""
    have = [-(-n // page) for n in lens]
    pages = sum(have) + spare
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    at = _dev(_starts(have), torch.int64)
    col = torch.arange(width, device=DEV)
    used = col < at.diff()[:, None]
    table = torch.where(used, order[torch.where(used, at[:-1, None] + col, 0)], -1)
    free = torch.cat((order[at[-1]:], torch.full((pages - spare,), -1, dtype=torch.int32, device=DEV)))
    return table.to(torch.int32).contiguous(), free, _dev([spare], torch.int32), pages


def prepare(case, seed):
    op, B = case["op"], case["B"]
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case=case)
    if op == "pages":
        lens, new = _lens(case, seed)
        page, width = case["page"], -(-case["cap"] // case["page"])
        held = sum(-(-n // page) for n in lens)
        spare = max(0, int(case["share"] * B * width) - held)
        s["table"], s["free"], s["free_count"], _ = _tables(lens, page, width, spare, g)
        s.update(lengths=_dev(lens, torch.int32), new=_dev(new, torch.int32), offsets=_dev(_starts(new), torch.int64), n=sum(new))
        return s
    Hq, Hkv, d, bf = case["Hq"], case["Hkv"], case["d"], torch.bfloat16
    if op in ("decode", "prefill"):
        kv, new = _lens(case, seed)
        page, qs = case["page"], _starts(new)
        width = -(-max(kv) // page)
        s["table"], _, _, pages = _tables(kv, page, width, B, g)
        s.update(q=_normal(g, qs[-1], Hq, d, dtype=bf), k_new=_normal(g, qs[-1], Hkv, d, dtype=bf),
                 v_new=_normal(g, qs[-1], Hkv, d, dtype=bf), k=_normal(g, pages * page, Hkv, d, dtype=bf),
                 v=_normal(g, pages * page, Hkv, d, dtype=bf), bias=_normal(g, Hq, case["buckets"], std=0.5),
                 bounds=_bounds(case["buckets"], case["reach"]), max_q=max(new), max_kv=max(kv),
                 q_offsets=_dev(qs, torch.int64), lengths=_dev(kv, torch.int32))
        s["bounds_dev"] = _dev(s["bounds"], torch.int64)
        # the new events' slots, as building the tables gave them
        seq = torch.repeat_interleave(torch.arange(B, device=DEV), s["q_offsets"].diff())
        at = s["lengths"][seq] - s["q_offsets"][seq + 1] + torch.arange(qs[-1], device=DEV)
        s["slots"] = s["table"][seq, at // page].long() * page + at % page
        return s
    lens = [1] * B if op == "step" else _lens(case, seed)[0]
    at = _starts(lens)
    N = at[-1]
    s.update(q=_normal(g, N, Hq, d, dtype=bf), k=_normal(g, N, Hkv, d, dtype=bf), v=_normal(g, N, Hkv, d, dtype=bf),
             offsets=_dev(at, torch.int64), longest=max(lens))
    if case["each"]:  # by the time since the event before: mostly short, now and then a long pause
        gap = torch.exp(_normal(g, N, Hkv)) * 0.05
        s["g"] = -torch.where(torch.rand(N, 1, generator=g, device=DEV) < 0.02, 15.0, gap)
    else:
        s["g"] = -torch.exp2(-2.0 - torch.arange(Hkv, device=DEV)) * (1 + 0.1 * torch.rand(Hkv, generator=g, device=DEV))
    if op == "train":
        s["do"] = _normal(g, N, Hq, d, dtype=bf)
    else:
        s["state"] = _normal(g, B, Hkv, d, d, std=2.0)
    return s


# ------------------------------------------------------------------------------- the plain forms

def _plain_pages(s):
    page, table, held, free = s["case"]["page"], s["table"], s["lengths"].long(), s["free"]
    offsets, width = s["offsets"], s["table"].shape[1]
    col = torch.arange(width, device=DEV)
    leave = held + s["new"] > s["case"]["cap"]
    have = (held + page - 1) // page
    # what those who leave held goes back onto the stack
    gone = torch.where(leave, have, 0)
    back = leave[:, None] & (col < have[:, None])
    to = s["free_count"] + (gone.cumsum(0) - gone)[:, None] + col
    free = torch.cat((free, free.new_zeros(1)))
    free[torch.where(back, to, free.shape[0] - 1)] = table
    free = free[:-1]
    top = s["free_count"] + gone.sum()
    held, have = torch.where(leave, 0, held), torch.where(leave, 0, have)
    table = torch.where(leave[:, None], -1, table)
    # those who grow take from its top, in order, as far as it goes
    n = offsets.diff()
    wide = held + n <= width * page
    want = torch.where(wide, (held + n + page - 1) // page - have, 0)
    upto = want.cumsum(0)
    fits = wide & ((want == 0) | (upto <= top))
    take = torch.where(fits, want, 0)
    k = (upto - want)[:, None] + col - have[:, None]
    fresh = (col >= have[:, None]) & (col < (have + take)[:, None])
    table = torch.where(fresh, free[torch.where(fresh, top - 1 - k, 0)], table)
    row = torch.arange(s["n"], device=DEV)
    seq = torch.searchsorted(offsets, row, right=True) - 1
    at = held[seq] + row - offsets[seq]
    slots = table[seq, (at // page).clamp(max=width - 1)].long() * page + at % page
    slots = torch.where(fits[seq], slots, -1)
    s["table"], s["free"] = table, free
    s["lengths"] = torch.where(fits, held + n, held).to(torch.int32)
    s["free_count"] = (top - take.sum()).to(torch.int32)
    return {"slots": slots, "table": s["table"], "lengths": s["lengths"], "free": s["free"], "free_count": s["free_count"],
            "refused": (~fits).sum().to(torch.int32).view(1)}


def _padded(x, offsets, longest):
    """[B, longest, H, d] of the jagged [tokens, H, d] in fp32, zeros past a sequence's end; and
    which places hold a token."""
    at = offsets[:-1, None] + torch.arange(longest, device=DEV)
    live = at < offsets[1:, None]
    full = torch.cat([x, x.new_zeros(1, *x.shape[1:])])
    return full[torch.where(live, at, x.shape[0])].float(), live


def _visible(n, j, window, sinks):
    """Key j is seen from n keys further on: not later, and inside the window or one of the first."""
    return (n >= 0) & ((n < window) | (j < sinks)) if window else n >= 0


def _rows(x, heads):
    """[B, L, H, d] with the query heads that share a key/value head as rows: [B * heads, H / heads * L, d]."""
    B, L, H, d = x.shape
    return x.view(B, L, heads, H // heads, d).permute(0, 2, 3, 1, 4).reshape(B * heads, -1, d)


def _jagged(x, live, heads, B):
    """The inverse of _rows, tokens laid end to end, in bf16."""
    return x.reshape(B, heads, live.shape[1], x.shape[-1]).permute(0, 2, 1, 3)[live].to(torch.bfloat16)


def _plain_paged(s):
    c = s["case"]
    Hq, Hkv, d, page = c["Hq"], c["Hkv"], c["d"], c["page"]
    s["k"][s["slots"]] = s["k_new"]
    s["v"][s["slots"]] = s["v_new"]
    j = torch.arange(s["max_kv"], device=DEV)
    live = j < s["lengths"][:, None]
    at = torch.where(live, s["table"][:, j // page].long() * page + j % page, 0)
    k = torch.where(live[..., None, None], s["k"][at], 0).float()
    v = torch.where(live[..., None, None], s["v"][at], 0).float()
    q, q_live = _padded(s["q"], s["q_offsets"], s["max_q"])
    B, Lq, Lk = q.shape[0], q.shape[1], k.shape[1]
    n = (s["lengths"] - s["q_offsets"].diff())[:, None, None] + torch.arange(Lq, device=DEV)[:, None] - j
    see = _visible(n, j, c["window"], c["sinks"]) & live[:, None, :] & q_live[:, :, None]
    bucket = torch.searchsorted(s["bounds_dev"], n.clamp(min=0), right=True) - 1
    logits = torch.bmm(_rows(q, Hkv), _rows(k, Hkv).transpose(1, 2)).view(B, Hkv, Hq // Hkv, Lq, Lk) / math.sqrt(d)
    logits = logits + s["bias"].view(Hkv, Hq // Hkv, -1)[:, :, bucket].permute(2, 0, 1, 3, 4)
    logits = torch.where(see[:, None, None], logits, float("-inf"))
    top = logits.amax(-1, keepdim=True)
    e = torch.exp(logits - torch.where(torch.isinf(top), 0.0, top))
    del logits
    total = e.sum(-1, keepdim=True)
    P = e / torch.where(total == 0, 1.0, total)
    o = torch.bmm(P.view(B * Hkv, -1, Lk), _rows(v, Hkv))
    return {"o": _jagged(o, q_live, Hq, B)}


def _plain_decay(s):
    c = s["case"]
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    group, scale = Hq // Hkv, 1.0 / math.sqrt(d)
    q, live = _padded(s["q"], s["offsets"], s["longest"])
    k, _ = _padded(s["k"], s["offsets"], s["longest"])
    v, _ = _padded(s["v"], s["offsets"], s["longest"])
    B, L = live.shape
    q, k, v = _rows(q, Hkv), _rows(k, Hkv), _rows(v, Hkv)
    # differences of the decays' sums, which grow with the length, in 64 bits
    g = s["g"] if s["g"].dim() == 2 else s["g"].expand(s["q"].shape[0], Hkv)
    G = _padded(g[:, :, None], s["offsets"], s["longest"])[0][..., 0].double().cumsum(1).transpose(1, 2)  # [B, Hkv, L]
    gap = (G[..., :, None] - G[..., None, :]).float()
    causal = torch.ones(L, L, dtype=torch.bool, device=DEV).tril()
    D = torch.where(causal, torch.exp(torch.where(causal, gap, 0.0)), 0.0).reshape(B * Hkv, 1, L, L)
    del gap
    A = torch.bmm(q, k.transpose(1, 2)).reshape(B * Hkv, group, L, L)
    W = A * D * scale
    o = torch.bmm(W.reshape(B * Hkv, group * L, L), v)
    if c["op"] == "state":
        S = s["state"].reshape(B * Hkv, d, d)
        first = torch.exp(G).float().reshape(B * Hkv, 1, L, 1)
        o = o.reshape(B * Hkv, group, L, d) + first * torch.bmm(q, S).reshape(B * Hkv, group, L, d) * scale
        last = G[..., -1:]  # no decay past a sequence's end
        w = torch.exp(last - G).float().reshape(B * Hkv, L, 1) * live.repeat_interleave(Hkv, 0)[..., None]
        state = torch.exp(last).float().reshape(-1, 1, 1) * S + torch.bmm((w * k).transpose(1, 2).contiguous(), v)
        return {"o": _jagged(o.reshape(B * Hkv, group * L, d), live, Hq, B), "state": state.reshape(B, Hkv, d, d)}
    do = _rows(_padded(s["do"], s["offsets"], s["longest"])[0], Hkv)
    M = torch.bmm(do, v.transpose(1, 2)).reshape(B * Hkv, group, L, L) * D * scale
    dq = torch.bmm(M.reshape(B * Hkv, group * L, L), k)
    dk = torch.bmm(M.reshape(B * Hkv, group * L, L).transpose(1, 2), q)
    dv = torch.bmm(W.reshape(B * Hkv, group * L, L).transpose(1, 2), do)
    # a pair's part reaches the decays between its two events: those whose query is at t or later, less
    # those whose key is
    T = A * M
    dG = (T.sum((1, 3), dtype=torch.float64) - T.sum((1, 2), dtype=torch.float64)).reshape(B, Hkv, L)
    dg = dG.flip(-1).cumsum(-1).flip(-1).permute(0, 2, 1)[live]
    dg = dg.float() if s["g"].dim() == 2 else dg.sum(0).float()
    return {"o": _jagged(o, live, Hq, B), "dq": _jagged(dq, live, Hq, B), "dk": _jagged(dk, live, Hkv, B),
            "dv": _jagged(dv, live, Hkv, B), "dg": dg}


def _plain_step(s):
    c = s["case"]
    g = s["g"] if s["g"].dim() == 2 else s["g"].expand(c["B"], c["Hkv"])
    k, v = s["k"].float(), s["v"].float()
    state = torch.exp(g)[..., None, None] * s["state"] + k[..., :, None] * v[..., None, :]
    s["state"].copy_(state)
    q = s["q"].float().view(c["B"], c["Hkv"], c["Hq"] // c["Hkv"], 1, c["d"])
    o = torch.matmul(q, state[:, :, None]).view(c["B"], c["Hq"], c["d"]) / math.sqrt(c["d"])
    return {"o": o.to(torch.bfloat16), "state": s["state"]}


# ----------------------------------------------------------------------------- the framework's own

def _own(s):
    import recommendation_model_sparse_amd as fw
    c = s["case"]
    op = c["op"]
    if op == "pages":
        leave = s["lengths"] + s["new"] > c["cap"]
        slots, refused = fw.dlrm_seq_pages_update(s["table"], s["lengths"], s["free"], s["free_count"], c["page"], s["offsets"],
                                                  s["n"], leave)
        return {"slots": slots, "table": s["table"], "lengths": s["lengths"], "free": s["free"], "free_count": s["free_count"],
                "refused": refused}
    if op in ("decode", "prefill"):
        how = dict(window=c["window"], sinks=c["sinks"], bias=s["bias"], bounds=s["bounds"])
        fw.dlrm_seq_pages_write(s["k_new"], s["v_new"], s["slots"], s["k"], s["v"])
        if op == "prefill":
            return {"o": fw.dlrm_seq_attn_paged_fwd(s["q"], s["k"], s["v"], s["q_offsets"], s["table"], s["lengths"], c["page"], **how)}
        return {"o": fw.dlrm_seq_attn_paged_decode(s["q"], s["k"], s["v"], s["table"], s["lengths"], c["page"],
                                                   max_kv_len=s["max_kv"], **how)}
    if op == "step":
        return {"o": fw.dlrm_seq_decay_step(s["q"], s["k"], s["v"], s["g"], s["state"]), "state": s["state"]}
    if op == "state":
        o, state = fw.dlrm_seq_decay_fwd(s["q"], s["k"], s["v"], s["g"], s["offsets"], state=s["state"], want_state=True,
                                         max_len=s["longest"])
        return {"o": o, "state": state}
    o = fw.dlrm_seq_decay_fwd(s["q"], s["k"], s["v"], s["g"], s["offsets"], max_len=s["longest"])
    dq, dk, dv, dg = fw.dlrm_seq_decay_bwd(s["do"], s["q"], s["k"], s["v"], s["g"], s["offsets"], max_len=s["longest"])
    return {"o": o, "dq": dq, "dk": dk, "dv": dv, "dg": dg}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "pages":
        return _plain_pages(state)
    if op in ("decode", "prefill"):
        return _plain_paged(state)
    return _plain_step(state) if op == "step" else _plain_decay(state)


# ------------------------------------------------------------------------------------ the work

def work(case):
    op, B = case["op"], case["B"]
    if op == "pages":
        # offsets, lengths in and out, who leaves; the slots; the new pages off the stack and into the tables
        _, new = _lens(case, 0)
        n = sum(new)
        grown = sum(max(1, m // case["page"]) for m in new) if case["new"] > 1 else B // case["page"]
        return {"bytes": 17 * B + 8 * n + 8 * grown, "flops": 4 * n + 8 * B}
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if op in ("decode", "prefill"):
        kv, new = _lens(case, 0)
        W, S = case["window"], case["sinks"]
        pairs = read = table = 0
        for n, m in zip(kv, new):
            first = n - m
            if not W:
                pairs += m * n - m * (m - 1) // 2
                seen = n
            else:
                pairs += sum(min(p + 1, W) + min(S, max(0, p + 1 - W)) for p in range(first, n))
                start = max(0, first - W + 1)
                seen = n - start + min(S, start)
            read += max(0, seen - m)
            table += -(-seen // case["page"])
        nq = sum(new)  # the new events' rows are read once and written to their slots
        return {"bytes": 4 * nq * Hq * d + 4 * (read + 2 * nq) * Hkv * d + 4 * table + 4 * Hq * case["buckets"],
                "flops": 4 * pairs * Hq * d}
    state = 4 * B * Hkv * d * d
    if op == "step":
        return {"bytes": 2 * state + 4 * B * (Hq + Hkv) * d, "flops": 2 * B * d * d * (Hq + 2 * Hkv)}
    N = sum(_lens(case, 0)[0])
    qb, kb, gb = 2 * N * Hq * d, 2 * N * Hkv * d, 4 * Hkv * (N if case["each"] else 1)
    if op == "state":
        return {"bytes": 2 * qb + 2 * kb + gb + 2 * state, "flops": 2 * N * d * d * (Hq + Hkv)}
    # q do o dq, k v dk dv, g dg; forward a state's update and its product with q, backward those of dq,
    # of the gradient's state, dk and dv
    return {"bytes": 4 * qb + 4 * kb + 2 * gb, "flops": 2 * N * d * d * (3 * Hq + 3 * Hkv)}


# ------------------------------------------------------------------------------ exact, in 64 bits

def _exact_paged(s):
    c = s["case"]
    Hq, Hkv, d, page = c["Hq"], c["Hkv"], c["d"], c["page"]
    qs, lens, table = s["q_offsets"].tolist(), s["lengths"].tolist(), s["table"].tolist()
    head = torch.arange(Hq, device=DEV) // (Hq // Hkv)
    edge = _dev(s["bounds"][1:], torch.int64)
    out = []
    for b, n in enumerate(lens):
        pages = [s["k"].view(-1, page, Hkv, d)[table[b][:-(-n // page)]], s["v"].view(-1, page, Hkv, d)[table[b][:-(-n // page)]]]
        old = [x.reshape(-1, Hkv, d)[:n - (qs[b + 1] - qs[b])] for x in pages]
        k, v = (torch.cat((x, y[qs[b]:qs[b + 1]])).double() for x, y in zip(old, (s["k_new"], s["v_new"])))
        q = s["q"][qs[b]:qs[b + 1]].double()
        at = torch.arange(n - len(q), n, device=DEV)[:, None]
        j = torch.arange(n, device=DEV)[None]
        hidden = (j > at) | ((at - j >= c["window"]) & (j >= c["sinks"]) if c["window"] else j < 0)
        z = torch.stack([q[:, h] @ k[:, head[h]].T for h in range(Hq)]) / d ** 0.5
        z = z + s["bias"].double()[:, torch.bucketize(at - j, edge, right=True)]
        a = torch.softmax(z.masked_fill(hidden, -math.inf), -1)
        out.append(torch.stack([a[h] @ v[:, head[h]] for h in range(Hq)], 1))
    return {"o": torch.cat(out)}


def _exact_decay(s):
    c = s["case"]
    Hq, Hkv, d, train = c["Hq"], c["Hkv"], c["d"], c["op"] == "train"
    at = s["offsets"].tolist()
    parts = {"o": [], "dq": [], "dk": [], "dv": [], "dg": [], "state": []}
    group = Hq // Hkv
    for b in range(len(at) - 1):
        rows = slice(at[b], at[b + 1])
        n = at[b + 1] - at[b]
        if not n:
            if not train:
                parts["state"].append(s["state"][b].double())
            continue
        q, k, v = (s[x][rows].double().requires_grad_(train) for x in "qkv")
        g = (s["g"][rows] if c["each"] else s["g"].expand(n, Hkv)).double().contiguous().requires_grad_(train)
        total = torch.cat((g.new_zeros(1, Hkv), g.cumsum(0))).T  # [Hkv, n + 1]: up to an event, from the first on
        outs, states = [], []
        for h in range(Hkv):
            age = total[h, 1:, None] - total[h, None, 1:]
            keep = torch.exp(age.masked_fill(torch.ones_like(age, dtype=torch.bool).triu(1), -math.inf))
            for i in range(h * group, (h + 1) * group):
                o = (q[:, i] @ k[:, h].T * keep) @ v[:, h]
                if not train:
                    o = o + torch.exp(total[h, 1:, None]) * (q[:, i] @ s["state"][b, h].double())
                outs.append(o / d ** 0.5)
            if not train:
                states.append(torch.exp(total[h, -1]) * s["state"][b, h].double() + (keep[-1][:, None] * k[:, h]).T @ v[:, h])
        o = torch.stack(outs, 1)
        parts["o"].append(o.detach())
        if train:
            for name, x in zip(("dq", "dk", "dv", "dg"), torch.autograd.grad(o, (q, k, v, g), s["do"][rows].double())):
                parts[name].append(x)
        else:
            parts["state"].append(torch.stack(states))
    if not train:
        return {"o": torch.cat(parts["o"]), "state": torch.stack(parts["state"])}
    out = {name: torch.cat(parts[name]) for name in ("o", "dq", "dk", "dv", "dg")}
    if not c["each"]:
        out["dg"] = out["dg"].sum(0)
    return out


def exact(case, seed):
    if case["op"] == "pages":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] in ("decode", "prefill"):
        return _exact_paged(s)
    if case["op"] != "step":
        return _exact_decay(s)
    head = torch.arange(case["Hq"], device=DEV) // (case["Hq"] // case["Hkv"])
    decay = torch.exp(s["g"].double().expand(case["B"], case["Hkv"]))
    S = torch.einsum("bhc,bhe->bhce", s["k"].double(), s["v"].double())
    S += decay[..., None, None] * s["state"].double()
    o = torch.einsum("bhc,bhce->bhe", s["q"].double(), S[:, head]) / case["d"] ** 0.5
    return {"o": o, "state": S}
