"""GPU parity of the paged cache (dlrm_seq_pages.h; needs an MI355X): the visit's tables, lengths and slots against
oracle/pages.py, entry by entry; attention over pages against the calls over rows that lie together, bit by bit (the
same products in the same order).

A few users' new events take the keys of a tile in parts, another order: either side rounds P and its
output to bf16 (2^-8 each of sum P |v|, which the call over |v| gives to 2^-6), so they are at most 2^-6 (1 + 2^-6) of it apart."""
import zlib

import numpy as np
import pytest
import torch

from oracle import pages as oracle
from recommendation_model_sparse_amd import (dlrm_seq_attn_decode, dlrm_seq_attn_fwd, dlrm_seq_attn_paged_decode,
                                             dlrm_seq_attn_paged_fwd, dlrm_seq_bucket_bounds, dlrm_seq_pages_update,
                                             dlrm_seq_pages_write)

from gpu_util import DEV, say, to_dev

pytestmark = pytest.mark.gpu


def rng_of(*a):
    return np.random.default_rng(zlib.crc32("-".join(map(str, a)).encode()))


def offsets(counts, dtype=np.int64):
    return np.cumsum([0] + list(counts)).astype(dtype)


def new_pool(B, width, pages):
    return [np.full((B, width), -1, np.int32), np.zeros(B, np.int32), np.arange(pages, dtype=np.int32), pages]


def visit(pool, page, off, n, leave, where=None):
    """One visit on the GPU (`where`: the device's buffers, which go on) and in Python; they must agree."""
    table, lengths, free, top = pool
    where = where or [to_dev(table), to_dev(lengths), to_dev(free), torch.tensor([top], dtype=torch.int32, device=DEV)]
    slots = torch.full((n,), -7, dtype=torch.int64, device=DEV)
    got, refused = dlrm_seq_pages_update(*where, page, to_dev(off), n, None if leave is None else to_dev(leave), slots=slots)
    torch.cuda.synchronize()
    want = oracle.update(table, lengths, free, top, page, off, n, leave)
    assert int(refused) == want[5]
    for x, y in zip(where + [got], want[:3] + (np.array([want[3]], np.int32), want[4])):
        assert np.array_equal(x.cpu().numpy(), y)
    return list(want[:4]), where


@pytest.mark.parametrize("B,page,width,pages,most", [
    (1, 8, 4, 4, 9), (5, 8, 10, 40, 30), (5, 64, 3, 6, 100), (64, 16, 8, 300, 40), (256, 16, 32, 6000, 1), (1023, 8, 6, 4000, 12), (1024, 8, 6, 4000, 20),
    (1025, 8, 6, 4000, 12), (1500, 4096, 2, 2000, 3000), (3000, 16, 9, 9000, 50), (2500, 32, 20, 50000, 200), (700, 8, 40, 20000, 100)])
@pytest.mark.parametrize("itype", [np.int64, np.int32])
def test_visits(B, page, width, pages, most, itype):
    """Visits one after the other: users come, grow, leave and come back, and are refused where their table or the pool
    is too small."""
    rng = rng_of("pages", B, page, width)
    pool, where = new_pool(B, width, pages), None
    rng.shuffle(pool[2])
    say(f"[pages] B={B} page={page} width={width} pages={pages} most={most} {itype.__name__}")
    total = 0
    for turn in range(6):
        counts = rng.integers(0, most + 1, B)
        if turn == 3:
            counts[rng.random(B) < 0.7] = 0
        leave = None if turn in (0, 4) else rng.random(B) < (1.0 if turn == 5 else 0.3)
        off = offsets(counts, itype)
        before = pool
        pool, where = visit(pool, page, off, int(off[-1]) + 3, leave, where)
        total += int(off[-1])
        held = pool[0][pool[0] >= 0]
        assert len(np.unique(held)) == len(held) and len(held) + pool[3] == pages
        del before
    assert total


@pytest.mark.parametrize("others", [0, 1100])
def test_whom_a_refused_user_refuses(others):
    """By hand, of a pool of four pages of 8: one user gets its page, one's table is too short, one wants 13 pages; the next
    wants one, which is there, and is refused with it; the last one's events fit the page that it holds."""
    B = others + 5
    held, counts = np.zeros(B, np.int64), np.zeros(B, np.int64)
    held[-1], counts[-5:] = 3, [1, 200, 100, 8, 2]
    say(f"[pages] whom a refused user refuses, {B} users")
    pool, where = visit(new_pool(B, 16, 4), 8, offsets(held), 3, None)
    assert pool[0][-1, 0] == 3 and pool[3] == 3
    pool, where = visit(pool, 8, offsets(counts), 311, None, where)
    table, lengths, _, count = (x.cpu().numpy() for x in where)
    assert lengths[-5:].tolist() == [1, 0, 0, 0, 5] and not lengths[:-5].any() and count[0] == 2
    assert table[-5:, 0].tolist() == [2, -1, -1, -1, 3]


def test_slots_outside_the_users_are_left():
    """Offsets that begin past 0 and end before n."""
    pool = new_pool(3, 4, 12)
    say("[pages] rows outside")
    visit(pool, 8, np.array([5, 9, 9, 20], np.int64), 30, None)
    visit(new_pool(1200, 4, 5000), 8, 5 + offsets([3] * 1200), 3700, None)
    visit(new_pool(2, 4000, 9000), 8, 5 + offsets([20000, 7000]), 28000, None)


def test_nobody():
    say("[pages] nobody")
    one = torch.tensor([3], dtype=torch.int32, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    for n in (0, 20000):
        slots, refused = dlrm_seq_pages_update(torch.zeros((0, 2), **i32), torch.zeros(0, **i32), torch.arange(3, **i32), one, 16,
                                               torch.zeros(1, dtype=torch.int64, device=DEV), n, slots=torch.full((n,), -7, dtype=torch.int64, device=DEV))
        torch.cuda.synchronize()
        assert int(refused) == 0 and (slots == -7).all() and int(one) == 3
    pool = new_pool(4, 0, 3)  # no pages a user: all events are refused
    visit(pool, 16, offsets([2, 0, 1, 0]), 3, None)


def test_a_table_with_longer_rows():
    """Rows of a wider table: the entries beside them stay."""
    i32 = dict(dtype=torch.int32, device=DEV)
    wide = torch.full((5, 9), 77, **i32)
    wide[:, 2:6] = -1
    lengths, free, count = torch.zeros(5, **i32), torch.arange(30, **i32), torch.tensor([30], **i32)
    off = offsets([8, 0, 20, 31, 1])
    say("[pages] a wider table")
    slots, _ = dlrm_seq_pages_update(wide[:, 2:6], lengths, free, count, 8, to_dev(off), 60)
    torch.cuda.synchronize()
    want = oracle.update(np.full((5, 4), -1, np.int32), np.zeros(5, np.int32), np.arange(30), 30, 8, off, 60)
    assert np.array_equal(wide[:, 2:6].cpu().numpy(), want[0]) and (wide[:, :2] == 77).all() and (wide[:, 6:] == 77).all()
    assert np.array_equal(slots.cpu().numpy(), want[4])


@pytest.mark.parametrize("B", [6, 1300])
def test_contents_that_cannot_be(B):
    """Lengths, counts and offsets outside of what can be: nothing outside the buffers is written."""
    rng = rng_of("pages-bad", B)
    i32 = dict(dtype=torch.int32, device=DEV)
    say(f"[pages] bad contents B={B}")
    for turn in range(6):
        room = torch.full((B + 4, 8), 55, **i32)
        table = room[2:B + 2]
        table.copy_(torch.from_numpy(rng.integers(-5, 1 << 30, (B, 8)).astype(np.int32)))
        lengths = to_dev(rng.integers(-1000, 100000, B).astype(np.int32))
        stack = torch.full((104,), 66, **i32)
        stack[2:102] = to_dev(rng.integers(-9, 1 << 30, 100).astype(np.int32))
        count = torch.tensor([[-5, 3, 100, 101, 1 << 30, 50][turn]], **i32)
        off = rng.integers(-100, 3000, B + 1)
        slots = torch.full((2048,), -7, dtype=torch.int64, device=DEV)
        leave = to_dev(rng.random(B) < 0.5)
        dlrm_seq_pages_update(table, lengths, stack[2:102], count, 16, to_dev(off), 1024, leave, slots=slots[512:1536])
        torch.cuda.synchronize()
        assert (room[:2] == 55).all() and (room[B + 2:] == 55).all() and (stack[:2] == 66).all() and (stack[102:] == 66).all()
        assert (slots[:512] == -7).all() and (slots[1536:] == -7).all()


@pytest.mark.parametrize("H,d", [(1, 8), (3, 40), (2, 128)])
def test_write(H, d):
    """Strided rows to slots in any order; those outside the pool are passed over."""
    rng = rng_of("pages-write", H, d)
    N, rows = 77, 200
    joint = torch.randn((N, 2 * H, d), device=DEV).bfloat16()
    k, v = joint[:, :H], joint[:, H:]
    slots = rng.permutation(rows)[:N].astype(np.int64)
    slots[[3, 10, 50]] = [-1, rows, 1 << 40]
    pools = [torch.full((rows, H, d), 9.0, dtype=torch.bfloat16, device=DEV), torch.full((H, rows, d), 9.0, dtype=torch.bfloat16, device=DEV).transpose(0, 1)]
    want = [p.clone() for p in pools]
    keep = (slots >= 0) & (slots < rows)
    for w, x in zip(want, (k, v)):
        w[to_dev(slots[keep])] = x[to_dev(np.flatnonzero(keep))]
    say(f"[pages] write H={H} d={d}")
    dlrm_seq_pages_write(k, v, to_dev(slots), *pools)
    torch.cuda.synchronize()
    assert all(torch.equal(p, w) for p, w in zip(pools, want))
    dlrm_seq_pages_write(k[:0], v[:0], to_dev(slots[:0]), *pools)
    torch.cuda.synchronize()
    assert all(torch.equal(p, w) for p, w in zip(pools, want))


def paged(rng, lens, page, Hkv, d, spare=3):
    """Keys and values that lie together, and the same in pages of a pool that holds NaN elsewhere."""
    off = offsets(lens)
    N = int(off[-1])
    k, v = (torch.randn((N, Hkv, d), device=DEV).bfloat16() for _ in range(2))
    have = [-(-n // page) for n in lens]
    pages = sum(have) + spare
    order = rng.permutation(pages)
    table, at = np.full((len(lens), max(have + [1]) + 1), -1, np.int32), 0
    rows = np.zeros(N, np.int64)
    for b, n in enumerate(lens):
        table[b, :have[b]] = order[at:at + have[b]]
        j = np.arange(n)
        rows[off[b]:off[b + 1]] = table[b, j // page].astype(np.int64) * page + j % page
        at += have[b]
    pools = [torch.full((pages * page, Hkv, d), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    dlrm_seq_pages_write(k, v, to_dev(rows), *pools)
    return off, k, v, pools, to_dev(table), to_dev(np.array(lens, np.int32))


def how_of(rng, Hq, window, sinks, buckets):
    how = dict(window=window, sinks=sinks)
    if buckets:
        how.update(bias=to_dev(rng.standard_normal((Hq, buckets)).astype(np.float32)), bounds=dlrm_seq_bucket_bounds(buckets, 200))
    return how


def check_several(got, want, call, v):
    """`call`: the attention over rows that lie together, of v."""
    room = 2.0 ** -6 * (1 + 2.0 ** -6) * call(v.abs()).float()
    assert ((got.float() - want.float()).abs() <= room).all()


CASES = [
    # lens, page, Hq, Hkv, d, window, sinks, buckets
    ([1], 8, 1, 1, 8, 0, 0, 0), ([5, 0, 17, 64], 8, 4, 2, 32, 0, 0, 8), ([63, 64, 65, 1], 64, 2, 1, 64, 0, 0, 8), ([300, 7, 129], 16, 8, 2, 128, 0, 0, 32),
    ([300, 7, 129], 32, 4, 4, 40, 50, 3, 16), ([700, 1000], 256, 6, 2, 96, 300, 70, 0), ([2000, 3, 900], 8, 40, 2, 64, 0, 0, 32), ([5000, 10], 512, 2, 1, 64, 0, 0, 0),
    ([40] * 300, 16, 2, 1, 32, 0, 0, 8), ([0, 0], 16, 2, 1, 32, 0, 0, 0), ([130, 3, 40] * 500, 16, 2, 1, 64, 0, 0, 8), ([70] * 1400, 32, 2, 2, 32, 30, 2, 8),
    ([130, 70, 9] * 60, 16, 4, 2, 64, 0, 0, 8), ([200, 90] * 30, 8, 8, 1, 128, 100, 130, 32), ([600, 1], 128, 2, 2, 32, 150, 130, 8), ([900, 300], 64, 2, 1, 128, 200, 5, 16),
    ([70] * 1400, 32, 2, 1, 128, 30, 2, 8)]


@pytest.mark.parametrize("lens,page,Hq,Hkv,d,window,sinks,buckets", CASES)
def test_one_event_over_pages(lens, page, Hq, Hkv, d, window, sinks, buckets):
    rng = rng_of("paged-decode", lens[:3], page, d, window)
    off, k, v, pools, table, lengths = paged(rng, lens, page, Hkv, d)
    q = torch.randn((len(lens), Hq, d), device=DEV).bfloat16()
    how = how_of(rng, Hq, window, sinks, buckets)
    off = to_dev(off)
    say(f"[pages] one event page={page} d={d} window={window}")
    for longest in (max(lens), 1, 70000):
        want = dlrm_seq_attn_decode(q, k, v, off[:-1], off[1:], max_kv_len=longest, **how)
        got = dlrm_seq_attn_paged_decode(q, *pools, table, lengths, page, max_kv_len=longest, **how)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    dlrm_seq_attn_paged_decode(q, *pools, table, lengths, page, **how)


@pytest.mark.parametrize("lens,page,Hq,Hkv,d,window,sinks,buckets", CASES)
def test_new_events_over_pages(lens, page, Hq, Hkv, d, window, sinks, buckets):
    rng = rng_of("paged-fwd", lens[:3], page, d, window)
    off, k, v, pools, table, lengths = paged(rng, lens, page, Hkv, d)
    new = [int(rng.integers(0, n + 1)) for n in lens]
    qo = to_dev(offsets(new))
    q = torch.randn((sum(new), Hq, d), device=DEV).bfloat16()
    how = how_of(rng, Hq, window, sinks, buckets)
    say(f"[pages] new events page={page} d={d} window={window}")
    want = dlrm_seq_attn_fwd(q, k, v, qo, to_dev(off), **how)
    got = dlrm_seq_attn_paged_fwd(q, *pools, qo, table, lengths, page, **how)
    narrow = dlrm_seq_attn_paged_fwd(q, *pools, qo.int(), table[:, :], lengths, page, **how)
    torch.cuda.synchronize()
    assert torch.equal(got, narrow)
    if len(lens) > 1000:  # many users: no parts
        assert torch.equal(got, want)
    check_several(got, want, lambda x: dlrm_seq_attn_fwd(q, k, x, qo, to_dev(off), **how), v)


@pytest.mark.parametrize("users", [1, 30, 700])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_what_is_not_finite_and_what_is_large(users, d):
    """Infinities and NaN in keys and values, which queries before them do not see, and values whose sum passes the largest
    number before it is divided: the same of them as over rows that lie together."""
    rng = rng_of("paged-wild", users, d)
    off, k, v, _, _, lengths = paged(rng, [300, 150] * users, 16, 1, d)
    for b in range(2 * users):
        x = int(off[b])
        if b % 2 == 0:
            v[x + 120, 0, 3], v[x + 130, 0, 5], k[x + 200, 0, 1] = float("inf"), float("-inf"), float("nan")
        else:
            v[x:x + 150] = 3e38
    have = [19, 10] * users
    at = np.concatenate([[0], np.cumsum(have)])
    pools = [torch.zeros((int(at[-1]) * 16, 1, d), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    table = np.full((2 * users, 19), -1, np.int32)
    rows = np.zeros(int(off[-1]), np.int64)
    for b in range(2 * users):
        table[b, :have[b]] = np.arange(at[b], at[b + 1])
        rows[off[b]:off[b + 1]] = at[b] * 16 + np.arange(off[b + 1] - off[b])
    dlrm_seq_pages_write(k, v, to_dev(rows), *pools)
    qo = to_dev(offsets([200, 150] * users))
    q = torch.randn((350 * users, 2, d), device=DEV).bfloat16()
    say(f"[pages] not finite, {users} users, d={d}")
    want = dlrm_seq_attn_fwd(q, k, v, qo, to_dev(off)).float()
    got = dlrm_seq_attn_paged_fwd(q, *pools, qo, to_dev(table), lengths, 16).float()
    room = 2.0 ** -6 * (1 + 2.0 ** -6) * dlrm_seq_attn_fwd(q, k, v.abs(), qo, to_dev(off)).float()
    torch.cuda.synchronize()
    finite = torch.isfinite(want)
    assert finite.any() and (~finite).any() and torch.equal(torch.isfinite(got), finite) and torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)])
    assert ((got - want).abs() <= room)[finite].all()


def test_heads_that_lie_apart_and_a_wider_pool():
    """A joint pool of keys and values, rows of a wider table."""
    rng = rng_of("paged-strides")
    off, k, v, pools, table, lengths = paged(rng, [100, 37], 16, 2, 64)
    joint = torch.cat(pools, 1)  # [rows, 4, 64]: keys and values of a row side by side
    wide = torch.full((2, 20), 1 << 20, dtype=torch.int32, device=DEV)
    wide[:, 3:3 + table.shape[1]] = table
    part = wide[:, 3:3 + table.shape[1]]
    q = torch.randn((2, 4, 64), device=DEV).bfloat16()
    off = to_dev(off)
    say("[pages] strides")
    want = dlrm_seq_attn_decode(q, k, v, off[:-1], off[1:])
    got = dlrm_seq_attn_paged_decode(q, joint[:, :2], joint[:, 2:], part, lengths, 16)
    assert torch.equal(got, want)
    qo = to_dev(offsets([1, 1]))
    check_several(dlrm_seq_attn_paged_fwd(q, joint[:, :2], joint[:, 2:], qo, part, lengths, 16), dlrm_seq_attn_fwd(q, k, v, qo, off),
                  lambda x: dlrm_seq_attn_fwd(q, k, x, qo, off), v)


def test_tables_that_cannot_be():
    """Pages outside the pool count as its last one, lengths past the table as what it holds: the others' results are
    what they were."""
    rng = rng_of("paged-bad")
    off, k, v, pools, table, lengths = paged(rng, [100, 37, 64], 16, 1, 64)
    q = torch.randn((3, 2, 64), device=DEV).bfloat16()
    qo = to_dev(offsets([1, 1, 1]))
    want = dlrm_seq_attn_paged_decode(q, *pools, table, lengths, 16)
    pools = [p.nan_to_num(1.0) for p in pools]
    bad, long = table.clone(), lengths.clone()
    bad[1] = to_dev(rng.integers(-(1 << 31), 1 << 31, table.shape[1]).astype(np.int32))
    long[1] = 1 << 30
    say("[pages] bad tables")
    one = dlrm_seq_attn_paged_decode(q, *pools, bad, long, 16)
    several = dlrm_seq_attn_paged_fwd(q, *pools, qo, bad, long, 16)
    long[1] = -5
    none = dlrm_seq_attn_paged_decode(q, *pools, bad, long, 16)
    torch.cuda.synchronize()
    for b in (0, 2):
        assert torch.equal(one[b], want[b]) and torch.equal(none[b], want[b])
        assert torch.equal(several[b], dlrm_seq_attn_paged_fwd(q, *pools, qo, table, lengths, 16)[b])
    assert torch.isfinite(one.float()).all() and torch.isfinite(several.float()).all() and (none[1] == 0).all()


def test_a_pool_past_two_to_the_31_elements():
    """Its last page lies past 2^31 elements."""
    page, Hkv, d = 64, 8, 128
    pages = (1 << 31) // (page * Hkv * d) + 40
    pools = [torch.zeros((pages * page, Hkv, d), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    n = 150
    k, v = (torch.randn((n, Hkv, d), device=DEV).bfloat16() for _ in range(2))
    table = torch.tensor([[pages - 1, pages - 30, 2]], dtype=torch.int32, device=DEV)
    j = torch.arange(n, device=DEV)
    slots = table[0, j // page].long() * page + j % page
    say("[pages] a large pool")
    dlrm_seq_pages_write(k, v, slots, *pools)
    lengths, off = torch.tensor([n], dtype=torch.int32, device=DEV), to_dev(offsets([n]))
    q = torch.randn((1, Hkv, d), device=DEV).bfloat16()
    got = dlrm_seq_attn_paged_decode(q, *pools, table, lengths, page, max_kv_len=n)
    want = dlrm_seq_attn_decode(q, k, v, off[:-1], off[1:], max_kv_len=n)
    q2, qo = torch.randn((70, Hkv, d), device=DEV).bfloat16(), to_dev(offsets([70]))
    assert torch.equal(got, want)
    check_several(dlrm_seq_attn_paged_fwd(q2, *pools, qo, table, lengths, page), dlrm_seq_attn_fwd(q2, k, v, qo, off),
                  lambda x: dlrm_seq_attn_fwd(q2, k, x, qo, off), v)


def test_captured_and_replayed():
    """A serving step (tables, rows to their slots, attention), captured and replayed: the histories grow from replay to
    replay as they do eagerly."""
    B, page, Hq, Hkv, d = 5, 8, 4, 2, 64
    i32 = dict(dtype=torch.int32, device=DEV)

    def fresh():
        g = torch.Generator(device=DEV).manual_seed(3)
        return dict(table=torch.full((B, 6), -1, **i32), lengths=torch.zeros(B, **i32), free=torch.arange(40, **i32), count=torch.tensor([40], **i32),
                    pools=[torch.zeros((320, Hkv, d), dtype=torch.bfloat16, device=DEV) for _ in range(2)],
                    x=torch.randn((B, Hq + 2 * Hkv, d), generator=g, device=DEV).bfloat16(), off=torch.arange(B + 1, device=DEV))

    def step(s):
        slots, refused = dlrm_seq_pages_update(s["table"], s["lengths"], s["free"], s["count"], page, s["off"], B, s["lengths"] >= 40)
        q, k, v = s["x"][:, :Hq], s["x"][:, Hq:Hq + Hkv], s["x"][:, Hq + Hkv:]
        dlrm_seq_pages_write(k, v, slots, *s["pools"])
        o = dlrm_seq_attn_paged_decode(q, *s["pools"], s["table"], s["lengths"], page, max_kv_len=48, window=30, sinks=2)
        return o, dlrm_seq_attn_paged_fwd(q, *s["pools"], s["off"], s["table"], s["lengths"], page), slots, refused

    say("[pages] captured")
    eager, mine = fresh(), fresh()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step(fresh())
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(mine)
    for turn in range(90):
        x = torch.randn(mine["x"].shape, device=DEV).bfloat16()
        mine["x"].copy_(x), eager["x"].copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        want = step(eager)
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
        for name in ("table", "lengths", "free", "count"):
            assert torch.equal(mine[name], eager[name]), turn
    assert (mine["lengths"] == 90 - 40 * 2).all()


def test_two_streams_at_once():
    """Two pools' visits under way on two streams."""
    rng = rng_of("pages-streams")
    say("[pages] two streams")
    streams, jobs = [torch.cuda.Stream() for _ in range(2)], []
    for B in (1800, 300):
        table, lengths, free, top = new_pool(B, 8, 4 * B)
        off = offsets(rng.integers(0, 40, B))
        dev = [to_dev(table), to_dev(lengths), to_dev(free), torch.tensor([top], dtype=torch.int32, device=DEV)]
        jobs.append((oracle.update(table, lengths, free, top, 8, off, int(off[-1])), dev, to_dev(off), int(off[-1])))
    torch.cuda.synchronize()
    got = []
    for s, (_, dev, off, n) in zip(streams, jobs):
        with torch.cuda.stream(s):
            got.append(dlrm_seq_pages_update(*dev, 8, off, n))
    torch.cuda.synchronize()
    for (want, dev, _, _), (slots, refused) in zip(jobs, got):
        assert np.array_equal(slots.cpu().numpy(), want[4]) and np.array_equal(dev[0].cpu().numpy(), want[0]) and int(refused) == want[5]
