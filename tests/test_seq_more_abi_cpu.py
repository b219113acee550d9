"""The calls of paged histories and of linear attention with a decay on a machine without a GPU: invalid arguments are
refused on the host before anything touches a device (fake device pointers are never dereferenced), and the wrappers
refuse CPU tensors and wrong shapes."""
import ctypes

import pytest
import torch

from recommendation_model_sparse_amd import binding
from recommendation_model_sparse_amd import (dlrm_seq_attn_paged_decode, dlrm_seq_attn_paged_fwd, dlrm_seq_decay_bwd,
                                             dlrm_seq_decay_fwd, dlrm_seq_decay_step, dlrm_seq_pages_update, dlrm_seq_pages_write)
from test_seq_abi_cpu import attn

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -5
FAKE = 0x7F0000000000
p, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


@pytest.fixture(scope="module")
def L():
    return binding.lib()


class Pages(ctypes.Structure):
    """dlrm_seq_pages as the header declares it."""
    _fields_ = [("B", i64), ("pages", i64), ("table_row", i64), ("width", i32), ("page", i32), ("table", p), ("lengths", p),
                ("free_list", p), ("free_count", p)]


class Decay(ctypes.Structure):
    """dlrm_seq_decay as the header declares it."""
    _fields_ = [("B", i64), ("N", i64), ("Hq", i32), ("Hkv", i32), ("d", i32), ("index_type", i32), ("offsets", p), ("max_len", i64),
                ("q", p), ("k", p), ("v", p), ("q_row", i64), ("q_head", i64), ("k_row", i64), ("k_head", i64), ("v_row", i64),
                ("v_head", i64), ("g", p), ("g_row", i64), ("scale", ctypes.c_float)]


def test_description_layouts():
    assert ctypes.sizeof(Pages) == binding._SEQ_PAGES.size and ctypes.sizeof(Decay) == binding._SEQ_DECAY.size


def pages(**over):
    f = dict(B=2, pages=10, table_row=4, width=4, page=16, table=FAKE, lengths=FAKE, free_list=FAKE, free_count=FAKE)
    return Pages(**dict(f, **over))


def decay(**over):
    f = dict(B=2, N=10, Hq=4, Hkv=2, d=32, index_type=0, offsets=FAKE, max_len=10, q=FAKE, k=FAKE, v=FAKE, q_row=128, q_head=32, k_row=64,
             k_head=32, v_row=64, v_head=32, g=FAKE, g_row=2, scale=1.0)
    return Decay(**dict(f, **over))


BAD_PAGES = [(dict(pages=0), INVALID), (dict(width=-1), INVALID), (dict(table_row=3), INVALID), (dict(page=4), UNSUPPORTED),
             (dict(page=24), UNSUPPORTED), (dict(page=8192), UNSUPPORTED), (dict(pages=1 << 27), UNSUPPORTED),
             (dict(width=1 << 26, table_row=1 << 26), UNSUPPORTED), (dict(table=0), INVALID), (dict(lengths=0), INVALID),
             (dict(lengths=FAKE + 2), INVALID), (dict(table=FAKE + 1), INVALID)]


@pytest.mark.parametrize("over,want", BAD_PAGES + [(dict(B=-1), INVALID), (dict(B=1 << 20), UNSUPPORTED), (dict(free_list=0), INVALID),
                                                   (dict(free_count=0), INVALID), (dict(free_count=FAKE + 1), INVALID)])
def test_update_refuses(L, over, want):
    assert L.dlrm_seq_pages_update(ctypes.byref(pages(**over)), FAKE, 0, 8, 0, FAKE, FAKE, FAKE, 1 << 20, None) == want


@pytest.mark.parametrize("args,want", [
    ((0, 0, 8, 0, FAKE, FAKE, FAKE, 1 << 20), INVALID), ((FAKE + 4, 0, 8, 0, FAKE, FAKE, FAKE, 1 << 20), INVALID),
    ((FAKE, 2, 8, 0, FAKE, FAKE, FAKE, 1 << 20), INVALID), ((FAKE, 0, -1, 0, FAKE, FAKE, FAKE, 1 << 20), INVALID),
    ((FAKE, 0, 1 << 31, 0, FAKE, FAKE, FAKE, 1 << 20), UNSUPPORTED), ((FAKE, 0, 8, 0, 0, FAKE, FAKE, 1 << 20), INVALID),
    ((FAKE, 0, 8, 0, FAKE + 4, FAKE, FAKE, 1 << 20), INVALID), ((FAKE, 0, 8, 0, FAKE, 0, FAKE, 1 << 20), INVALID),
    ((FAKE, 0, 8, 0, FAKE, FAKE, 0, 1 << 20), WORKSPACE), ((FAKE, 0, 8, 0, FAKE, FAKE, FAKE + 8, 1 << 20), WORKSPACE),
    ((FAKE, 0, 8, 0, FAKE, FAKE, FAKE, 8), WORKSPACE)])
def test_update_refuses_arguments(L, args, want):
    assert L.dlrm_seq_pages_update(ctypes.byref(pages()), *args, None) == want


def test_update_workspace(L):
    assert L.dlrm_seq_pages_update_workspace_size(-1, 0) == 0 and L.dlrm_seq_pages_update_workspace_size(1 << 20, 0) == 0
    assert L.dlrm_seq_pages_update_workspace_size(1, 1 << 31) == 0 and L.dlrm_seq_pages_update_workspace_size(5000, 9) >= 4 * 5000
    assert L.dlrm_seq_pages_update(None, FAKE, 0, 8, 0, FAKE, FAKE, FAKE, 1 << 20, None) == INVALID


@pytest.mark.parametrize("over,want", [
    (dict(N=-1), INVALID), (dict(rows=-1), INVALID), (dict(H=0), INVALID), (dict(d=12), UNSUPPORTED), (dict(H=1 << 18), UNSUPPORTED),
    (dict(N=1 << 31), UNSUPPORTED), (dict(k_row=33), INVALID), (dict(v_pool_head=24), INVALID), (dict(k=0), INVALID), (dict(v=FAKE + 8), INVALID),
    (dict(k_pool=0), INVALID), (dict(slots=0), INVALID), (dict(slots=FAKE + 4), INVALID), (dict(N=0, k=0), OK), (dict(rows=0, k_pool=0), OK)])
def test_write_refuses(L, over, want):
    f = dict(k=FAKE, k_row=64, k_head=32, v=FAKE, v_row=64, v_head=32, N=5, H=2, d=32, slots=FAKE, k_pool=FAKE, k_pool_row=64, k_pool_head=32,
             v_pool=FAKE, v_pool_row=64, v_pool_head=32, rows=100)
    f.update(over)
    assert L.dlrm_seq_pages_write(*f.values(), None) == want


@pytest.mark.parametrize("over,want", BAD_PAGES + [(dict(B=3), INVALID), (dict(pages=11), INVALID)])
@pytest.mark.parametrize("call", ["fwd", "decode"])
def test_paged_attention_refuses_pages(L, call, over, want):
    a = attn(Nq=2 if call == "decode" else 10, Nkv=over.get("pages", 10) * over.get("page", 16) if want != INVALID else 160, kv_begin=0, kv_end=0)
    pg = pages(**over)
    if call == "fwd":
        assert L.dlrm_seq_attn_paged_fwd(ctypes.byref(a), ctypes.byref(pg), FAKE, None) == want
    else:
        assert L.dlrm_seq_attn_paged_decode(ctypes.byref(a), ctypes.byref(pg), 40, FAKE, FAKE, 1 << 20, None) == want


def test_paged_attention_refuses_the_rest(L):
    pg = pages()
    for over in (dict(Nkv=159), dict(Hq=3), dict(q_row=7), dict(window=-1)):
        a = attn(**dict(dict(Nkv=160, kv_begin=0, kv_end=0), **over))
        assert L.dlrm_seq_attn_paged_fwd(ctypes.byref(a), ctypes.byref(pg), FAKE, None) == INVALID
    a = attn(Nkv=160, q_offsets=0)
    assert L.dlrm_seq_attn_paged_fwd(ctypes.byref(a), ctypes.byref(pg), FAKE, None) == INVALID
    a = attn(Nkv=160)
    assert L.dlrm_seq_attn_paged_fwd(ctypes.byref(a), None, FAKE, None) == INVALID
    assert L.dlrm_seq_attn_paged_fwd(ctypes.byref(a), ctypes.byref(pg), 0, None) == INVALID
    assert L.dlrm_seq_attn_paged_decode(ctypes.byref(a), ctypes.byref(pg), 40, FAKE, FAKE, 1 << 20, None) == INVALID  # Nq != B
    a = attn(Nq=2, Nkv=160)
    assert L.dlrm_seq_attn_paged_decode(ctypes.byref(a), ctypes.byref(pg), -1, FAKE, FAKE, 1 << 20, None) == INVALID
    assert L.dlrm_seq_attn_paged_decode(ctypes.byref(a), ctypes.byref(pg), 1 << 16, FAKE, 0, 0, None) == WORKSPACE


BAD_DECAY = [(dict(B=-1), INVALID), (dict(N=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=3), INVALID), (dict(d=0), INVALID), (dict(d=12), UNSUPPORTED),
             (dict(d=136, q_row=1088, q_head=136, k_row=272, k_head=136, v_row=272, v_head=136), UNSUPPORTED), (dict(Hq=8192), UNSUPPORTED),
             (dict(index_type=2), INVALID), (dict(B=1 << 24), UNSUPPORTED), (dict(N=1 << 31), UNSUPPORTED), (dict(max_len=-1), INVALID),
             (dict(q=0), INVALID), (dict(k=FAKE + 8), INVALID), (dict(g=0), INVALID), (dict(g=FAKE + 2), INVALID), (dict(g_row=1), INVALID),
             (dict(g_row=-2), INVALID), (dict(q_row=129), INVALID), (dict(v_head=24), INVALID), (dict(k_row=1 << 24), UNSUPPORTED),
             (dict(g_row=1 << 24), UNSUPPORTED), (dict(scale=float("nan")), INVALID)]
BAD_OFFSETS = [(dict(offsets=0), INVALID), (dict(offsets=FAKE + 4), INVALID), (dict(N=(1 << 29) + 64), UNSUPPORTED),
               (dict(N=1 << 28, Hq=1, Hkv=1, d=128, q_row=128, q_head=128, k_row=128, k_head=128, v_row=128, v_head=128), UNSUPPORTED)]


@pytest.mark.parametrize("over,want", BAD_DECAY + BAD_OFFSETS)
def test_decay_refuses(L, over, want):
    a = decay(**over)
    assert L.dlrm_seq_decay_fwd(ctypes.byref(a), None, None, FAKE, FAKE, 1 << 40, None) == want
    assert L.dlrm_seq_decay_bwd(ctypes.byref(a), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 40, None) == want
    assert L.dlrm_seq_decay_fwd_workspace_size(ctypes.byref(a)) == 0 and L.dlrm_seq_decay_bwd_workspace_size(ctypes.byref(a)) == 0


@pytest.mark.parametrize("over,want", BAD_DECAY + [(dict(), INVALID), (dict(B=10, Hq=1 << 12, Hkv=1 << 12), INVALID)])
def test_step_refuses(L, over, want):
    """(N != B too.)"""
    assert L.dlrm_seq_decay_step(ctypes.byref(decay(**over)), FAKE, FAKE, None) == want


def test_decay_refuses_outputs(L):
    a = decay()
    need = L.dlrm_seq_decay_bwd_workspace_size(ctypes.byref(a))
    good = [FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 40]
    for i in range(4):
        for bad in (0, FAKE + 8):
            assert L.dlrm_seq_decay_bwd(ctypes.byref(a), *good[:i], bad, *good[i + 1:], None) == INVALID
    assert L.dlrm_seq_decay_bwd(ctypes.byref(a), *good[:4], FAKE + 2, *good[5:], None) == INVALID
    for ws, size in ((0, 1 << 40), (FAKE + 8, 1 << 40), (FAKE, need - 1)):
        assert L.dlrm_seq_decay_bwd(ctypes.byref(a), *good[:5], ws, size, None) == WORKSPACE
    assert L.dlrm_seq_decay_fwd(ctypes.byref(a), FAKE + 4, None, FAKE, FAKE, 1 << 40, None) == INVALID
    assert L.dlrm_seq_decay_fwd(ctypes.byref(a), None, FAKE + 4, FAKE, FAKE, 1 << 40, None) == INVALID
    assert L.dlrm_seq_decay_fwd(ctypes.byref(a), None, None, 0, FAKE, 1 << 40, None) == INVALID
    long = decay(B=1, N=100000, max_len=100000)
    assert L.dlrm_seq_decay_fwd_workspace_size(ctypes.byref(long)) > 1 << 20  # it is cut into runs
    assert L.dlrm_seq_decay_fwd(ctypes.byref(long), None, None, FAKE, 0, 0, None) == WORKSPACE
    one = decay(N=2)
    assert L.dlrm_seq_decay_step(ctypes.byref(one), 0, FAKE, None) == INVALID
    assert L.dlrm_seq_decay_step(ctypes.byref(one), FAKE + 4, FAKE, None) == INVALID
    assert L.dlrm_seq_decay_step(ctypes.byref(one), FAKE, 0, None) == INVALID
    many = decay(B=1 << 14, N=1 << 14, Hq=1 << 10, Hkv=1 << 10, g_row=1 << 10)
    assert L.dlrm_seq_decay_step(ctypes.byref(many), FAKE, FAKE, None) == UNSUPPORTED


@pytest.mark.parametrize("B,each_len", [(65536, 64), (200000, 8)])
@pytest.mark.parametrize("each", [True, False])
def test_backward_workspace_of_many_short_sequences(L, B, each_len, each):
    """States at marks (64 d d bytes for 512 events of a key head, or 128 with one decay a head) go by the rows, not by the
    sequences; beside them two floats an event and what goes by the sequences, an order and a sum each."""
    N, H, d = B * each_len, 4, 128
    a = decay(B=B, N=N, Hq=H, Hkv=H, d=d, max_len=each_len, q_row=H * d, q_head=d, k_row=H * d, k_head=d, v_row=H * d, v_head=d, g_row=H if each else 0)
    size = L.dlrm_seq_decay_bwd_workspace_size(ctypes.byref(a))
    assert 0 < size <= 4 * d * d * H * (N // (512 if each else 128)) + 8 * N * H + 12 * B * H + 4096


@pytest.mark.parametrize("B,each_len,H,d", [(20000, 60, 4, 128), (65536, 64, 4, 128), (200000, 8, 4, 128), (1024, 256, 4, 128), (4096, 30, 16, 64), (3000, 100, 32, 96)])
def test_workspace_where_the_longest_is_not_known(L, B, each_len, H, d):
    """Told that one of many sequences may be all rows, a call keeps its runs' states, each direction's, to 256 MB or to the rows of
    q, k, v and o (with a float a state beside); the backward's marks, terms, order and sums come on top."""
    N = B * each_len
    rows = max(1 << 28, 8 * N * H * d)
    for g_row in (0, H):
        a = decay(B=B, N=N, Hq=H, Hkv=H, d=d, max_len=N, q_row=H * d, q_head=d, k_row=H * d, k_head=d, v_row=H * d, v_head=d, g_row=g_row)
        states = rows + rows // (d * d) + 4096
        assert 0 < L.dlrm_seq_decay_fwd_workspace_size(ctypes.byref(a)) <= states
        marks = 4 * 128 * 128 * H * (N // 64)  # one a chunk at most
        assert 0 < L.dlrm_seq_decay_bwd_workspace_size(ctypes.byref(a)) <= 2 * states + marks + 8 * N * H + 8 * H * (N // 64 + B) + 4 * B + 4096


def test_nothing_to_do(L):
    assert L.dlrm_seq_decay_fwd(ctypes.byref(decay(B=0, N=0)), None, None, None, None, 0, None) == OK
    assert L.dlrm_seq_decay_step(ctypes.byref(decay(B=0, N=0)), None, None, None) == OK
    a = attn(Nq=0, Nkv=160)
    assert L.dlrm_seq_attn_paged_fwd(ctypes.byref(a), ctypes.byref(pages()), None, None) == OK


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_wrappers_refuse():
    i = lambda *x: torch.zeros(x, dtype=torch.int32)  # noqa: E731
    q, k, pool, off = bf(5, 4, 32), bf(5, 2, 32), bf(160, 2, 32), torch.zeros(3, dtype=torch.int64)
    table, lengths, free, one, g = i(2, 4), i(2), i(10), i(1), torch.zeros(5, 2)
    every = [
        (dlrm_seq_pages_update, (table, lengths, free, one, 16, off, 5)),                          # on the CPU
        (dlrm_seq_pages_update, (table.long(), lengths, free, one, 16, off, 5)),
        (dlrm_seq_pages_update, (table, i(3), free, one, 16, off, 5)),
        (dlrm_seq_pages_update, (table, lengths, free, i(2), 16, off, 5)),
        (dlrm_seq_pages_update, (table, lengths, free, one, 12, off, 5)),
        (dlrm_seq_pages_update, (table, lengths, free, one, 16, off[:2], 5)),
        (dlrm_seq_pages_update, (table, lengths, free, one, 16, off, -1)),
        (dlrm_seq_pages_update, (table, lengths, free, one, 16, off, 5, torch.zeros(3, dtype=torch.bool))),
        (dlrm_seq_pages_update, (i(1, 4).expand(2, 4), lengths, free, one, 16, off, 5)),           # one row for two users
        (dlrm_seq_pages_write, (k, k, torch.zeros(5, dtype=torch.int64), pool, pool)),
        (dlrm_seq_pages_write, (k, k[:4], torch.zeros(5, dtype=torch.int64), pool, pool)),
        (dlrm_seq_pages_write, (k, k, torch.zeros(5, dtype=torch.int32), pool, pool)),
        (dlrm_seq_pages_write, (k, k, torch.zeros(5, dtype=torch.int64), pool, pool[:100])),
        (dlrm_seq_attn_paged_fwd, (q, pool, pool, off, table, lengths, 16)),
        (dlrm_seq_attn_paged_fwd, (q, pool, pool, off, table, i(3), 16)),
        (dlrm_seq_attn_paged_fwd, (q, pool[:150], pool[:150], off, table, lengths, 16)),
        (dlrm_seq_attn_paged_decode, (q, pool, pool, table, lengths, 16)),
        (dlrm_seq_attn_paged_decode, (q[:2], pool, pool, table, lengths, 16)),
        (dlrm_seq_decay_fwd, (q, k, k, g, off)),
        (dlrm_seq_decay_fwd, (q, k, k, g[:, :1], off)),
        (dlrm_seq_decay_fwd, (q, k, k, g.double(), off)),
        (dlrm_seq_decay_fwd, (q, k, k, g[:1].expand(5, 2), off)),                                  # one row for all events
        (dlrm_seq_decay_fwd, (q, k[:4], k, g, off)),
        (dlrm_seq_decay_fwd, (bf(5, 3, 32), k, k, g, off)),
        (dlrm_seq_decay_bwd, (q, q, k, k, g, off)),
        (dlrm_seq_decay_bwd, (q[:4], q, k, k, g, off)),
        (dlrm_seq_decay_step, (q, k, k, g, torch.zeros(5, 2, 32, 32))),
        (dlrm_seq_decay_step, (q, k, k, g, torch.zeros(5, 2, 32, 16))),
    ]
    for call, args in every:
        with pytest.raises((ValueError, TypeError)):
            call(*args)
    with pytest.raises(ValueError):
        dlrm_seq_decay_fwd(q, k, k, g, off, max_len=-1)
    with pytest.raises(ValueError):
        dlrm_seq_attn_paged_decode(q[:2], pool, pool, table, lengths, 16, max_kv_len=-1)
