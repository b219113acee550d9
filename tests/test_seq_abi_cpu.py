"""The user-history calls on a machine without a GPU: invalid arguments are rejected on the host before
anything touches a device (fake device pointers are never dereferenced), and the wrappers refuse CPU
tensors and wrong shapes."""
import ctypes

import pytest
import torch

from recommendation_model_sparse_amd import binding
from recommendation_model_sparse_amd import (dlrm_add_rmsnorm_bwd, dlrm_add_rmsnorm_fwd, dlrm_dropout, dlrm_seq_attn_decode,
                                             dlrm_seq_attn_fwd, dlrm_seq_bucket_bounds)

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -5
FAKE = 0x7F0000000000


@pytest.fixture(scope="module")
def L():
    return binding.lib()


class SeqAttn(ctypes.Structure):
    """dlrm_seq_attn as the header declares it."""
    _fields_ = [("B", ctypes.c_int64), ("Nq", ctypes.c_int64), ("Nkv", ctypes.c_int64), ("Hq", ctypes.c_int32),
                ("Hkv", ctypes.c_int32), ("d", ctypes.c_int32), ("index_type", ctypes.c_int32),
                ("q_offsets", ctypes.c_void_p), ("kv_begin", ctypes.c_void_p), ("kv_end", ctypes.c_void_p),
                ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("q_row", ctypes.c_int64),
                ("q_head", ctypes.c_int64), ("k_row", ctypes.c_int64), ("k_head", ctypes.c_int64),
                ("v_row", ctypes.c_int64), ("v_head", ctypes.c_int64), ("window", ctypes.c_int32),
                ("sinks", ctypes.c_int32), ("scale", ctypes.c_float), ("buckets", ctypes.c_int32),
                ("bias", ctypes.c_void_p), ("bounds", ctypes.c_void_p)]


def test_description_layout():
    assert ctypes.sizeof(SeqAttn) == binding._SEQ_ATTN.size


def attn(**over):
    keep = (ctypes.c_int32 * 4)(*over.pop("edges", [0, 1, 2, 3]))
    f = dict(B=2, Nq=10, Nkv=10, Hq=4, Hkv=2, d=32, index_type=0, q_offsets=FAKE, kv_begin=FAKE, kv_end=FAKE + 8, q=FAKE,
             k=FAKE, v=FAKE, q_row=128, q_head=32, k_row=64, k_head=32, v_row=64, v_head=32, window=0, sinks=0, scale=1.0,
             buckets=4, bias=FAKE, bounds=ctypes.addressof(keep))
    f.update(over)
    a = SeqAttn(**f)
    a.keep = keep
    return a


BAD = [(dict(B=-1), INVALID), (dict(Nq=-1), INVALID), (dict(Hq=3), INVALID), (dict(Hkv=0), INVALID), (dict(d=0), INVALID),
       (dict(d=12, q_row=48, q_head=16), UNSUPPORTED), (dict(d=136, q_row=544, q_head=136, k_row=272, k_head=136, v_row=272,
                                                             v_head=136), UNSUPPORTED),
       (dict(index_type=2), INVALID), (dict(kv_begin=None), INVALID), (dict(kv_end=FAKE + 4), INVALID), (dict(q=None), INVALID),
       (dict(k=FAKE + 8), INVALID), (dict(v=None), INVALID), (dict(q_row=31), INVALID), (dict(q_head=36), INVALID),
       (dict(k_row=24), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(scale=float("nan")), INVALID),
       (dict(bounds=None), INVALID), (dict(buckets=0), INVALID), (dict(buckets=129), UNSUPPORTED),
       (dict(edges=[1, 2, 3, 4]), INVALID), (dict(edges=[0, 2, 2, 4]), INVALID), (dict(bias=FAKE + 2), INVALID),
       (dict(B=1 << 24), UNSUPPORTED), (dict(Nkv=1 << 31), UNSUPPORTED), (dict(k_row=1 << 24), UNSUPPORTED), (dict(Hq=8192), UNSUPPORTED)]


@pytest.mark.parametrize("over,want", BAD)
def test_attention_rejects(L, over, want):
    a = attn(**over)
    assert L.dlrm_seq_attn_fwd(ctypes.byref(a), FAKE, None, None, None) == want
    assert L.dlrm_seq_attn_bwd(ctypes.byref(a), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 30, None) == want
    if "B" not in over:
        a.Nq = a.B
    if "Nq" not in over:
        assert L.dlrm_seq_attn_decode(ctypes.byref(a), 100, FAKE, FAKE, 1 << 30, None) == want


def test_attention_outputs_rejected(L):
    a = attn()
    fwd, bwd, dec = L.dlrm_seq_attn_fwd, L.dlrm_seq_attn_bwd, L.dlrm_seq_attn_decode
    assert fwd(None, FAKE, None, None, None) == INVALID
    assert fwd(ctypes.byref(a), None, None, None, None) == INVALID
    assert fwd(ctypes.byref(a), FAKE + 2, None, None, None) == INVALID
    assert fwd(ctypes.byref(a), FAKE, FAKE, None, None) == INVALID
    assert fwd(ctypes.byref(attn(q_offsets=None)), FAKE, None, None, None) == INVALID
    good = [FAKE] * 8 + [FAKE, 1 << 30]
    for i in (0, 1, 2, 3, 4, 5, 6, 7):
        args = list(good)
        args[i] = None
        assert bwd(ctypes.byref(a), *args, None) == INVALID, i
    assert bwd(ctypes.byref(a), *good[:8], None, 1 << 30, None) == WORKSPACE
    assert bwd(ctypes.byref(a), *good[:8], FAKE + 16, 1 << 30, None) == WORKSPACE
    need = L.dlrm_seq_attn_bwd_workspace_size(ctypes.byref(a))
    assert need > 0 and bwd(ctypes.byref(a), *good[:8], FAKE, need - 1, None) == WORKSPACE
    assert bwd(ctypes.byref(attn(kv_end=FAKE + 256)), *good, None) == INVALID  # regions, not offsets
    assert bwd(ctypes.byref(attn(bias=None)), *good, None) == INVALID          # dbias without a bias
    one = attn(Nq=2)
    assert dec(ctypes.byref(a), 100, FAKE, FAKE, 1 << 30, None) == INVALID     # a query a sequence
    assert dec(ctypes.byref(one), -1, FAKE, FAKE, 1 << 30, None) == INVALID
    assert dec(ctypes.byref(one), 100, None, FAKE, 1 << 30, None) == INVALID
    assert dec(ctypes.byref(one), 1 << 20, FAKE, None, 0, None) == WORKSPACE
    assert fwd(ctypes.byref(attn(B=0, Nq=0, Nkv=0)), FAKE, None, None, None) == OK


def test_workspace_sizes(L):
    assert L.dlrm_seq_attn_bwd_workspace_size(ctypes.byref(attn(B=-1))) == 0
    assert L.dlrm_seq_attn_bwd_workspace_size(ctypes.byref(attn(Nq=1000))) >= 1000 * 4 * 4
    assert L.dlrm_seq_attn_tiles(-1, 5) == 0 and L.dlrm_seq_attn_tiles(3, 64) >= 3
    assert L.dlrm_seq_attn_decode_workspace_size(1, 3, 2, 32, 0, 0, 10) == 0
    assert L.dlrm_seq_attn_decode_workspace_size(1, 4, 2, 32, 0, 0, 1 << 20) > L.dlrm_seq_attn_decode_workspace_size(1, 4, 2, 32, 100, 4, 1 << 20)
    assert L.dlrm_add_rmsnorm_bwd_workspace_size(5, 0) == 0 and L.dlrm_add_rmsnorm_bwd_workspace_size(5, 4097) == 0
    assert L.dlrm_add_rmsnorm_bwd_workspace_size(5, 16384) > 16384 * 4


def test_norm_and_dropout_reject(L):
    spec = lambda p=0.1, dev=None: ctypes.byref(binding._Dropout(p, 1, 0, dev))  # noqa: E731
    drop = L.dlrm_dropout
    for args in ((FAKE, 2, 8, spec(), FAKE), (FAKE, 0, -1, spec(), FAKE), (FAKE, 0, 8, None, FAKE), (FAKE, 0, 8, spec(1.5), FAKE),
                 (FAKE, 0, 8, spec(float("nan")), FAKE), (FAKE, 0, 8, spec(0.1, FAKE + 4), FAKE), (None, 0, 8, spec(), FAKE),
                 (FAKE + 4, 0, 8, spec(), FAKE), (FAKE, 0, 8, spec(), FAKE + 8)):
        assert drop(*args, None) == INVALID
    assert drop(None, 0, 0, spec(), None, None) == OK
    good = dict(x=FAKE, xt=0, res=FAKE, rt=0, w=FAKE, eps=1e-6, drop=None, M=4, D=16, s=FAKE, y=FAKE, yt=1, sc=None, rstd=FAKE)
    for over, want in ((dict(xt=2), INVALID), (dict(rt=3), INVALID), (dict(yt=3), INVALID), (dict(eps=-1.0), INVALID),
                       (dict(eps=float("nan")), INVALID), (dict(M=-1), INVALID), (dict(D=0), INVALID), (dict(D=16392), UNSUPPORTED),
                       (dict(D=4097), UNSUPPORTED), (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=FAKE + 8), INVALID),
                       (dict(yt=2), INVALID), (dict(drop=spec(-0.5)), INVALID), (dict(M=0, x=None, y=None), OK)):
        assert L.dlrm_add_rmsnorm_fwd(*{**good, **over}.values(), None) == want, over
    good = dict(dy=FAKE, gt=0, ds=None, s=FAKE, rt=0, w=FAKE, rstd=FAKE, drop=None, M=4, D=16, dx=FAKE, xt=0, dres=None, dw=FAKE,
                ws=FAKE, n=1 << 30)
    for over, want in ((dict(gt=2), INVALID), (dict(xt=2), INVALID), (dict(dw=None), INVALID), (dict(dx=None), INVALID),
                       (dict(rstd=None), INVALID), (dict(ds=FAKE + 4), INVALID), (dict(D=4097), UNSUPPORTED),
                       (dict(ws=None), WORKSPACE), (dict(n=16), WORKSPACE)):
        assert L.dlrm_add_rmsnorm_bwd(*{**good, **over}.values(), None) == want, over


def test_wrappers_refuse_cpu_tensors():
    q = torch.zeros((6, 2, 32), dtype=torch.bfloat16)
    off = torch.tensor([0, 6])
    x, w = torch.zeros((4, 16)), torch.ones(16)
    for call in (lambda: dlrm_seq_attn_fwd(q, q, q, off), lambda: dlrm_seq_attn_decode(q[:1], q, q, off[:1], off[1:]),
                 lambda: dlrm_dropout(x, 0.1, 1), lambda: dlrm_add_rmsnorm_fwd(x, x, w),
                 lambda: dlrm_add_rmsnorm_bwd(x, x, x, w, torch.ones(4))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for bad in ((0, 5), (129, 5)):
        with pytest.raises(ValueError):
            dlrm_seq_bucket_bounds(*bad)


@pytest.mark.parametrize("d,ok,over", [(32, (1 << 31) - 64 * 64, (1 << 31) - 1), (128, (1 << 30) - 64 * 64, 1 << 30)])
def test_attention_past_one_launch_rejected(L, d, ok, over):
    """Tiles by threads reach 2^32 work-items; the sizes just below pass this check and fail a later one."""
    heads = dict(d=d, q_row=4 * d, q_head=d, k_row=2 * d, k_head=d, v_row=2 * d, v_head=d)
    for n, want in ((ok, INVALID), (over, UNSUPPORTED)):
        a = attn(Nq=n, q=None, **heads)
        assert L.dlrm_seq_attn_fwd(ctypes.byref(a), FAKE, None, None, None) == want
        a = attn(Nkv=n, k=None, **heads)
        assert L.dlrm_seq_attn_bwd(ctypes.byref(a), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 30, None) == want
    a = attn(B=1 << 23, Nq=1 << 23, **heads)
    assert L.dlrm_seq_attn_decode(ctypes.byref(a), 100, FAKE, FAKE, 1 << 62, None) == UNSUPPORTED


@pytest.mark.parametrize("bias", [None, FAKE])
def test_backward_without_queries_takes_no_tiles(L, bias):
    """The forward of no queries writes no tiles and takes NULL; the backward then has nothing to look up:
    without keys and a bias it launches nothing, and with them only what does not read tiles."""
    a = attn(Nq=0, Nkv=0, q=None, k=None, v=None, bias=bias, sinks=3, window=5)
    assert L.dlrm_seq_attn_fwd(ctypes.byref(a), None, None, None, None) == OK
    need = L.dlrm_seq_attn_bwd_workspace_size(ctypes.byref(a))
    assert need == L.dlrm_seq_attn_bwd_workspace_size(ctypes.byref(attn(B=0, Nq=0, Nkv=0, bias=bias)))  # no slots of queries
    if bias is None:
        assert L.dlrm_seq_attn_bwd(ctypes.byref(a), *[None] * 8, FAKE, need, None) == OK


def test_decode_sizes_past_one_launch(L):
    """Refused sizes have a workspace of 0, as the header says, not of what their product wraps to; they are
    refused whatever the workspace."""
    size = L.dlrm_seq_attn_decode_workspace_size
    assert size((1 << 24) - 1, 1, 1, 8, 0, 0, 1 << 20) > 0
    for B, Hq, Hkv in (((1 << 24) - 1, 4096, 4096), (1 << 20, 256, 16), (1 << 20, 17 * 8, 8)):
        assert size(B, Hq, Hkv, 8, 0, 0, 1 << 30) == 0
        a = attn(B=B, Nq=B, Hq=Hq, Hkv=Hkv, d=8, q_row=Hq * 8, q_head=8, k_row=Hkv * 8, k_head=8, v_row=Hkv * 8, v_head=8)
        assert L.dlrm_seq_attn_decode(ctypes.byref(a), 1 << 30, FAKE, None, 0, None) == UNSUPPORTED


def test_strides_of_one_row_are_of_no_account():
    far = torch.zeros((4, 65536, 64), dtype=torch.bfloat16)
    assert binding._head_rows(far.transpose(0, 1)[:1], "q") == (1, 4, 64, 64, 65536 * 64)
    assert binding._head_rows(far[:1].transpose(0, 1)[:1], "q") == (1, 1, 64, 64, 64)
    assert binding._head_rows(far.transpose(0, 1)[:2], "q") == (2, 4, 64, 64, 65536 * 64)
