"""Python binding of ``libdlrm_sparse.so`` (ctypes; argument marshalling only).

Each function has the name of the C entry point it calls and passes device
pointers of torch tensors plus the current HIP stream.  Every step of the
computation runs in the library's HIP kernels; there is no fallback: if the
library is not built, loading it raises.
"""
from __future__ import annotations

import array
import ctypes
import operator
import os
import struct
from typing import List, Optional, Sequence, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdlrm_sparse.so")

DLRM_F32, DLRM_BF16 = 0, 1
DLRM_INDEX_I64, DLRM_INDEX_I32 = 0, 1
DLRM_OPT_ADAGRAD, DLRM_OPT_SGD = 0, 1
DLRM_ACT_NONE, DLRM_ACT_RELU = 0, 1
DLRM_FLAG_CHECK_INDICES = 1
DLRM_GRAM_AUTO, DLRM_GRAM_MFMA, DLRM_GRAM_VALU = 0, 1, 2
DLRM_F8_E4M3 = 2
DLRM_SEQ_MAX_BUCKETS = 128

_lib = None


class DlrmError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


# dlrm_seq_attn (dlrm_seq.h), field by field
_SEQ_ATTN = struct.Struct("@3q4i6Q6q2ifi2Q")
# dlrm_seq_pages (dlrm_seq_pages.h) and dlrm_seq_decay (dlrm_seq_decay.h)
_SEQ_PAGES = struct.Struct("@3q2i4Q")
_SEQ_DECAY = struct.Struct("@2q4iQq3Q6qQqf4x")


class _Dropout(ctypes.Structure):
    """dlrm_dropout_spec (dlrm_seq.h)."""
    _fields_ = [("p", ctypes.c_float), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
                ("offset_dev", ctypes.c_void_p)]


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m recommendation_model_sparse_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        p, i32, i64, u32, u64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                                          ctypes.c_uint32, ctypes.c_uint64, ctypes.c_float,
                                          ctypes.c_size_t)
        L.emb_bag_fwd.argtypes = [p, p, i32, i32, i32, p, p, p, i64, i64, p, u32, p]
        L.emb_bag_fwd_ex.argtypes = [p, p, i32, i32, i32, p, p, i32, p, i64, i64, p, i32, u32, p]
        L.emb_bag_bwd_update.argtypes = [p, p, p, i32, i32, i32, p, p, i32, p, i64, i64, p, i32, f32, f32,
                                         p, sz, p, p, p, p, u32, p]
        L.emb_bag_bwd_plan.argtypes = [p, i32, i32, p, p, i32, p, i64, i64, p, sz, p, p, p, p, u32, p]
        L.emb_bag_bwd_apply.argtypes = [p, p, p, i32, i32, i32, i64, i64, i32, p, i32, f32, f32, p, sz, p, p]
        L.dlrm_interact_fwd.argtypes = [p, p, i64, i32, i32, p, p]
        L.dlrm_interact_fwd_ex.argtypes = [p, p, i64, i32, i32, p, i32, p]
        L.dlrm_interact_fwd_ex.restype = ctypes.c_int
        L.emb_bag_interact_fwd.argtypes = [p, p, i32, i32, i32, p, p, p, i64, i64, p, p, u32, p]
        L.dlrm_interact_bwd.argtypes = [p, p, p, i64, i32, i32, p, p, p]
        L.emb_bag_bwd_workspace_size.argtypes = [i32, p, i32, i64, i64]
        L.emb_bag_bwd_workspace_size.restype = sz
        L.emb_bag_bwd_adagrad.argtypes = [p, p, p, i32, i32, i32, p, p, p, i64, i64, p, f32, f32,
                                          p, sz, p, p, p, p, u32, p]
        L.dlrm_linear_workspace_size.argtypes = [i64, i32, i32]
        L.dlrm_linear_workspace_size.restype = sz
        L.dlrm_bce_head_workspace_size.argtypes = [i64, i32]
        L.dlrm_bce_head_workspace_size.restype = sz
        L.dlrm_linear_fwd.argtypes = [p, p, p, i64, i32, i32, i32, p, i32, p, sz, p]
        L.dlrm_linear_bwd.argtypes = [p, p, i32, i32, p, p, i64, i32, i32, p, p, p, p, p, sz, p]
        L.dlrm_bce_head.argtypes = [p, p, p, p, i64, i32, p, p, p, p, p, p, sz, p]
        L.dlrm_sgd_dense.argtypes = [p, p, p, i64, f32, p]
        L.dlrm_sgd_dense_multi.argtypes = [i32, p, p, p, p, f32, p]
        L.dlrm_cast_rows.argtypes = [p, i32, i64, i64, i32, p, i32, i32, p]
        for f in (L.dlrm_linear_fwd, L.dlrm_linear_bwd, L.dlrm_bce_head, L.dlrm_sgd_dense, L.dlrm_cast_rows):
            f.restype = ctypes.c_int
        L.dlrm_seq_attn_fwd.argtypes = [p, p, p, p, p]
        L.dlrm_seq_attn_bwd_workspace_size.argtypes = [p]
        L.dlrm_seq_attn_tiles.argtypes = [i64, i64]
        L.dlrm_seq_attn_bwd.argtypes = [p, p, p, p, p, p, p, p, p, p, sz, p]
        L.dlrm_seq_attn_decode_workspace_size.argtypes = [i64, i32, i32, i32, i32, i32, i64]
        L.dlrm_seq_attn_decode.argtypes = [p, i64, p, p, sz, p]
        L.dlrm_dropout.argtypes = [p, i32, i64, p, p, p]
        L.dlrm_add_rmsnorm_fwd.argtypes = [p, i32, p, i32, p, f32, p, i64, i32, p, p, i32, p, p, p]
        L.dlrm_add_rmsnorm_bwd_workspace_size.argtypes = [i64, i32]
        L.dlrm_add_rmsnorm_bwd.argtypes = [p, i32, p, p, i32, p, p, p, i64, i32, p, i32, p, p, p, sz, p]
        for f in (L.dlrm_seq_attn_fwd, L.dlrm_seq_attn_bwd, L.dlrm_seq_attn_decode, L.dlrm_dropout, L.dlrm_add_rmsnorm_fwd,
                  L.dlrm_add_rmsnorm_bwd):
            f.restype = ctypes.c_int
        for f in (L.dlrm_seq_attn_bwd_workspace_size, L.dlrm_seq_attn_tiles, L.dlrm_seq_attn_decode_workspace_size,
                  L.dlrm_add_rmsnorm_bwd_workspace_size):
            f.restype = sz
        L.dlrm_seq_pages_update_workspace_size.argtypes = [i64, i64]
        L.dlrm_seq_pages_update.argtypes = [p, p, i32, i64, p, p, p, p, sz, p]
        L.dlrm_seq_pages_write.argtypes = [p, i64, i64, p, i64, i64, i64, i32, i32, p, p, i64, i64, p, i64, i64, i64, p]
        L.dlrm_seq_attn_paged_fwd.argtypes = [p, p, p, p]
        L.dlrm_seq_attn_paged_decode.argtypes = [p, p, i64, p, p, sz, p]
        L.dlrm_seq_decay_fwd_workspace_size.argtypes = [p]
        L.dlrm_seq_decay_fwd.argtypes = [p, p, p, p, p, sz, p]
        L.dlrm_seq_decay_bwd_workspace_size.argtypes = [p]
        L.dlrm_seq_decay_bwd.argtypes = [p, p, p, p, p, p, p, sz, p]
        L.dlrm_seq_decay_step.argtypes = [p, p, p, p]
        for f in (L.dlrm_seq_pages_update, L.dlrm_seq_pages_write, L.dlrm_seq_attn_paged_fwd, L.dlrm_seq_attn_paged_decode,
                  L.dlrm_seq_decay_fwd, L.dlrm_seq_decay_bwd, L.dlrm_seq_decay_step):
            f.restype = ctypes.c_int
        for f in (L.dlrm_seq_pages_update_workspace_size, L.dlrm_seq_decay_fwd_workspace_size, L.dlrm_seq_decay_bwd_workspace_size):
            f.restype = sz
        L.dlrm_status_string.argtypes = [ctypes.c_int]
        L.dlrm_status_string.restype = ctypes.c_char_p
        L.dlrm_synth_fill_table.argtypes = [p, i32, i64, i32, i32, u64, f32, p]
        L.emb_bag_bwd_update_noalloc.argtypes = [p, p, p, i32, i32, i32, p, p, i32, p, i64, i64, p, i32, f32,
                                                 f32, p, p, p, p, u32, p]
        L.emb_bag_bwd_update_noalloc.restype = ctypes.c_int
        L.emb_bag_bwd_noalloc_max_bytes.argtypes = []
        L.emb_bag_bwd_noalloc_max_bytes.restype = sz
        L.dlrm_probe_read.argtypes = [p, u64, p, u32, p]
        L.dlrm_probe_gather.argtypes = [p, i64, i32, p, i64, p, u32, p]
        L.dlrm_trace_enable.argtypes = [ctypes.c_int]
        L.dlrm_trace_read.argtypes = [i32, p, p, p, p]
        for f in (L.emb_bag_fwd, L.emb_bag_fwd_ex, L.emb_bag_bwd_update, L.dlrm_interact_fwd, L.emb_bag_interact_fwd, L.dlrm_interact_bwd, L.emb_bag_bwd_adagrad,
                  L.dlrm_synth_fill_table, L.dlrm_trace_enable, L.dlrm_trace_read, L.dlrm_probe_read,
                  L.dlrm_probe_gather):
            f.restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().dlrm_status_string(int(status)).decode()


dlrm_status_string = status_string


def _check(rc: int, what: str):
    if rc != 0:
        raise DlrmError(rc, what)


def _stream(dev: torch.device) -> ctypes.c_void_p:
    # the raw handle: torch.cuda.current_stream(dev) builds a Stream object around it, 2 us a call
    return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(dev.index))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# ---------------------------------------------------------------- argument checks
#
# The C entry points see plain pointers and sizes, so they cannot tell a CPU tensor, a wrong-sized
# output or a buffer of the wrong type from a good one; a kernel would read or write out of bounds.
# Every wrapper therefore checks each tensor (type, dtype, exact shape, contiguity, one CUDA device,
# workspace and output sizes) and raises ValueError before it calls the library.

def _need(t, name, dtype=None, shape=None, min_numel: Optional[int] = None) -> torch.Tensor:
    """`name` is a string, or a callable giving it (only called to word an error)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{_name(name)} must be a torch.Tensor, got {type(t).__name__}")
    if dtype is not None:
        ok = dtype if isinstance(dtype, tuple) else (dtype,)
        if t.dtype not in ok:
            raise ValueError(f"{_name(name)} must be {' or '.join(str(d) for d in ok)}, got {t.dtype}")
    if shape is not None and t.shape != shape:  # torch.Size compares with a tuple of ints
        raise ValueError(f"{_name(name)} must have shape {tuple(int(x) for x in shape)}, got {tuple(t.shape)}")
    if min_numel is not None and t.numel() < min_numel:
        raise ValueError(f"{_name(name)} must hold at least {min_numel} elements, got {t.numel()}")
    if not t.is_contiguous():
        raise ValueError(f"{_name(name)} must be contiguous")
    return t


def _is(t, name: str, dtype: torch.dtype, shape) -> torch.Tensor:
    """_need for one type and shape, at half its cost where the tensor is right."""
    if type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return t
    return _need(t, name, dtype, shape)


def _name(name) -> str:
    return name() if callable(name) else name


def _opt(t, name: str, dtype=None, shape=None, min_numel: Optional[int] = None):
    return None if t is None else _need(t, name, dtype, shape, min_numel)


def _device(*tensors) -> torch.device:
    """The one CUDA device every given tensor (None entries skipped) lives on."""
    ts = [t for t in tensors if t is not None]
    dev = ts[0].device
    if dev.type != "cuda":
        raise ValueError(f"tensors must be on a CUDA (HIP) device, got {dev}")
    for t in ts[1:]:
        if t.device != dev:
            raise ValueError(f"all tensors must be on {dev}, found one on {t.device}")
    return dev


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return DLRM_F32
    if t.dtype == torch.bfloat16:
        return DLRM_BF16
    raise ValueError(f"table dtype {t.dtype} is not float32 or bfloat16")


def _tables(tables: Sequence[torch.Tensor]):
    T = len(tables)
    if T == 0:
        raise ValueError("no tables")
    for t in tables:
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise ValueError("tables must be 2-D tensors [V_t, D]")
    D = tables[0].shape[1]
    code = _dtype_code(tables[0])
    for t in tables:
        if t.shape[1] != D or _dtype_code(t) != code or not t.is_contiguous():
            raise ValueError("tables must be contiguous [V_t, D] of one dtype")
    ptrs = (ctypes.c_void_p * T)(*[t.data_ptr() for t in tables])
    rows = (ctypes.c_int64 * T)(*[t.shape[0] for t in tables])
    return T, D, code, ptrs, rows


def _states(state, tables, required: bool):
    if state is None:
        if required:
            raise ValueError("row-wise Adagrad needs one state vector per table")
        return None
    if len(state) != len(tables):
        raise ValueError("one state vector per table")
    for i, (st, t) in enumerate(zip(state, tables)):
        _need(st, lambda: f"state[{i}]", torch.float32, (t.shape[0],))
    return (ctypes.c_void_p * len(state))(*[st.data_ptr() for st in state])


class TableSet:
    """Tables, and optionally their row-wise Adagrad states, checked once for repeated calls.

    Every wrapper that takes a list of tables also takes a TableSet, and then takes its states
    when its `state` argument is None or the set's own list.  The per-call checks then reduce to
    re-reading the tensors' data pointers and row counts; if one changed (a tensor replaced in the
    set's lists, re-allocated or resized), the set is checked again in full before the call.  It
    behaves as the sequence of its tables."""

    def __init__(self, tables: Sequence[torch.Tensor], states: Optional[Sequence[torch.Tensor]] = None):
        # the caller's own lists are kept (not copies), so passing that state list to a call is
        # recognized as the set's, and a tensor swapped into either list is seen by the next call
        self.tables = tables if isinstance(tables, list) else list(tables)
        self.states = None if states is None else (states if isinstance(states, list) else list(states))
        self._build()

    def _pointers(self):
        return ([t.data_ptr() for t in self.tables] + [t.shape[0] for t in self.tables] +
                [s.data_ptr() for s in (self.states or ())] + [s.shape[0] for s in (self.states or ())])

    def _build(self):
        self.T, self.D, self.code, self.ptrs, self.rows = _tables(self.tables)
        self.row_counts = [int(t.shape[0]) for t in self.tables]
        self.sptrs = None if self.states is None else _states(self.states, self.tables, True)
        self.device = _device(*self.tables, *(self.states or ()))
        self._key = self._pointers()

    def refresh(self) -> "TableSet":
        if self._pointers() != self._key:
            self._build()
        return self

    def __len__(self):
        return len(self.tables)

    def __iter__(self):
        return iter(self.tables)

    def __getitem__(self, i):
        return self.tables[i]


def _prepared(tables, state=None, need_state=False, with_state=False):
    """(T, D, dtype code, table pointers, row counts as C array and as list, state pointers, the
    tensors whose device the call must check) of a table list or a TableSet."""
    if isinstance(tables, TableSet):
        tables.refresh()
        sptrs, extra = None, ()
        if with_state:
            if state is None or state is tables.states:
                if tables.sptrs is None and need_state:
                    raise ValueError("row-wise Adagrad needs one state vector per table")
                sptrs = tables.sptrs
            else:
                sptrs, extra = _states(state, tables.tables, need_state), tuple(state)
        return (tables.T, tables.D, tables.code, tables.ptrs, tables.rows, tables.row_counts, sptrs,
                (tables.tables[0],) + extra)
    T, D, code, ptrs, rows = _tables(tables)
    sptrs = _states(state, tables, need_state) if with_state else None
    dev_tensors = tuple(tables) + (tuple(state) if with_state and state is not None else ())
    return T, D, code, ptrs, rows, [int(t.shape[0]) for t in tables], sptrs, dev_tensors


def _batch(T: int, indices, offsets, per_sample_weights, index_dtypes=(torch.int64,)):
    """Checks the CSR batch; returns (indices, offsets, weights, index code, B, nnz)."""
    _need(indices, "indices", index_dtypes)
    _need(offsets, "offsets", indices.dtype)
    if indices.dim() != 1 or offsets.dim() != 1:
        raise ValueError("indices and offsets must be 1-D")
    B = (offsets.numel() - 1) // T
    if offsets.numel() < 1 or offsets.numel() != T * B + 1:
        raise ValueError(f"offsets must have T*B+1 entries (T={T}), got {offsets.numel()}")
    nnz = indices.numel()
    w = _opt(per_sample_weights, "per_sample_weights", torch.float32, (nnz,))
    code = DLRM_INDEX_I32 if indices.dtype == torch.int32 else DLRM_INDEX_I64
    return indices, offsets, w, code, B, nnz


def _outputs(o, nnz: int):
    """The optional integer outputs of the embedding backward, each sized for nnz lookups."""
    if o is None:
        return None
    _need(o.unique_keys, "outputs.unique_keys", torch.int64, min_numel=nnz)
    _need(o.segment_offsets, "outputs.segment_offsets", torch.int64, min_numel=nnz + 1)
    _need(o.sorted_pos, "outputs.sorted_pos", torch.int32, min_numel=nnz)
    _need(o.num_unique, "outputs.num_unique", torch.int64, min_numel=1)
    return o


def _workspace(workspace, need: int, dev):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8)
    if workspace.numel() < need:
        raise ValueError(f"workspace holds {workspace.numel()} bytes, the call needs {need}")
    return workspace


def emb_bag_fwd(tables: Sequence[torch.Tensor], indices: torch.Tensor, offsets: torch.Tensor,
                per_sample_weights: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, flags: int = 0) -> torch.Tensor:
    """Pooled embeddings [B, T, D] fp32 (C: emb_bag_fwd)."""
    T, D, code, ptrs, rows, _, _, dt = _prepared(tables)
    indices, offsets, w, _, B, nnz = _batch(T, indices, offsets, per_sample_weights)
    out = _opt(out, "out", torch.float32, (B, T, D))
    dev = _device(*dt, indices, offsets, w, out)
    if out is None:
        out = torch.empty((B, T, D), dtype=torch.float32, device=dev)
    _check(lib().emb_bag_fwd(ptrs, rows, T, D, code, _ptr(indices), _ptr(offsets), _ptr(w), B,
                             nnz, _ptr(out), flags, _stream(dev)), "emb_bag_fwd")
    return out


def emb_bag_fwd_ex(tables: Sequence[torch.Tensor], indices: torch.Tensor, offsets: torch.Tensor,
                   per_sample_weights: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   out_dtype: torch.dtype = torch.float32, flags: int = 0) -> torch.Tensor:
    """Pooled embeddings [B, T, D] in out_dtype (fp32 or bf16), int64 or int32 indices and
    offsets (C: emb_bag_fwd_ex)."""
    T, D, code, ptrs, rows, _, _, dt = _prepared(tables)
    indices, offsets, w, icode, B, nnz = _batch(T, indices, offsets, per_sample_weights,
                                                (torch.int64, torch.int32))
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"out_dtype must be float32 or bfloat16, got {out_dtype}")
    ocode = DLRM_F32 if out_dtype == torch.float32 else DLRM_BF16
    out = _opt(out, "out", out_dtype, (B, T, D))
    dev = _device(*dt, indices, offsets, w, out)
    if out is None:
        out = torch.empty((B, T, D), dtype=out_dtype, device=dev)
    _check(lib().emb_bag_fwd_ex(ptrs, rows, T, D, code, _ptr(indices), _ptr(offsets), icode, _ptr(w), B,
                                nnz, _ptr(out), ocode, flags, _stream(dev)), "emb_bag_fwd_ex")
    return out


def _interaction_shapes(dense: torch.Tensor, pooled: torch.Tensor):
    _need(dense, "dense", torch.float32)
    _need(pooled, "pooled", torch.float32)
    if dense.dim() != 2 or pooled.dim() != 3:
        raise ValueError("dense must be [B, D] and pooled [B, N-1, D]")
    B, D = dense.shape
    if pooled.shape[0] != B or pooled.shape[2] != D:
        raise ValueError(f"pooled must be [B={B}, N-1, D={D}], got {tuple(pooled.shape)}")
    N = pooled.shape[1] + 1
    return B, N, D, N * (N - 1) // 2


def dlrm_interact_fwd(dense: torch.Tensor, pooled: torch.Tensor,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """[B, N(N-1)/2 + D] fp32 (C: dlrm_interact_fwd); pooled is [B, N-1, D]."""
    B, N, D, P = _interaction_shapes(dense, pooled)
    out = _opt(out, "out", torch.float32, (B, P + D))
    dev = _device(dense, pooled, out)
    if out is None:
        out = torch.empty((B, P + D), dtype=torch.float32, device=dev)
    _check(lib().dlrm_interact_fwd(_ptr(dense), _ptr(pooled), B, N, D, _ptr(out),
                                   _stream(dev)), "dlrm_interact_fwd")
    return out


def dlrm_interact_fwd_ex(dense: torch.Tensor, pooled: torch.Tensor, path: int = DLRM_GRAM_AUTO,
                         out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dlrm_interact_fwd with the Gram path chosen: DLRM_GRAM_AUTO, _MFMA or _VALU (C: dlrm_interact_fwd_ex)."""
    B, N, D, P = _interaction_shapes(dense, pooled)
    out = _opt(out, "out", torch.float32, (B, P + D))
    dev = _device(dense, pooled, out)
    if out is None:
        out = torch.empty((B, P + D), dtype=torch.float32, device=dev)
    _check(lib().dlrm_interact_fwd_ex(_ptr(dense), _ptr(pooled), B, N, D, _ptr(out), int(path), _stream(dev)),
           "dlrm_interact_fwd_ex")
    return out


def emb_bag_interact_fwd(tables: Sequence[torch.Tensor], indices: torch.Tensor, offsets: torch.Tensor,
                         per_sample_weights: Optional[torch.Tensor], dense: torch.Tensor,
                         out: Optional[torch.Tensor] = None, flags: int = 0) -> torch.Tensor:
    """[B, N(N-1)/2 + D] fp32, N = T + 1: lookup fused with the interaction (C: emb_bag_interact_fwd)."""
    T, D, code, ptrs, rows, _, _, dt = _prepared(tables)
    indices, offsets, w, _, B, nnz = _batch(T, indices, offsets, per_sample_weights)
    _need(dense, "dense", torch.float32, (B, D))
    N = T + 1
    out = _opt(out, "out", torch.float32, (B, N * (N - 1) // 2 + D))
    dev = _device(*dt, indices, offsets, w, dense, out)
    if out is None:
        out = torch.empty((B, N * (N - 1) // 2 + D), dtype=torch.float32, device=dev)
    _check(lib().emb_bag_interact_fwd(ptrs, rows, T, D, code, _ptr(indices), _ptr(offsets), _ptr(w), B,
                                      nnz, _ptr(dense), _ptr(out), flags, _stream(dev)),
           "emb_bag_interact_fwd")
    return out


def dlrm_interact_bwd(grad_out: torch.Tensor, dense: torch.Tensor, pooled: torch.Tensor,
                      grad_dense: Optional[torch.Tensor] = None,
                      grad_pooled: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(grad_dense [B, D], grad_pooled [B, N-1, D]) (C: dlrm_interact_bwd)."""
    B, N, D, P = _interaction_shapes(dense, pooled)
    _need(grad_out, "grad_out", torch.float32, (B, P + D))
    grad_dense = _opt(grad_dense, "grad_dense", torch.float32, (B, D))
    grad_pooled = _opt(grad_pooled, "grad_pooled", torch.float32, (B, N - 1, D))
    dev = _device(grad_out, dense, pooled, grad_dense, grad_pooled)
    if grad_dense is None:
        grad_dense = torch.empty_like(dense)
    if grad_pooled is None:
        grad_pooled = torch.empty_like(pooled)
    _check(lib().dlrm_interact_bwd(_ptr(grad_out), _ptr(dense), _ptr(pooled), B, N, D,
                                   _ptr(grad_dense), _ptr(grad_pooled), _stream(dev)),
           "dlrm_interact_bwd")
    return grad_dense, grad_pooled


def emb_bag_bwd_workspace_size(rows: Sequence[int], D: int, B: int, nnz: int) -> int:
    T = len(rows)
    r = (ctypes.c_int64 * T)(*rows)
    return int(lib().emb_bag_bwd_workspace_size(T, r, D, B, nnz))


class AdagradOutputs:
    """Optional integer outputs of emb_bag_bwd_adagrad (device tensors)."""

    def __init__(self, nnz: int, device):
        n1 = max(nnz, 1)
        self.unique_keys = torch.empty(n1, dtype=torch.int64, device=device)
        self.segment_offsets = torch.empty(n1 + 1, dtype=torch.int64, device=device)
        self.sorted_pos = torch.empty(n1, dtype=torch.int32, device=device)
        self.num_unique = torch.empty(1, dtype=torch.int64, device=device)


def _out_ptrs(o):
    if o is None:
        return None, None, None, None
    return _ptr(o.unique_keys), _ptr(o.segment_offsets), _ptr(o.sorted_pos), _ptr(o.num_unique)


def _out_tensors(o):
    return () if o is None else (o.unique_keys, o.segment_offsets, o.sorted_pos, o.num_unique)


def emb_bag_bwd_adagrad(tables: Sequence[torch.Tensor], state: Sequence[torch.Tensor],
                        indices: torch.Tensor, offsets: torch.Tensor,
                        per_sample_weights: Optional[torch.Tensor], grad_pooled: torch.Tensor,
                        lr: float, eps: float, workspace: Optional[torch.Tensor] = None,
                        outputs: Optional[AdagradOutputs] = None, flags: int = 0) -> Optional[AdagradOutputs]:
    """Row-wise Adagrad on the tables and states, in place (C: emb_bag_bwd_adagrad); `state` may
    be None when `tables` is a TableSet with states."""
    T, D, code, ptrs, rows, counts, sptrs, dt = _prepared(tables, state, True, True)
    indices, offsets, w, _, B, nnz = _batch(T, indices, offsets, per_sample_weights)
    _need(grad_pooled, "grad_pooled", torch.float32, (B, T, D))
    o = _outputs(outputs, nnz)
    need = emb_bag_bwd_workspace_size(counts, D, B, nnz)
    workspace = _opt(workspace, "workspace", torch.uint8, min_numel=need)
    dev = _device(*dt, indices, offsets, w, grad_pooled, workspace, *_out_tensors(o))
    workspace = _workspace(workspace, need, dev)
    _check(lib().emb_bag_bwd_adagrad(
        ptrs, sptrs, rows, T, D, code, _ptr(indices), _ptr(offsets), _ptr(w), B, nnz,
        _ptr(grad_pooled), float(lr), float(eps), _ptr(workspace), workspace.numel(), *_out_ptrs(o), flags,
        _stream(dev)), "emb_bag_bwd_adagrad")
    return o


def emb_bag_bwd_update(tables: Sequence[torch.Tensor], state: Optional[Sequence[torch.Tensor]],
                       indices: torch.Tensor, offsets: torch.Tensor,
                       per_sample_weights: Optional[torch.Tensor], grad_pooled: torch.Tensor,
                       optimizer: int, lr: float, eps: float = 0.0,
                       workspace: Optional[torch.Tensor] = None, outputs: Optional[AdagradOutputs] = None,
                       flags: int = 0) -> Optional[AdagradOutputs]:
    """Embedding backward with DLRM_OPT_ADAGRAD (state required) or DLRM_OPT_SGD (state may be
    None), int64 or int32 indices and offsets (C: emb_bag_bwd_update)."""
    T, D, code, ptrs, rows, counts, sptrs, dt = _prepared(tables, state, optimizer == DLRM_OPT_ADAGRAD, True)
    indices, offsets, w, icode, B, nnz = _batch(T, indices, offsets, per_sample_weights,
                                                (torch.int64, torch.int32))
    _need(grad_pooled, "grad_pooled", torch.float32, (B, T, D))
    o = _outputs(outputs, nnz)
    need = emb_bag_bwd_workspace_size(counts, D, B, nnz)
    workspace = _opt(workspace, "workspace", torch.uint8, min_numel=need)
    dev = _device(*dt, indices, offsets, w, grad_pooled, workspace, *_out_tensors(o))
    workspace = _workspace(workspace, need, dev)
    _check(lib().emb_bag_bwd_update(
        ptrs, sptrs, rows, T, D, code, _ptr(indices), _ptr(offsets), icode, _ptr(w), B, nnz,
        _ptr(grad_pooled), int(optimizer), float(lr), float(eps), _ptr(workspace), workspace.numel(),
        *_out_ptrs(o), flags, _stream(dev)), "emb_bag_bwd_update")
    return o


def emb_bag_bwd_noalloc_max_bytes() -> int:
    return int(lib().emb_bag_bwd_noalloc_max_bytes())


def emb_bag_bwd_update_noalloc(tables: Sequence[torch.Tensor], state: Optional[Sequence[torch.Tensor]],
                               indices: torch.Tensor, offsets: torch.Tensor,
                               per_sample_weights: Optional[torch.Tensor], grad_pooled: torch.Tensor,
                               optimizer: int, lr: float, eps: float = 0.0,
                               outputs: Optional[AdagradOutputs] = None, flags: int = 0) -> Optional[AdagradOutputs]:
    """emb_bag_bwd_update with the library's fixed per-GPU scratch as the workspace: allocates
    nothing (C: emb_bag_bwd_update_noalloc).  Calls that overlap on one GPU race."""
    T, D, code, ptrs, rows, _, sptrs, dt = _prepared(tables, state, optimizer == DLRM_OPT_ADAGRAD, True)
    indices, offsets, w, icode, B, nnz = _batch(T, indices, offsets, per_sample_weights,
                                                (torch.int64, torch.int32))
    _need(grad_pooled, "grad_pooled", torch.float32, (B, T, D))
    o = _outputs(outputs, nnz)
    dev = _device(*dt, indices, offsets, w, grad_pooled, *_out_tensors(o))
    _check(lib().emb_bag_bwd_update_noalloc(
        ptrs, sptrs, rows, T, D, code, _ptr(indices), _ptr(offsets), icode, _ptr(w), B, nnz,
        _ptr(grad_pooled), int(optimizer), float(lr), float(eps), *_out_ptrs(o), flags, _stream(dev)),
        "emb_bag_bwd_update_noalloc")
    return o


def emb_bag_bwd_plan(rows: Sequence[int], D: int, indices: torch.Tensor, offsets: torch.Tensor,
                     per_sample_weights: Optional[torch.Tensor], workspace: torch.Tensor,
                     outputs: Optional[AdagradOutputs] = None, flags: int = 0) -> Optional[AdagradOutputs]:
    """The batch-only half of the embedding backward (C: emb_bag_bwd_plan), on the current stream
    of the indices' device; `rows` are the tables' row counts."""
    T = len(rows)
    r = (ctypes.c_int64 * T)(*rows)
    indices, offsets, w, icode, B, nnz = _batch(T, indices, offsets, per_sample_weights,
                                                (torch.int64, torch.int32))
    o = _outputs(outputs, nnz)
    _need(workspace, "workspace", torch.uint8, min_numel=emb_bag_bwd_workspace_size(rows, D, B, nnz))
    dev = _device(indices, offsets, w, workspace, *_out_tensors(o))
    _check(lib().emb_bag_bwd_plan(
        r, T, D, _ptr(indices), _ptr(offsets), icode, _ptr(w), B, nnz, _ptr(workspace), workspace.numel(),
        *_out_ptrs(o), flags, _stream(dev)), "emb_bag_bwd_plan")
    return o


def emb_bag_bwd_apply(tables: Sequence[torch.Tensor], state: Optional[Sequence[torch.Tensor]], B: int, nnz: int,
                      weighted: bool, grad_pooled: torch.Tensor, optimizer: int, lr: float, eps: float,
                      workspace: torch.Tensor, outputs: Optional[AdagradOutputs] = None) -> None:
    """The update half of the embedding backward from a planned workspace (C: emb_bag_bwd_apply);
    `outputs` is the plan's, when it was given one (its segment offsets are read)."""
    T, D, code, ptrs, rows, counts, sptrs, dt = _prepared(tables, state, optimizer == DLRM_OPT_ADAGRAD, True)
    B, nnz = int(B), int(nnz)
    _need(grad_pooled, "grad_pooled", torch.float32, (B, T, D))
    seg = None
    if outputs is not None:
        seg = _need(outputs.segment_offsets, "outputs.segment_offsets", torch.int64, min_numel=nnz + 1)
    _need(workspace, "workspace", torch.uint8, min_numel=emb_bag_bwd_workspace_size(counts, D, B, nnz))
    dev = _device(*dt, grad_pooled, workspace, seg)
    _check(lib().emb_bag_bwd_apply(
        ptrs, sptrs, rows, T, D, code, B, nnz, 1 if weighted else 0, _ptr(grad_pooled), int(optimizer),
        float(lr), float(eps), _ptr(workspace), workspace.numel(), _ptr(seg), _stream(dev)),
        "emb_bag_bwd_apply")


def dlrm_synth_fill_table(table: torch.Tensor, t: int, seed: int, scale: float) -> None:
    """Fill ``table`` with the counter-hash contents of table ``t`` (input generation)."""
    _need(table, "table", (torch.float32, torch.bfloat16))
    if table.dim() != 2:
        raise ValueError("table must be [V, D]")
    dev = _device(table)
    _check(lib().dlrm_synth_fill_table(_ptr(table), _dtype_code(table), table.shape[0],
                                       table.shape[1], t, seed, float(scale),
                                       _stream(dev)), "dlrm_synth_fill_table")


# ---------------------------------------------------------------- HBM read probes (dlrm_probe.h)

def dlrm_probe_read(buf: torch.Tensor, sink: torch.Tensor) -> None:
    """Stream-read every byte of ``buf`` once (C: dlrm_probe_read); ``sink`` is uint32/int32 scratch."""
    _need(buf, "buf")
    _need(sink, "sink", (torch.int32,))
    nbytes = buf.numel() * buf.element_size()
    if nbytes == 0 or nbytes % 16:
        raise ValueError("buf must hold a positive multiple of 16 bytes")
    dev = _device(buf, sink)
    _check(lib().dlrm_probe_read(_ptr(buf), nbytes, _ptr(sink), sink.numel(), _stream(dev)), "dlrm_probe_read")


def dlrm_probe_gather(table: torch.Tensor, idx: torch.Tensor, sink: torch.Tensor) -> None:
    """Read rows ``idx`` of the 2-D ``table`` with no output (C: dlrm_probe_gather)."""
    _need(table, "table")
    if table.dim() != 2:
        raise ValueError("table must be [rows, cols]")
    _need(idx, "idx", torch.int64)
    _need(sink, "sink", (torch.int32,))
    dev = _device(table, idx, sink)
    _check(lib().dlrm_probe_gather(_ptr(table), table.shape[0], table.shape[1] * table.element_size(), _ptr(idx),
                                   idx.numel(), _ptr(sink), sink.numel(), _stream(dev)), "dlrm_probe_gather")


# ---------------------------------------------------------------- dense layers (dlrm_mlp.h)

_TORCH_CODE = {torch.float32: DLRM_F32, torch.bfloat16: DLRM_BF16}
_NORM_CODE = {**_TORCH_CODE, torch.float8_e4m3fn: DLRM_F8_E4M3}


def dlrm_linear_workspace_size(M: int, N: int, K: int) -> int:
    return int(lib().dlrm_linear_workspace_size(M, N, K))


def dlrm_bce_head_workspace_size(M: int, K: int) -> int:
    return int(lib().dlrm_bce_head_workspace_size(M, K))


def _ws(nbytes: int, dev, workspace: Optional[torch.Tensor]) -> torch.Tensor:
    """The caller's workspace when it is large enough, else a new one."""
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8)
        if workspace.device != dev:
            raise ValueError(f"workspace must be on {dev}, found it on {workspace.device}")
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    return workspace


def _ws_if(nbytes: int, dev, workspace: Optional[torch.Tensor]):
    """_ws of a call that uses none where its size is 256: (its address, its bytes) and the tensor, which keeps it."""
    if nbytes <= 256 and workspace is None:
        return None, 0, None
    workspace = _ws(nbytes, dev, workspace)
    return workspace.data_ptr(), workspace.numel(), workspace


def _mat(t, name: str, dtype) -> torch.Tensor:
    _need(t, name, dtype)
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix, got shape {tuple(t.shape)}")
    return t


def dlrm_linear_fwd(x: torch.Tensor, W: torch.Tensor, b: torch.Tensor, act: int = DLRM_ACT_RELU,
                    y: Optional[torch.Tensor] = None, y_dtype: torch.dtype = torch.bfloat16,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y = act(x W^T + b), x [M][K] bf16, W [N][K] bf16, b [N] fp32 (C: dlrm_linear_fwd)."""
    M, K = _mat(x, "x", torch.bfloat16).shape
    N = _mat(W, "W", torch.bfloat16).shape[0]
    if W.shape[1] != K:
        raise ValueError(f"W must be [N, K={K}], got {tuple(W.shape)}")
    _need(b, "b", torch.float32, (N,))
    y = _opt(y, "y", (torch.float32, torch.bfloat16) if y is not None else None, (M, N))
    dev = _device(x, W, b, y)
    if y is None:
        if y_dtype not in _TORCH_CODE:
            raise ValueError(f"y_dtype must be float32 or bfloat16, got {y_dtype}")
        y = torch.empty((M, N), dtype=y_dtype, device=dev)
    ws = _ws(dlrm_linear_workspace_size(M, N, K), dev, workspace)
    _check(lib().dlrm_linear_fwd(_ptr(x), _ptr(W), _ptr(b), M, N, K, act, _ptr(y), _TORCH_CODE[y.dtype], _ptr(ws),
                                 ws.numel(), _stream(dev)), "dlrm_linear_fwd")
    return y


def dlrm_linear_bwd(dy: torch.Tensor, y: Optional[torch.Tensor], act: int, x: torch.Tensor, W: torch.Tensor,
                    want_dx: bool = True, dz_bf16: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                    dW: Optional[torch.Tensor] = None, db: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None):
    """(dx or None, dW, db) of y = act(x W^T + b) given dy fp32 (C: dlrm_linear_bwd)."""
    M, K = _mat(x, "x", torch.bfloat16).shape
    N = _mat(W, "W", torch.bfloat16).shape[0]
    if W.shape[1] != K:
        raise ValueError(f"W must be [N, K={K}], got {tuple(W.shape)}")
    _need(dy, "dy", torch.float32, (M, N))
    if act == DLRM_ACT_RELU and y is None:
        raise ValueError("the ReLU backward needs the forward output y")
    y = _opt(y, "y", (torch.float32, torch.bfloat16), (M, N))
    dz_bf16 = _opt(dz_bf16, "dz_bf16", torch.bfloat16, (M, N))
    dx = _opt(dx, "dx", torch.float32, (M, K)) if want_dx else None
    dW = _opt(dW, "dW", torch.float32, (N, K))
    db = _opt(db, "db", torch.float32, (N,))
    dev = _device(dy, y, x, W, dz_bf16, dx, dW, db)
    if dz_bf16 is None:
        dz_bf16 = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    if want_dx and dx is None:
        dx = torch.empty((M, K), dtype=torch.float32, device=dev)
    if dW is None:
        dW = torch.empty((N, K), dtype=torch.float32, device=dev)
    if db is None:
        db = torch.empty(N, dtype=torch.float32, device=dev)
    ycode = _TORCH_CODE[y.dtype] if y is not None else DLRM_F32
    ws = _ws(dlrm_linear_workspace_size(M, N, K), dev, workspace)
    _check(lib().dlrm_linear_bwd(_ptr(dy), _ptr(y), ycode, act, _ptr(x), _ptr(W), M, N, K, _ptr(dz_bf16),
                                 _ptr(dx) if want_dx else None, _ptr(dW), _ptr(db), _ptr(ws), ws.numel(),
                                 _stream(dev)), "dlrm_linear_bwd")
    return (dx if want_dx else None), dW, db


def dlrm_bce_head(x: torch.Tensor, w: torch.Tensor, b: torch.Tensor, t: torch.Tensor,
                  workspace: Optional[torch.Tensor] = None, out: Optional[dict] = None) -> dict:
    """Sigmoid head + mean BCE, forward and backward: dict p, loss, dx, dw, db (C: dlrm_bce_head)."""
    M, K = _mat(x, "x", torch.bfloat16).shape
    _need(w, "w", torch.bfloat16, (K,))
    _need(b, "b", torch.float32, (1,))
    _need(t, "t", torch.float32, (M,))
    if out is not None:
        for k, shp in (("p", (M,)), ("loss", (1,)), ("dx", (M, K)), ("dw", (K,)), ("db", (1,))):
            _need(out[k], f"out[{k!r}]", torch.float32, shp)
    dev = _device(x, w, b, t, *(out.values() if out is not None else ()))
    o = out if out is not None else {
        "p": torch.empty(M, dtype=torch.float32, device=dev), "loss": torch.empty(1, dtype=torch.float32, device=dev),
        "dx": torch.empty((M, K), dtype=torch.float32, device=dev), "dw": torch.empty(K, dtype=torch.float32, device=dev),
        "db": torch.empty(1, dtype=torch.float32, device=dev)}
    ws = _ws(dlrm_bce_head_workspace_size(M, K), dev, workspace)
    _check(lib().dlrm_bce_head(_ptr(x), _ptr(w), _ptr(b), _ptr(t), M, K, _ptr(o["p"]), _ptr(o["loss"]), _ptr(o["dx"]),
                               _ptr(o["dw"]), _ptr(o["db"]), _ptr(ws), ws.numel(), _stream(dev)), "dlrm_bce_head")
    return o


def dlrm_sgd_dense(w32: torch.Tensor, w16: Optional[torch.Tensor], g: torch.Tensor, lr: float) -> None:
    """w32 -= lr * g; w16 <- bf16(w32) when given (C: dlrm_sgd_dense)."""
    _need(w32, "w32", torch.float32)
    _need(g, "g", torch.float32, tuple(w32.shape))
    w16 = _opt(w16, "w16", torch.bfloat16, tuple(w32.shape))
    dev = _device(w32, w16, g)
    _check(lib().dlrm_sgd_dense(_ptr(w32), _ptr(w16), _ptr(g), w32.numel(), float(lr),
                                _stream(dev)), "dlrm_sgd_dense")


def dlrm_sgd_dense_multi(params: Sequence, lr: float) -> None:
    """For each (w32, w16 or None, g): w32 -= lr * g and w16 <- bf16(w32), in one launch
    (C: dlrm_sgd_dense_multi)."""
    count = len(params)
    if count == 0:
        return
    w32s, w16s, gs, ns, every = [], [], [], [], []
    for i, (w32, w16, g) in enumerate(params):
        _need(w32, f"params[{i}].w32", torch.float32)
        _need(g, f"params[{i}].g", torch.float32, tuple(w32.shape))
        _opt(w16, f"params[{i}].w16", torch.bfloat16, tuple(w32.shape))
        every += [w32, w16, g]
        w32s.append(w32.data_ptr())
        w16s.append(w16.data_ptr() if w16 is not None else None)
        gs.append(g.data_ptr())
        ns.append(w32.numel())
    dev = _device(*every)
    vp = ctypes.c_void_p * count
    _check(lib().dlrm_sgd_dense_multi(count, vp(*w32s), vp(*w16s), vp(*gs), (ctypes.c_int64 * count)(*ns), float(lr),
                                      _stream(dev)), "dlrm_sgd_dense_multi")


def dlrm_cast_rows(src: torch.Tensor, cols: int, dst_cols: int, dst_dtype: torch.dtype,
                   dst: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dst [M][dst_cols]: the first `cols` columns of src converted, the rest zero (C: dlrm_cast_rows)."""
    if not isinstance(src, torch.Tensor) or src.dim() != 2 or src.stride(1) != 1:
        raise ValueError("src must be a 2-D matrix with packed rows")
    if src.dtype not in _TORCH_CODE:
        raise ValueError(f"src must be float32 or bfloat16, got {src.dtype}")
    if not (0 <= cols <= src.shape[1] and cols <= dst_cols):
        raise ValueError(f"need cols <= src columns ({src.shape[1]}) and cols <= dst_cols ({dst_cols})")
    M = src.shape[0]
    if dst_dtype not in _TORCH_CODE:
        raise ValueError(f"dst_dtype must be float32 or bfloat16, got {dst_dtype}")
    dst = _opt(dst, "dst", dst_dtype, (M, dst_cols))
    dev = _device(src, dst)
    if dst is None:
        dst = torch.empty((M, dst_cols), dtype=dst_dtype, device=dev)
    _check(lib().dlrm_cast_rows(_ptr(src), _TORCH_CODE[src.dtype], src.stride(0), M, cols, _ptr(dst),
                                _TORCH_CODE[dst.dtype], dst_cols, _stream(dev)), "dlrm_cast_rows")
    return dst


# ---------------------------------------------------------------- user histories (dlrm_seq.h)

def dlrm_seq_bucket_bounds(buckets: int, reach: int) -> List[int]:
    """First distances of `buckets` distance buckets for dlrm_seq_attn_*: one distance a bucket for the
    first half, then growing by an equal factor up to `reach`; the last bucket is open."""
    if buckets < 1 or buckets > DLRM_SEQ_MAX_BUCKETS:
        raise ValueError(f"buckets must be 1 to {DLRM_SEQ_MAX_BUCKETS}, got {buckets}")
    half = max(1, buckets // 2)
    out = list(range(half))
    for i in range(half, buckets):
        f = (i - half) / max(1, buckets - 1 - half)
        out.append(max(out[-1] + 1, int(round(half * (max(reach, half + 1) / half) ** f))))
    return out


def _out(t, name: str, dtype: torch.dtype, shape, dev: torch.device) -> torch.Tensor:
    """The caller's output tensor, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _is(t, name, dtype, shape)
    if t.device != dev:
        raise ValueError(f"all tensors must be on {dev}, found one on {t.device}")
    return t


def _out_like(t, name: str, like: torch.Tensor, shape, dev: torch.device) -> torch.Tensor:
    """_out of `like`'s type, which costs two thirds where it has the shape."""
    if t is None and like.is_contiguous() and like.shape == shape:
        return torch.empty_like(like)
    return _out(t, name, like.dtype, shape, dev)


def _head_rows(t, name: str, heads: Optional[int] = None, d: Optional[int] = None):
    """Checks [rows, heads, d] bf16 whose heads are packed and whose row and head strides are free (a
    part of a joint projection, for instance); returns (rows, heads, d, row stride, head stride)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype is not torch.bfloat16:
        raise ValueError(f"{name} must be torch.bfloat16, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or (heads is not None and shape[1] != heads) or (d is not None and shape[2] != d):
        raise ValueError(f"{name} must be [rows, heads={heads}, d={d}], got {tuple(shape)}")
    rows, H, w = shape
    if H < 1 or w < 1:
        raise ValueError(f"{name} must have heads and columns, got {tuple(shape)}")
    row, head, one = t.stride()
    if one != 1 and rows and w > 1:
        raise ValueError(f"{name} must have packed heads (stride 1 in the last dimension)")
    if H == 1 or not rows:  # the stride of a dimension of one entry is of no account
        head = w
    if rows < 2:  # as is that of one row: H * head may pass the limit on row strides
        row = w
    return rows, H, w, row, head


def _offsets(t, name: str, n: Optional[int] = None) -> torch.Tensor:
    _need(t, name, (torch.int64, torch.int32))
    if t.dim() != 1 or t.numel() < 1 or (n is not None and t.numel() != n):
        raise ValueError(f"{name} must be 1-D with {n if n is not None else 'B+1'} entries, got {tuple(t.shape)}")
    return t


def _count(v, name: str) -> int:
    v = int(v)
    if not 0 <= v < 1 << 31:
        raise ValueError(f"{name} must be 0 or more and below 2^31, got {v}")
    return v


def _seq_attn(q, k, v, q_offsets, begin, end, B, window, sinks, scale, bias, bounds):
    """The checked description of an attention call: (its bytes, what they point to, device, (Nq, Hq, d),
    buckets)."""
    Nq, Hq, d, q_row, q_head = _head_rows(q, "q")
    Nkv, Hkv, _, k_row, k_head = _head_rows(k, "k", None, d)
    Nv, _, _, v_row, v_head = _head_rows(v, "v", Hkv, d)
    if Nv != Nkv:
        raise ValueError(f"k and v must have the same rows, got {Nkv} and {Nv}")
    if Hq % Hkv:
        raise ValueError(f"q's heads must be a multiple of k's, got {Hq} and {Hkv}")
    if d % 8 or d > 128:
        raise ValueError(f"a head must have a multiple of 8 columns, at most 128, got {d}")
    index = q_offsets if begin is None else begin  # without ranges the keys are in pages
    if (q_offsets is not None and index.dtype != q_offsets.dtype) or (begin is not None and end.dtype != begin.dtype):
        raise ValueError("all offsets must have one type")
    if (bias is None) != (bounds is None):
        raise ValueError("bias and bounds go together")
    n, edges, at = 0, None, 0
    if bias is not None:
        n = len(bounds)
        if not 1 <= n <= DLRM_SEQ_MAX_BUCKETS or bounds[0] != 0 or not all(map(operator.lt, bounds, bounds[1:])):
            raise ValueError(f"bounds must be 1 to {DLRM_SEQ_MAX_BUCKETS} strictly increasing distances from 0 on")
        if bounds[-1] >= 1 << 31:
            raise ValueError("bounds must be below 2^31")
        _need(bias, "bias", torch.float32, (Hq, n))
        edges = array.array("i", bounds)
        at = edges.buffer_info()[0]
    dev = _device(q, k, v, q_offsets, begin, end, bias)
    code = DLRM_INDEX_I32 if index is not None and index.dtype is torch.int32 else DLRM_INDEX_I64
    desc = _SEQ_ATTN.pack(B, Nq, Nkv, Hq, Hkv, d, code, 0 if q_offsets is None else q_offsets.data_ptr(),
                          0 if begin is None else begin.data_ptr(), 0 if end is None else end.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), q_row, q_head, k_row, k_head, v_row, v_head,
                          _count(window, "window"), _count(sinks, "sinks"), d ** -0.5 if scale is None else float(scale), n,
                          0 if bias is None else bias.data_ptr(), at)
    return desc, edges, dev, (Nq, Hq, d), n


def _kv_ranges(kv_offsets, B: int):
    """(begin, end) of B sequences' keys, from offsets [B+1] or from such a pair."""
    if isinstance(kv_offsets, (tuple, list)):
        begin, end = kv_offsets
        return _offsets_b(begin, "kv_begin", B), _offsets_b(end, "kv_end", B)
    _offsets(kv_offsets, "kv_offsets", B + 1)
    return kv_offsets[:-1], kv_offsets[1:]


def _offsets_b(t, name: str, B: int) -> torch.Tensor:
    return _need(t, name, (torch.int64, torch.int32), (B,))


def dlrm_seq_attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_offsets: torch.Tensor, kv_offsets=None, *,
                      window: int = 0, sinks: int = 0, scale: Optional[float] = None,
                      bias: Optional[torch.Tensor] = None, bounds: Optional[Sequence[int]] = None,
                      for_backward: bool = False, out: Optional[torch.Tensor] = None,
                      tiles: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None):
    """Causal attention over jagged sequences (C: dlrm_seq_attn_fwd): o [Nq, Hq, d] bf16, or with
    for_backward (o, tiles, lse), what dlrm_seq_attn_bwd takes.  q is [Nq, Hq, d], k and v
    [Nkv, Hkv, d]; the queries are the last events of their sequence.  kv_offsets: offsets [B+1], a
    (begin, end) pair of [B], or None: the queries' own.  scale: None is 1 / sqrt(d).
    bias [Hq, buckets] with bounds, the first distance of each bucket (dlrm_seq_bucket_bounds)."""
    _offsets(q_offsets, "q_offsets")
    B = q_offsets.numel() - 1
    begin, end = _kv_ranges(q_offsets if kv_offsets is None else kv_offsets, B)
    a, edges, dev, shape, _ = _seq_attn(q, k, v, q_offsets, begin, end, B, window, sinks, scale, bias, bounds)
    for_backward = for_backward or tiles is not None or lse is not None
    out = _out(out, "out", torch.bfloat16, shape, dev)
    if for_backward:
        tiles = _out(tiles, "tiles", torch.int32, (lib().dlrm_seq_attn_tiles(B, shape[0]),), dev)
        lse = _out(lse, "lse", torch.float32, shape[:2], dev)
    _check(lib().dlrm_seq_attn_fwd(a, _ptr(out), _ptr(lse), _ptr(tiles), _stream(dev)), "dlrm_seq_attn_fwd")
    return (out, tiles, lse) if for_backward else out


def dlrm_seq_attn_bwd(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                      tiles: torch.Tensor, lse: torch.Tensor, q_offsets: torch.Tensor,
                      kv_offsets: Optional[torch.Tensor] = None, *, window: int = 0, sinks: int = 0,
                      scale: Optional[float] = None, bias: Optional[torch.Tensor] = None,
                      bounds: Optional[Sequence[int]] = None, dq: Optional[torch.Tensor] = None,
                      dk: Optional[torch.Tensor] = None, dv: Optional[torch.Tensor] = None,
                      dbias: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """(dq, dk, dv, dbias or None) of dlrm_seq_attn_fwd (C: dlrm_seq_attn_bwd); o, tiles and lse are what
    it gave with for_backward, the other arguments its own; kv_offsets is None or offsets [B+1]."""
    _offsets(q_offsets, "q_offsets")
    B = q_offsets.numel() - 1
    if isinstance(kv_offsets, (tuple, list)):
        raise ValueError("the backward takes kv_offsets [B+1]: every key row in one sequence")
    begin, end = _kv_ranges(q_offsets if kv_offsets is None else kv_offsets, B)
    a, edges, dev, qs, _ = _seq_attn(q, k, v, q_offsets, begin, end, B, window, sinks, scale, bias, bounds)
    ks = tuple(k.shape)
    bf = torch.bfloat16
    _is(dout, "dout", bf, qs)
    _is(o, "o", bf, qs)
    _is(tiles, "tiles", torch.int32, (lib().dlrm_seq_attn_tiles(B, qs[0]),))
    _is(lse, "lse", torch.float32, qs[:2])
    _device(q, dout, o, tiles, lse)
    if bias is None and dbias is not None:
        raise ValueError("dbias without a bias")
    dq, dk, dv = _out(dq, "dq", bf, qs, dev), _out(dk, "dk", bf, ks, dev), _out(dv, "dv", bf, ks, dev)
    if bias is not None:
        dbias = _out(dbias, "dbias", torch.float32, tuple(bias.shape), dev)
    ws = _ws(lib().dlrm_seq_attn_bwd_workspace_size(a), dev, workspace)
    _check(lib().dlrm_seq_attn_bwd(a, _ptr(dout), _ptr(o), _ptr(lse), _ptr(tiles), _ptr(dq), _ptr(dk), _ptr(dv),
                                   _ptr(dbias), _ptr(ws), ws.numel(), _stream(dev)), "dlrm_seq_attn_bwd")
    return dq, dk, dv, dbias


def dlrm_seq_attn_decode_workspace_size(B: int, Hq: int, Hkv: int, d: int, window: int, sinks: int, max_kv_len: int) -> int:
    return int(lib().dlrm_seq_attn_decode_workspace_size(B, Hq, Hkv, d, window, sinks, max_kv_len))


def dlrm_seq_attn_decode(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, kv_begin: torch.Tensor, kv_end: torch.Tensor, *,
                         window: int = 0, sinks: int = 0, scale: Optional[float] = None,
                         bias: Optional[torch.Tensor] = None, bounds: Optional[Sequence[int]] = None,
                         max_kv_len: Optional[int] = None, out: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of one new event a sequence over its cached keys (C: dlrm_seq_attn_decode): o [B, Hq, d]
    bf16.  q is [B, Hq, d]; sequence b's keys are the rows kv_begin[b] .. kv_end[b] - 1 of k and v
    [rows, Hkv, d], the event's own the last.  max_kv_len (the sequences' longest, None: k's rows)
    only chooses how far a sequence is split."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be [B, heads, d]")
    B = q.shape[0]
    begin, end = _offsets_b(kv_begin, "kv_begin", B), _offsets_b(kv_end, "kv_end", B)
    a, edges, dev, shape, _ = _seq_attn(q, k, v, None, begin, end, B, window, sinks, scale, bias, bounds)
    longest = k.shape[0] if max_kv_len is None else int(max_kv_len)
    if longest < 0:
        raise ValueError(f"max_kv_len must not be negative, got {longest}")
    out = _out(out, "out", torch.bfloat16, shape, dev)
    ws = _ws(lib().dlrm_seq_attn_decode_workspace_size(B, shape[1], k.shape[1], shape[2], window, sinks, longest), dev, workspace)
    _check(lib().dlrm_seq_attn_decode(a, longest, _ptr(out), _ptr(ws), ws.numel(), _stream(dev)),
           "dlrm_seq_attn_decode")
    return out


def _drop_spec(p: float, seed: int, offset: int, offset_dev: Optional[torch.Tensor]) -> _Dropout:
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p must be between 0 and 1, got {p}")
    for x, name in ((seed, "seed"), (offset, "offset")):
        if not 0 <= x < 1 << 64:
            raise ValueError(f"{name} must be 0 or more and below 2^64, got {x}")
    _opt(offset_dev, "offset_dev", torch.int64, min_numel=1)
    return _Dropout(p, seed, offset, None if offset_dev is None else offset_dev.data_ptr())


def dlrm_dropout(x: torch.Tensor, p: float, seed: int, offset: int = 0, *, offset_dev: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Dropout by counter-based random numbers, no mask stored; its derivative is the same call on
    the gradient (C: dlrm_dropout).  out may be x; offset_dev: one int64 on the device, added."""
    _need(x, "x", (torch.float32, torch.bfloat16))
    out = _opt(out, "out", x.dtype, tuple(x.shape))
    spec = _drop_spec(p, seed, offset, offset_dev)
    dev = _device(x, out, offset_dev)
    if out is None:
        out = torch.empty_like(x)
    _check(lib().dlrm_dropout(_ptr(x), _TORCH_CODE[x.dtype], x.numel(), ctypes.byref(spec), _ptr(out), _stream(dev)),
           "dlrm_dropout")
    return out


def dlrm_add_rmsnorm_fwd(x: torch.Tensor, residual: Optional[torch.Tensor], w: torch.Tensor, eps: float = 1e-6, *,
                         p: float = 0.0, seed: int = 0, offset: int = 0, offset_dev: Optional[torch.Tensor] = None,
                         y_dtype: torch.dtype = torch.bfloat16, res_dtype: Optional[torch.dtype] = None,
                         s: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                         rstd: Optional[torch.Tensor] = None, y_scale: Optional[torch.Tensor] = None):
    """(s, y, rstd, y_scale or None): s = residual + dropout(x), y = s * rstd * w (C:
    dlrm_add_rmsnorm_fwd).  x and residual are [M, D]; y_dtype float8_e4m3fn gives 8-bit values to be
    multiplied by y_scale [M].  s may be the residual.  res_dtype is for a residual of None."""
    _mat(x, "x", (torch.float32, torch.bfloat16))
    M, D = x.shape
    rt = residual.dtype if isinstance(residual, torch.Tensor) else res_dtype or x.dtype
    if residual is not None:
        _is(residual, "residual", rt, (M, D))
    if rt not in _TORCH_CODE:
        raise ValueError(f"res_dtype must be float32 or bfloat16, got {rt}")
    _is(w, "w", torch.float32, (D,))
    yt = y_dtype if y is None else y.dtype
    if yt not in _NORM_CODE:
        raise ValueError(f"y_dtype must be float32, bfloat16 or float8_e4m3fn, got {yt}")
    spec = _drop_spec(p, seed, offset, offset_dev)
    dev = _device(x, residual, w, offset_dev)
    s, y = _out(s, "s", rt, (M, D), dev), _out(y, "y", yt, (M, D), dev)
    rstd = _out(rstd, "rstd", torch.float32, (M,), dev)
    if yt == torch.float8_e4m3fn:
        y_scale = _out(y_scale, "y_scale", torch.float32, (M,), dev)
    _check(lib().dlrm_add_rmsnorm_fwd(_ptr(x), _TORCH_CODE[x.dtype], _ptr(residual), _TORCH_CODE[rt], _ptr(w), float(eps),
                                      ctypes.byref(spec), M, D, _ptr(s), _ptr(y), _NORM_CODE[yt], _ptr(y_scale), _ptr(rstd),
                                      _stream(dev)), "dlrm_add_rmsnorm_fwd")
    return s, y, rstd, (y_scale if yt == torch.float8_e4m3fn else None)


def dlrm_add_rmsnorm_bwd_workspace_size(M: int, D: int) -> int:
    return int(lib().dlrm_add_rmsnorm_bwd_workspace_size(M, D))


def dlrm_add_rmsnorm_bwd(dy: torch.Tensor, ds: Optional[torch.Tensor], s: torch.Tensor, w: torch.Tensor, rstd: torch.Tensor, *,
                         x_dtype: torch.dtype = torch.bfloat16, p: float = 0.0, seed: int = 0, offset: int = 0,
                         offset_dev: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                         dresidual: Optional[torch.Tensor] = None, dw: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None):
    """(dx, dresidual, dw) of dlrm_add_rmsnorm_fwd, given dy and (or None) ds, the gradient that reaches
    s past the norm; s, w, rstd and the dropout arguments are the forward's (C: dlrm_add_rmsnorm_bwd).
    dresidual may be ds."""
    _mat(s, "s", (torch.float32, torch.bfloat16))
    M, D = s.shape
    _need(dy, "dy", (torch.float32, torch.bfloat16), (M, D))
    if ds is not None:
        _is(ds, "ds", s.dtype, (M, D))
    _is(w, "w", torch.float32, (D,))
    _is(rstd, "rstd", torch.float32, (M,))
    xt = x_dtype if dx is None else dx.dtype
    if xt not in _TORCH_CODE:
        raise ValueError(f"x_dtype must be float32 or bfloat16, got {xt}")
    spec = _drop_spec(p, seed, offset, offset_dev)
    dev = _device(dy, ds, s, w, rstd, offset_dev)
    dx, dresidual = _out(dx, "dx", xt, (M, D), dev), _out(dresidual, "dresidual", s.dtype, (M, D), dev)
    dw = _out(dw, "dw", torch.float32, (D,), dev)
    ws = _ws(lib().dlrm_add_rmsnorm_bwd_workspace_size(M, D), dev, workspace)
    _check(lib().dlrm_add_rmsnorm_bwd(_ptr(dy), _TORCH_CODE[dy.dtype], _ptr(ds), _ptr(s), _TORCH_CODE[s.dtype], _ptr(w),
                                      _ptr(rstd), ctypes.byref(spec), M, D, _ptr(dx), _TORCH_CODE[xt], _ptr(dresidual),
                                      _ptr(dw), _ptr(ws), ws.numel(), _stream(dev)), "dlrm_add_rmsnorm_bwd")
    return dx, dresidual, dw


# ---------------------------------------------------------------- paged histories (dlrm_seq_pages.h)

def _seq_pages(table, lengths, page: int, rows: int, free=None, free_count=None, pages: Optional[int] = None):
    """The checked description of the users' pages, its device's tensors."""
    if not isinstance(table, torch.Tensor) or table.dim() != 2 or table.dtype is not torch.int32:
        raise ValueError("table must be a 2-D tensor of torch.int32 [users, pages of a user]")
    B, width = table.shape
    if width > 1 and table.stride(1) != 1:
        raise ValueError("table must have packed rows")
    _is(lengths, "lengths", torch.int32, (B,))
    page = int(page)
    if page < 8 or page > 4096 or page & (page - 1):
        raise ValueError(f"page must be a power of two from 8 to 4096, got {page}")
    if pages is None:
        pages = rows // page
        if rows % page or pages < 1:
            raise ValueError(f"the pool must be whole pages of {page} rows, at least one, got {rows} rows")
    row = table.stride(0) if B > 1 else width
    if row < width:
        raise ValueError("table must have rows of its own for each user")
    return _SEQ_PAGES.pack(B, pages, row, width, page, table.data_ptr(), lengths.data_ptr(),
                           0 if free is None else free.data_ptr(), 0 if free_count is None else free_count.data_ptr())


def dlrm_seq_pages_update(table: torch.Tensor, lengths: torch.Tensor, free: torch.Tensor, free_count: torch.Tensor, page: int,
                          offsets: torch.Tensor, n: int, leave: Optional[torch.Tensor] = None, *,
                          slots: Optional[torch.Tensor] = None, refused: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(slots [n] int64, refused [1] int32): users who leave give their pages back, new events get theirs
    (C: dlrm_seq_pages_update).  table [users, width], lengths [users], free [pages], free_count [1], all int32, are
    updated in place; offsets [users+1] of the new events, n at least their last; leave [users] bool.  A refused
    user's slots are -1; behind one for whom the pool is too small everyone who wants a page is refused."""
    _offsets(offsets, "offsets")
    free = _need(free, "free", torch.int32)
    _is(free_count, "free_count", torch.int32, (1,))
    if free.dim() != 1 or free.numel() < 1:
        raise ValueError("free must be 1-D with an entry for each page of the pool, at least one")
    desc = _seq_pages(table, lengths, page, 0, free, free_count, free.numel())
    B = lengths.numel()
    if offsets.numel() != B + 1:
        raise ValueError(f"offsets must have {B + 1} entries, got {offsets.numel()}")
    n = _count(n, "n")
    leave = _opt(leave, "leave", (torch.bool, torch.uint8), (B,))
    dev = _device(table, lengths, free, free_count, offsets, leave)
    slots, refused = _out(slots, "slots", torch.int64, (n,), dev), _out(refused, "refused", torch.int32, (1,), dev)
    ws = _ws(lib().dlrm_seq_pages_update_workspace_size(B, n), dev, workspace)
    code = DLRM_INDEX_I32 if offsets.dtype is torch.int32 else DLRM_INDEX_I64
    _check(lib().dlrm_seq_pages_update(desc, _ptr(offsets), code, n, _ptr(leave), _ptr(slots), _ptr(refused), _ptr(ws), ws.numel(),
                                       _stream(dev)), "dlrm_seq_pages_update")
    return slots, refused


def dlrm_seq_pages_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor) -> None:
    """Rows of k and v [N, heads, d] to the rows slots [N] of k_pool and v_pool [rows, heads, d]; slots outside
    are passed over, no two others may be equal (C: dlrm_seq_pages_write)."""
    N, H, d, k_row, k_head = _head_rows(k, "k")
    Nv, _, _, v_row, v_head = _head_rows(v, "v", H, d)
    rows, _, _, kp_row, kp_head = _head_rows(k_pool, "k_pool", H, d)
    rows_v, _, _, vp_row, vp_head = _head_rows(v_pool, "v_pool", H, d)
    if Nv != N or rows_v != rows:
        raise ValueError(f"k and v must have the same rows, and their pools, got {N} and {Nv}, {rows} and {rows_v}")
    _is(slots, "slots", torch.int64, (N,))
    dev = _device(k, v, slots, k_pool, v_pool)
    _check(lib().dlrm_seq_pages_write(_ptr(k), k_row, k_head, _ptr(v), v_row, v_head, N, H, d, _ptr(slots), _ptr(k_pool), kp_row,
                                      kp_head, _ptr(v_pool), vp_row, vp_head, rows, _stream(dev)), "dlrm_seq_pages_write")


def dlrm_seq_attn_paged_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_offsets: torch.Tensor, table: torch.Tensor,
                            lengths: torch.Tensor, page: int, *, window: int = 0, sinks: int = 0, scale: Optional[float] = None,
                            bias: Optional[torch.Tensor] = None, bounds: Optional[Sequence[int]] = None,
                            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dlrm_seq_attn_fwd with keys and values in pages (C: dlrm_seq_attn_paged_fwd): k and v are the pool
    [pages * page, Hkv, d], table and lengths as dlrm_seq_pages_update left them; the queries are the users'
    last events."""
    _offsets(q_offsets, "q_offsets")
    B = q_offsets.numel() - 1
    a, edges, dev, shape, _ = _seq_attn(q, k, v, q_offsets, None, None, B, window, sinks, scale, bias, bounds)
    pg = _seq_pages(table, lengths, page, k.shape[0])
    if lengths.numel() != B:
        raise ValueError(f"table and lengths must be of the {B} users of q_offsets, got {lengths.numel()}")
    _device(q, table, lengths)
    out = _out_like(out, "out", q, shape, dev)
    _check(lib().dlrm_seq_attn_paged_fwd(a, pg, _ptr(out), _stream(dev)), "dlrm_seq_attn_paged_fwd")
    return out


def dlrm_seq_attn_paged_decode(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, lengths: torch.Tensor,
                               page: int, *, window: int = 0, sinks: int = 0, scale: Optional[float] = None,
                               bias: Optional[torch.Tensor] = None, bounds: Optional[Sequence[int]] = None,
                               max_kv_len: Optional[int] = None, out: Optional[torch.Tensor] = None,
                               workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dlrm_seq_attn_decode with keys and values in pages (C: dlrm_seq_attn_paged_decode): q [B, Hq, d] is one
    event of each user, the last of those that lengths counts; max_kv_len (None: what the table can hold) only
    chooses how far a history is split."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be [B, heads, d]")
    B = q.shape[0]
    a, edges, dev, shape, _ = _seq_attn(q, k, v, None, None, None, B, window, sinks, scale, bias, bounds)
    pg = _seq_pages(table, lengths, page, k.shape[0])
    if lengths.numel() != B:
        raise ValueError(f"table and lengths must be of q's {B} users, got {lengths.numel()}")
    _device(q, table, lengths)
    longest = table.shape[1] * int(page) if max_kv_len is None else int(max_kv_len)
    if longest < 0:
        raise ValueError(f"max_kv_len must not be negative, got {longest}")
    out = _out_like(out, "out", q, shape, dev)
    at, n, workspace = _ws_if(lib().dlrm_seq_attn_decode_workspace_size(B, shape[1], k.shape[1], shape[2], window, sinks, longest), dev, workspace)
    _check(lib().dlrm_seq_attn_paged_decode(a, pg, longest, _ptr(out), at, n, _stream(dev)), "dlrm_seq_attn_paged_decode")
    return out


# ---------------------------------------------------------------- linear attention with a decay (dlrm_seq_decay.h)

def _seq_decay(q, k, v, g, offsets, B: int, scale, max_len):
    """The checked description of a call: (its bytes, device, (N, Hq, d), Hkv)."""
    N, Hq, d, q_row, q_head = _head_rows(q, "q")
    Nk, Hkv, _, k_row, k_head = _head_rows(k, "k", None, d)
    Nv, _, _, v_row, v_head = _head_rows(v, "v", Hkv, d)
    if Nk != N or Nv != N:
        raise ValueError(f"q, k and v must have the same rows, got {N}, {Nk} and {Nv}")
    if Hq % Hkv:
        raise ValueError(f"q's heads must be a multiple of k's, got {Hq} and {Hkv}")
    if d % 8 or d > 128:
        raise ValueError(f"a head must have a multiple of 8 columns, at most 128, got {d}")
    if not isinstance(g, torch.Tensor) or g.dtype is not torch.float32:
        raise ValueError("g must be a tensor of torch.float32")
    if g.shape == (Hkv,) and g.is_contiguous():
        g_row = 0
    elif g.shape == (N, Hkv) and (Hkv == 1 or N == 0 or g.stride(1) == 1):
        g_row = g.stride(0) if N > 1 else Hkv
        if g_row < Hkv:
            raise ValueError("g must have rows of its own for each event; one decay for a head is [heads]")
    else:
        raise ValueError(f"g must be [{N}, {Hkv}] with packed rows, or [{Hkv}], got {tuple(g.shape)}")
    if max_len is not None and max_len < 0:
        raise ValueError(f"max_len must not be negative, got {max_len}")
    dev = _device(q, k, v, g, offsets)
    code = DLRM_INDEX_I32 if offsets is not None and offsets.dtype is torch.int32 else DLRM_INDEX_I64
    desc = _SEQ_DECAY.pack(B, N, Hq, Hkv, d, code, 0 if offsets is None else offsets.data_ptr(), N if max_len is None else int(max_len),
                           q.data_ptr(), k.data_ptr(), v.data_ptr(), q_row, q_head, k_row, k_head, v_row, v_head, g.data_ptr(), g_row,
                           d ** -0.5 if scale is None else float(scale))
    return desc, dev, (N, Hq, d), Hkv


def dlrm_seq_decay_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, offsets: torch.Tensor, *,
                       scale: Optional[float] = None, state: Optional[torch.Tensor] = None, want_state: bool = False,
                       max_len: Optional[int] = None, out: Optional[torch.Tensor] = None,
                       state_out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Linear attention with a decay over jagged sequences (C: dlrm_seq_decay_fwd): o [N, Hq, d] bf16, or with
    want_state or state_out (o, the states after each sequence).  q [N, Hq, d], k and v [N, Hkv, d]; g, the logarithms
    of the decays, <= 0: [N, Hkv], or [Hkv]; state [B, Hkv, d, d] fp32: what sequences begin with, None: zeros;
    state_out may be state.  max_len: the longest sequence, None: not known; it only chooses how a call works."""
    _offsets(offsets, "offsets")
    B = offsets.numel() - 1
    a, dev, shape, Hkv = _seq_decay(q, k, v, g, offsets, B, scale, max_len)
    ss = (B, Hkv, shape[2], shape[2])
    if state is not None:
        _is(state, "state", torch.float32, ss)
        _device(q, state)
    out = _out_like(out, "out", q, shape, dev)
    want_state = want_state or state_out is not None
    if want_state:
        state_out = _out(state_out, "state_out", torch.float32, ss, dev)
    at, n, workspace = _ws_if(lib().dlrm_seq_decay_fwd_workspace_size(a), dev, workspace)
    _check(lib().dlrm_seq_decay_fwd(a, _ptr(state), _ptr(state_out), _ptr(out), at, n, _stream(dev)), "dlrm_seq_decay_fwd")
    return (out, state_out) if want_state else out


def dlrm_seq_decay_bwd(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, offsets: torch.Tensor, *,
                       scale: Optional[float] = None, max_len: Optional[int] = None, want_dg: bool = True,
                       dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None, dv: Optional[torch.Tensor] = None,
                       dg: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """(dq, dk, dv, dg or None) of dlrm_seq_decay_fwd without states (C: dlrm_seq_decay_bwd); dg has g's shape, and is
    left out without want_dg, which takes 0.7 to 1 of the time (the most for heads above 64 cut into runs)."""
    _offsets(offsets, "offsets")
    B = offsets.numel() - 1
    a, dev, qs, Hkv = _seq_decay(q, k, v, g, offsets, B, scale, max_len)
    ks, bf = (qs[0], Hkv, qs[2]), torch.bfloat16
    _is(dout, "dout", bf, qs)
    _device(q, dout)
    dq, dk, dv = _out_like(dq, "dq", q, qs, dev), _out_like(dk, "dk", k, ks, dev), _out_like(dv, "dv", v, ks, dev)
    if dg is not None and not want_dg:
        raise ValueError("dg without want_dg")
    if want_dg:
        dg = _out_like(dg, "dg", g, g.shape, dev)
    ws = _ws(lib().dlrm_seq_decay_bwd_workspace_size(a), dev, workspace)
    _check(lib().dlrm_seq_decay_bwd(a, _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(ws), ws.numel(), _stream(dev)),
           "dlrm_seq_decay_bwd")
    return dq, dk, dv, dg


def dlrm_seq_decay_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, state: torch.Tensor, *,
                        scale: Optional[float] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One event of each of B sequences (C: dlrm_seq_decay_step): o [B, Hq, d] bf16; q [B, Hq, d], k and v
    [B, Hkv, d], g [B, Hkv] or [Hkv]; state [B, Hkv, d, d] fp32 is updated in place."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be [B, heads, d]")
    a, dev, shape, Hkv = _seq_decay(q, k, v, g, None, q.shape[0], scale, 1)
    _is(state, "state", torch.float32, (shape[0], Hkv, shape[2], shape[2]))
    _device(q, state)
    out = _out_like(out, "out", q, shape, dev)
    _check(lib().dlrm_seq_decay_step(a, _ptr(state), _ptr(out), _stream(dev)), "dlrm_seq_decay_step")
    return out


def dlrm_trace_enable(on: bool = True) -> None:
    """Bracket every library kernel launch with HIP events (C: dlrm_trace_enable)."""
    _check(lib().dlrm_trace_enable(1 if on else 0), "dlrm_trace_enable")


def dlrm_trace_read(max_entries: int = 64) -> dict:
    """{kernel name: (launches, total ms)} since the last read (C: dlrm_trace_read)."""
    names = ctypes.create_string_buffer(64 * max_entries)
    launches = (ctypes.c_int64 * max_entries)()
    ms = (ctypes.c_double * max_entries)()
    n = ctypes.c_int32(0)
    _check(lib().dlrm_trace_read(max_entries, names, launches, ms, ctypes.byref(n)), "dlrm_trace_read")
    out = {}
    for i in range(n.value):
        name = names.raw[64 * i:64 * (i + 1)].split(b"\0", 1)[0].decode()
        out[name] = (int(launches[i]), float(ms[i]))
    return out
