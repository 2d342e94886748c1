"""Python binding of libdsa.so, the B200 (sm_100a) DeepSeek Sparse Attention hot path.

Argument marshalling only: every stage runs in the library's CUDA kernels on
the caller's current torch stream; torch provides device memory and streams.
There is no CPU fallback -- if the shared library is missing, importing the
binding's entry points raises.

    import long_context_sparse_lightning_b200 as dsa
    batch = dsa.Batch(cu_q, kv_len, kv_start, max_q_per_seq, max_kv_len, total_keys)
    ws = dsa.workspace(dsa.OP_FORWARD, batch, k_sel=2048, n_heads=128)
    dsa.forward(batch, q8, q_scale, w, k8, k_scale, 2048, q, kv, sm_scale, idx, out, lse, ws)
"""

from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdsa.so")

OP_INDEXER, OP_TOPK, OP_SPARSE_MLA, OP_FORWARD, OP_CACHE_WRITE, OP_INDEXER_TOPK = 0, 1, 2, 3, 4, 5
OP_DENSE_MLA, OP_PREFIX_MLA, OP_EXPANDED_MLA, OP_PAGE_TABLES = 6, 7, 8, 9
INDEX_HEADS, INDEX_DIM, LATENT_DIM, VALUE_DIM, MAX_K_SEL = 64, 128, 576, 512, 2048

STATUS = {
    0: "DSA_OK",
    1: "DSA_ERR_INVALID_ARG",
    2: "DSA_ERR_UNSUPPORTED",
    3: "DSA_ERR_CUDA",
    4: "DSA_ERR_WORKSPACE",
    5: "DSA_ERR_DEVICE_TIMEOUT",
    6: "DSA_ERR_DEVICE_BOUNDS",
}

# every entry point declared in include/dsa.h
EXPORTS = [
    "dsa_workspace_size",
    "dsa_indexer_scores",
    "dsa_topk",
    "dsa_indexer_topk",
    "dsa_topk_candidates",
    "dsa_topk_merge",
    "dsa_sparse_mla",
    "dsa_forward",
    "dsa_sparse_mla_no_alloc",
    "dsa_check_device_error",
    "dsa_status_string",
    "dsa_version",
    "dsa_forward_launches",
    "dsa_quantize_fp8",
    "dsa_indexer_prep",
    "dsa_cache_write",
    "dsa_dense_mla",
    "dsa_prefix_mla",
    "dsa_expanded_mla",
    "dsa_page_tables",
]


class DSAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({_lib().dsa_status_string(status).decode()})")


class _BatchC(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int32),
        ("total_q", ctypes.c_int32),
        ("max_q_per_seq", ctypes.c_int32),
        ("max_kv_len", ctypes.c_int32),
        ("total_keys", ctypes.c_int64),
        ("cu_q", ctypes.c_void_p),
        ("kv_len", ctypes.c_void_p),
        ("kv_start", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p),
        ("page_size", ctypes.c_int32),
        ("blocks_per_seq", ctypes.c_int32),
    ]


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m long_context_sparse_lightning_b200.build` "
                "(there is no fallback implementation)")
        lib = ctypes.CDLL(LIB_PATH)
        P, I32, I64, SZ, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
        BP = ctypes.POINTER(_BatchC)
        lib.dsa_workspace_size.argtypes = [ctypes.c_int, BP, I32, I32]
        lib.dsa_workspace_size.restype = SZ
        lib.dsa_indexer_scores.argtypes = [BP, P, P, P, P, P, P, I64, P, SZ, P]
        lib.dsa_indexer_scores.restype = ctypes.c_int
        lib.dsa_topk.argtypes = [BP, P, I64, I32, P, P, SZ, P]
        lib.dsa_topk.restype = ctypes.c_int
        lib.dsa_indexer_topk.argtypes = [BP, P, P, P, P, P, I32, P, P, SZ, P]
        lib.dsa_indexer_topk.restype = ctypes.c_int
        lib.dsa_topk_candidates.argtypes = [BP, P, I64, I32, P, P, P, P, SZ, P]
        lib.dsa_topk_candidates.restype = ctypes.c_int
        lib.dsa_topk_merge.argtypes = [I32, I32, I32, P, P, P, P]
        lib.dsa_topk_merge.restype = ctypes.c_int
        lib.dsa_sparse_mla.argtypes = [BP, P, I32, P, P, I32, F, P, P, P, SZ, P]
        lib.dsa_sparse_mla.restype = ctypes.c_int
        lib.dsa_forward.argtypes = [BP, P, P, P, P, P, I32, P, I32, P, F, P, P, P, P, SZ, P]
        lib.dsa_forward.restype = ctypes.c_int
        lib.dsa_sparse_mla_no_alloc.argtypes = [BP, P, I32, P, P, I32, F, P, P, P]
        lib.dsa_sparse_mla_no_alloc.restype = ctypes.c_int
        lib.dsa_check_device_error.argtypes = [P, P, ctypes.POINTER(ctypes.c_uint32), ctypes.POINTER(ctypes.c_uint32)]
        lib.dsa_check_device_error.restype = ctypes.c_int
        lib.dsa_status_string.argtypes = [ctypes.c_int]
        lib.dsa_status_string.restype = ctypes.c_char_p
        lib.dsa_version.argtypes = []
        lib.dsa_version.restype = I32
        lib.dsa_forward_launches.argtypes = [BP, I32, I32]
        lib.dsa_forward_launches.restype = I32
        lib.dsa_quantize_fp8.argtypes = [P, I64, P, P, P]
        lib.dsa_quantize_fp8.restype = ctypes.c_int
        lib.dsa_indexer_prep.argtypes = [P, I64, I32, P, P, P, I32, P, P, P, SZ, P]
        lib.dsa_indexer_prep.restype = ctypes.c_int
        lib.dsa_cache_write.argtypes = [BP, P, P, P, P, P, P, SZ, P]
        lib.dsa_cache_write.restype = ctypes.c_int
        lib.dsa_dense_mla.argtypes = [BP, P, I32, P, F, P, P, P, SZ, P]
        lib.dsa_dense_mla.restype = ctypes.c_int
        lib.dsa_prefix_mla.argtypes = [BP, I32, P, I32, P, F, P, P, P, SZ, P]
        lib.dsa_prefix_mla.restype = ctypes.c_int
        lib.dsa_expanded_mla.argtypes = [BP, P, I32, P, P, I64, F, P, P, P, SZ, P]
        lib.dsa_expanded_mla.restype = ctypes.c_int
        lib.dsa_page_tables.argtypes = [I32, P, P, P, I32, I32, P, I32, I32, P, P, P, P, P, P, SZ, P]
        lib.dsa_page_tables.restype = ctypes.c_int
        _LIB = lib
    return _LIB


def library():
    """The loaded ctypes library (raises if it was not built)."""
    return _lib()


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


# the current stream's handle of a device without building a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(fn, where, device, stream, *args):
    """fn(*args, stream)'s status on device number `device`, on its current stream unless one is given."""
    if device < 0:
        raise ValueError(f"{where}: tensors on a CUDA device")
    handle = _raw_stream(device) if stream is None else stream.cuda_stream
    if device == torch.cuda.current_device():
        return fn(*args, handle)
    with torch.cuda.device(device):
        return fn(*args, handle)


def _launch(fn, where, device, stream, *args):
    status = _call(fn, where, device, stream, *args)
    if status != 0:
        raise DSAError(status, where)


def _one_device(where, first, *others):
    device = first.get_device()
    for t in others:
        if t is not None and t.get_device() != device:
            raise ValueError(f"{where}: tensors on one device")
    return device


def _check(status: int, where: str):
    if status != 0:
        raise DSAError(status, where)


class Batch:
    """Ragged batch: device arrays cu_q [B+1] int32, kv_len [B] int32, kv_start [B] int64,
    plus the host-side sizes that shape the launch grids.

    Paged caches: pass ``block_table`` (int32 [B, blocks_per_seq] page ids) and
    ``page_size`` (a multiple of 64); ``kv_start`` may then be None and
    ``total_keys`` is the pool's row count."""

    def __init__(self, cu_q: torch.Tensor, kv_len: torch.Tensor, kv_start: Optional[torch.Tensor], total_q: int,
                 max_q_per_seq: int, max_kv_len: int, total_keys: int, block_table: Optional[torch.Tensor] = None,
                 page_size: int = 0):
        if cu_q.dtype != torch.int32 or kv_len.dtype != torch.int32 or \
                (kv_start is not None and kv_start.dtype != torch.int64):
            raise TypeError("cu_q/kv_len must be int32 and kv_start int64")
        if block_table is not None and (block_table.dtype != torch.int32 or block_table.dim() != 2
                                        or not block_table.is_contiguous()):
            raise TypeError("block_table must be a contiguous int32 [num_seqs, blocks_per_seq] tensor")
        # kernels read these by address: all of num_seqs entries, on the device that the calls check cu_q to be on
        for t, n in ((cu_q, kv_len.shape[0] + 1), (kv_len, 0), (kv_start, kv_len.shape[0]),
                     (block_table, kv_len.shape[0] if block_table is not None else 0)):
            if t is not None and (t.device != cu_q.device or not t.is_contiguous() or t.shape[0] < n):
                raise ValueError("Batch: contiguous cu_q [num_seqs + 1], kv_len [num_seqs], kv_start [num_seqs] and "
                                 "block_table [num_seqs, blocks_per_seq] on one device")
        self.cu_q, self.kv_len, self.kv_start, self.block_table = cu_q, kv_len, kv_start, block_table
        self.num_seqs = int(kv_len.shape[0])
        self.total_q = int(total_q)
        self.c = _BatchC()
        self.c.num_seqs = self.num_seqs
        self.c.total_q = self.total_q
        self.c.max_q_per_seq = int(max_q_per_seq)
        self.c.max_kv_len = int(max_kv_len)
        self.c.total_keys = int(total_keys)
        self.c.cu_q = cu_q.data_ptr()
        self.c.kv_len = kv_len.data_ptr()
        self.c.kv_start = kv_start.data_ptr() if kv_start is not None else None
        if block_table is not None:
            self.c.block_table = block_table.data_ptr()
            self.c.page_size = int(page_size)
            self.c.blocks_per_seq = int(block_table.shape[1])

    @staticmethod
    def from_host(cu_q, kv_len, kv_start, device="cuda", total_keys: Optional[int] = None):
        """Build from host sequences / numpy arrays; copies the arrays to `device`."""
        import numpy as np
        cu = np.asarray(cu_q, dtype=np.int32)
        kl = np.asarray(kv_len, dtype=np.int32)
        ks = np.asarray(kv_start, dtype=np.int64)
        q_len = np.diff(cu)
        if total_keys is None:
            total_keys = int((ks + kl).max()) if kl.size else 0
        return Batch(torch.from_numpy(cu).to(device), torch.from_numpy(kl).to(device),
                     torch.from_numpy(ks).to(device), int(cu[-1]), int(q_len.max()) if q_len.size else 0,
                     int(kl.max()) if kl.size else 0, int(total_keys))

    @staticmethod
    def from_requests(q_len: torch.Tensor, kv_before: torch.Tensor, free_pages: torch.Tensor, page_size: int,
                      block_table: torch.Tensor, ws: torch.Tensor, total_q: int, max_q_per_seq: int, max_kv_len: int,
                      total_keys: int, stream=None):
        """A paged step's batch from its requests' lengths, on the device (page_tables): each request has
        kv_before[b] positions and takes q_len[b] new tokens, whose pages come from free_pages in order and are
        entered in block_table.  The host sizes may be bounds, as for a captured step: total_q rows are the
        padded count.  Returns the batch, the rows' positions (indexer_prep's pos) and cache rows, and the
        number of pages taken (int32 [1]).  These tensors are allocated on the stream that fills them (`stream`, or the
        current one): another stream waits for it before it reads them, and calls record_stream on what it may still be
        reading when the last reference goes."""
        with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
            device = q_len.device
            cu_q = torch.empty(q_len.numel() + 1, dtype=torch.int32, device=device)
            kv_len = torch.empty(q_len.numel(), dtype=torch.int32, device=device)
            pos = torch.empty(total_q, dtype=torch.int32, device=device)
            slots = torch.empty(total_q, dtype=torch.int64, device=device)
            used = torch.empty(1, dtype=torch.int32, device=device)
        page_tables(q_len, kv_before, free_pages, page_size, block_table, cu_q, kv_len, pos, slots, used, ws, stream)
        batch = Batch(cu_q, kv_len, None, total_q, max_q_per_seq, max_kv_len, total_keys, block_table=block_table,
                      page_size=page_size)
        return batch, pos, slots, used

    @property
    def ref(self):
        return ctypes.byref(self.c)


def workspace_size(op: int, batch: Batch, k_sel: int = MAX_K_SEL, n_heads: int = 128) -> int:
    return int(_lib().dsa_workspace_size(op, batch.ref, k_sel, n_heads))


def workspace(op: int, batch: Batch, k_sel: int = MAX_K_SEL, n_heads: int = 128, device="cuda") -> torch.Tensor:
    """A zeroed device workspace (the zero error word is part of the contract)."""
    n = workspace_size(op, batch, k_sel, n_heads)
    if n == 0:
        raise DSAError(1, "dsa_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def indexer_scores(batch: Batch, q_fp8, q_scale, w, k_fp8, k_scale, scores, ws, stream=None):
    _check(_lib().dsa_indexer_scores(batch.ref, _ptr(q_fp8), _ptr(q_scale), _ptr(w), _ptr(k_fp8), _ptr(k_scale),
                                     _ptr(scores), scores.shape[-1], _ptr(ws), ws.numel(), _stream(stream)),
           "dsa_indexer_scores")


def topk(batch: Batch, scores, k_sel: int, idx, ws, stream=None):
    _check(_lib().dsa_topk(batch.ref, _ptr(scores), scores.shape[-1], k_sel, _ptr(idx), _ptr(ws), ws.numel(),
                           _stream(stream)), "dsa_topk")


def indexer_topk(batch: Batch, q_fp8, q_scale, w, k_fp8, k_scale, k_sel: int, idx, ws, stream=None):
    """Indexer scores and top-k in one call (fused on chip for decode batches)."""
    _check(_lib().dsa_indexer_topk(batch.ref, _ptr(q_fp8), _ptr(q_scale), _ptr(w), _ptr(k_fp8), _ptr(k_scale), k_sel,
                                   _ptr(idx), _ptr(ws), ws.numel(), _stream(stream)), "dsa_indexer_topk")


def topk_candidates(batch: Batch, scores, k_sel: int, cand_pos, cand_val, ws, pos_offset=None, stream=None):
    """One key shard's top k as global positions (+ pos_offset per sequence) and their scores."""
    _check(_lib().dsa_topk_candidates(batch.ref, _ptr(scores), scores.shape[-1], k_sel, _ptr(pos_offset),
                                      _ptr(cand_pos), _ptr(cand_val), _ptr(ws), ws.numel(), _stream(stream)),
           "dsa_topk_candidates")


def topk_merge(cand_pos, cand_val, k_sel: int, idx, stream=None):
    """Top k per row over [n_rows, n_src, k_sel] candidate lists (shards in position order)."""
    if cand_pos.dim() != 3 or cand_pos.shape != cand_val.shape or cand_pos.shape[2] != k_sel:
        raise ValueError("topk_merge: cand_pos / cand_val [n_rows, n_src, k_sel]")
    _check(_lib().dsa_topk_merge(int(cand_pos.shape[0]), int(cand_pos.shape[1]), k_sel, _ptr(cand_pos),
                                 _ptr(cand_val), _ptr(idx), _stream(stream)), "dsa_topk_merge")


def sparse_mla(batch: Batch, q, kv, idx, k_sel: int, sm_scale: float, out, lse, ws, stream=None):
    n_heads = int(q.shape[1])
    _check(_lib().dsa_sparse_mla(batch.ref, _ptr(q), n_heads, _ptr(kv), _ptr(idx), k_sel, float(sm_scale), _ptr(out),
                                 _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)), "dsa_sparse_mla")


def forward(batch: Batch, q_fp8, q_scale, w, k_fp8, k_scale, k_sel: int, q, kv, sm_scale: float, idx, out, lse, ws,
            stream=None):
    n_heads = int(q.shape[1])
    _check(_lib().dsa_forward(batch.ref, _ptr(q_fp8), _ptr(q_scale), _ptr(w), _ptr(k_fp8), _ptr(k_scale), k_sel,
                              _ptr(q), n_heads, _ptr(kv), float(sm_scale), _ptr(idx), _ptr(out), _ptr(lse), _ptr(ws),
                              ws.numel(), _stream(stream)), "dsa_forward")


def _check_mla(where, batch, q, q_dim, out, out_dim, lse):
    n, h = batch.total_q, q.shape[1] if q.dim() == 3 else 0
    if q.dtype != torch.bfloat16 or q.shape != (n, h, q_dim) or out.dtype != torch.bfloat16 \
            or out.shape != (n, h, out_dim) or (lse is not None and (lse.dtype != torch.float32 or lse.shape != (n, h))):
        raise ValueError(f"{where}: q bf16 [total_q, heads, {q_dim}], out bf16 [total_q, heads, {out_dim}], "
                         "lse fp32 [total_q, heads] or None")
    return h


def _check_cache(where, batch, kv):
    if kv.dtype != torch.bfloat16 or kv.dim() != 2 or kv.shape[1] != LATENT_DIM or kv.shape[0] < batch.c.total_keys:
        raise ValueError(f"{where}: kv bf16 [total_keys, {LATENT_DIM}]")


def dense_mla(batch: Batch, q, kv, sm_scale: float, out, lse, ws, stream=None):
    """Latent attention over every position a token may see (absorbed form): q [total_q, heads, 576],
    kv [total_keys, 576] -> out [total_q, heads, 512], lse (natural log) or None; ws of OP_DENSE_MLA."""
    n_heads = _check_mla("dense_mla", batch, q, LATENT_DIM, out, VALUE_DIM, lse)
    _check_cache("dense_mla", batch, kv)
    dev = _one_device("dense_mla", q, kv, out, lse, ws, batch.cu_q)
    _launch(_lib().dsa_dense_mla, "dsa_dense_mla", dev, stream, batch.ref, _ptr(q), n_heads, _ptr(kv), sm_scale,
            _ptr(out), _ptr(lse), _ptr(ws), ws.numel())


def prefix_mla(batch: Batch, prefix_len: int, q, kv, sm_scale: float, out, lse, ws, stream=None):
    """dense_mla of a paged batch whose sequences share their first prefix_len positions (those of block-table
    row 0), which are read and multiplied once for all; ws of OP_PREFIX_MLA."""
    n_heads = _check_mla("prefix_mla", batch, q, LATENT_DIM, out, VALUE_DIM, lse)
    _check_cache("prefix_mla", batch, kv)
    dev = _one_device("prefix_mla", q, kv, out, lse, ws, batch.cu_q)
    _launch(_lib().dsa_prefix_mla, "dsa_prefix_mla", dev, stream, batch.ref, prefix_len, _ptr(q), n_heads, _ptr(kv),
            sm_scale, _ptr(out), _ptr(lse), _ptr(ws), ws.numel())


def expanded_mla(batch: Batch, q, kv_up, rope, sm_scale: float, out, lse, ws, stream=None):
    """Latent attention in the expanded form: q [total_q, heads, 192], kv_up [total_keys, heads, 256] (128 key dims, then
    128 value dims), rope [total_keys, 64] (rows may lie apart, e.g. latent[:, 512:]) -> out [total_q, heads, 128],
    lse or None; flat caches; ws of OP_EXPANDED_MLA."""
    n_heads = _check_mla("expanded_mla", batch, q, 192, out, 128, lse)
    keys = batch.c.total_keys
    if kv_up.dtype != torch.bfloat16 or kv_up.dim() != 3 or kv_up.shape[1:] != (n_heads, 256) \
            or kv_up.shape[0] < keys or rope.dtype != torch.bfloat16 or rope.dim() != 2 \
            or rope.shape[1] != 64 or rope.shape[0] < keys or rope.stride(1) != 1:
        raise ValueError("expanded_mla: kv_up bf16 [total_keys, heads, 256], rope bf16 [total_keys, 64]")
    # a single row has no stride of its own
    stride = rope.stride(0) if rope.shape[0] > 1 else 64
    dev = _one_device("expanded_mla", q, kv_up, rope, out, lse, ws, batch.cu_q)
    _launch(_lib().dsa_expanded_mla, "dsa_expanded_mla", dev, stream, batch.ref, _ptr(q), n_heads, _ptr(kv_up),
            rope.data_ptr(), stride, sm_scale, _ptr(out), _ptr(lse), _ptr(ws), ws.numel())


def page_tables(q_len, kv_before, free_pages, page_size: int, block_table, cu_q, kv_len, pos, slots, pages_used, ws,
                stream=None):
    """Block tables, offsets, positions and cache slots of a step's new tokens from the requests' lengths:
    q_len, kv_before int32 [B], free_pages int32 -> block_table int32 [B, blocks] (new pages written behind the
    held ones), cu_q int32 [B + 1], kv_len int32 [B], pos int32 and slots int64 [max_tokens], pages_used int32 [1]."""
    n, tokens, i32, dev = q_len.numel(), pos.numel(), torch.int32, q_len.get_device()
    for t in (q_len, kv_before, free_pages, block_table, cu_q, kv_len, pos, pages_used):
        if t.dtype is not i32 or t.get_device() != dev or not t.is_contiguous():
            raise ValueError("page_tables: contiguous int32 tensors on one device (int64 slots)")
    blocks = block_table.shape[1] if block_table.dim() == 2 else 0
    if slots.dtype is not torch.int64 or slots.get_device() != dev or not slots.is_contiguous() \
            or ws.get_device() != dev or kv_before.numel() != n or block_table.numel() != n * blocks \
            or cu_q.numel() != n + 1 or kv_len.numel() != n or slots.numel() != tokens or pages_used.numel() != 1:
        raise ValueError("page_tables: int32 q_len, kv_before, kv_len [B], cu_q [B + 1], block_table [B, blocks], "
                         "free_pages, pos [max_tokens], pages_used [1]; int64 slots [max_tokens]")
    _launch(_lib().dsa_page_tables, "dsa_page_tables", dev, stream, n, q_len.data_ptr(), kv_before.data_ptr(),
            free_pages.data_ptr(), free_pages.numel(), page_size, block_table.data_ptr(), blocks, tokens,
            cu_q.data_ptr(), kv_len.data_ptr(), pos.data_ptr(), slots.data_ptr(), pages_used.data_ptr(), ws.data_ptr(),
            ws.numel())


def quantize_fp8(x, codes, scales, stream=None):
    """Per-128 FP8 e4m3 quantisation: x bf16 [..., 128] -> codes uint8 [..., 128], scales fp32 [...]."""
    if x.dtype != torch.bfloat16 or x.shape[-1] != INDEX_DIM or codes.dtype != torch.uint8 \
            or codes.numel() != x.numel() or scales.dtype != torch.float32 or scales.numel() * INDEX_DIM != x.numel():
        raise ValueError("quantize_fp8: x bf16 [..., 128], codes uint8 of the same size, scales fp32 [...]")
    n_vec = x.numel() // INDEX_DIM
    _check(_lib().dsa_quantize_fp8(_ptr(x), n_vec, _ptr(codes), _ptr(scales), _stream(stream)), "dsa_quantize_fp8")


def indexer_prep(x, pos, rope_cos, rope_sin, codes, scales, ws, vecs_per_pos: int, stream=None):
    """Non-interleaved RoPE on dims 0..63, normalised Walsh-Hadamard, per-128 FP8: x bf16 [..., 128]."""
    if x.dtype != torch.bfloat16 or x.shape[-1] != INDEX_DIM or codes.dtype != torch.uint8 \
            or codes.numel() != x.numel() or scales.dtype != torch.float32 or scales.numel() * INDEX_DIM != x.numel() \
            or pos.dtype != torch.int32 or rope_cos.dtype != torch.float32 or rope_sin.shape != rope_cos.shape \
            or rope_cos.shape[-1] != 32:
        raise ValueError("indexer_prep: x bf16 [..., 128], pos int32, rope tables fp32 [n_pos, 32]")
    n_vec = x.numel() // INDEX_DIM
    _check(_lib().dsa_indexer_prep(_ptr(x), n_vec, int(vecs_per_pos), _ptr(pos), _ptr(rope_cos), _ptr(rope_sin),
                                   int(rope_cos.shape[0]), _ptr(codes), _ptr(scales), _ptr(ws), ws.numel(),
                                   _stream(stream)), "dsa_indexer_prep")


def cache_write(batch: Batch, k, latent, k_cache, k_scale, latent_cache, ws, stream=None):
    """New tokens' keys (FP8 + scale) and latent rows into the flat caches at their positions."""
    _check(_lib().dsa_cache_write(batch.ref, _ptr(k), _ptr(latent), _ptr(k_cache), _ptr(k_scale), _ptr(latent_cache),
                                  _ptr(ws), ws.numel(), _stream(stream)), "dsa_cache_write")


def check_device_error(ws, stream=None):
    """Synchronise (the current stream of the workspace's device, or `stream`), read and clear the workspace's device
    error word; raise if set."""
    site = ctypes.c_uint32(0)
    info = ctypes.c_uint32(0)
    st = _call(lambda p, handle: _lib().dsa_check_device_error(p, handle, ctypes.byref(site), ctypes.byref(info)),
               "check_device_error", ws.get_device(), stream, _ptr(ws))
    if st != 0:
        err = DSAError(st, f"device error (site {site.value}, info {info.value})")
        err.site, err.info = site.value, info.value
        raise err


def forward_launches(batch: Batch, k_sel: int, n_heads: int) -> int:
    """Kernel launches one dsa_forward call makes for this batch (host only)."""
    return int(_lib().dsa_forward_launches(batch.ref, k_sel, n_heads))


def version() -> int:
    return int(_lib().dsa_version())
