"""The dense latent attentions and the page tables without a GPU: workspace sizes
and refusals, all before any launch."""

import ctypes

import pytest
import torch

import long_context_sparse_lightning_b200 as dsa
from long_context_sparse_lightning_b200 import _BatchC

P = ctypes.c_void_p
FAKE = P(0x10000)                   # aligned, never dereferenced
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4


def host_batch(B=2, total_q=10, max_q=6, max_kv=100, total_keys=192, page=0, blocks=2):
    c = _BatchC()
    c.num_seqs, c.total_q, c.max_q_per_seq, c.max_kv_len, c.total_keys = B, total_q, max_q, max_kv, total_keys
    c.cu_q = c.kv_len = 0x1000
    if page:
        c.block_table, c.page_size, c.blocks_per_seq = 0x2000, page, blocks
    else:
        c.kv_start = 0x1000
    return c


def test_workspace_sizes():
    lib = dsa.library()
    size = lambda op, c, h=16: lib.dsa_workspace_size(op, ctypes.byref(c), 0, h)  # noqa: E731
    flat, paged = host_batch(), host_batch(page=64)
    # records (16 bytes a row), 2 x 148 slots of the item's rows: 16 or 32 (a CTA each), 148 of 128 (a pair each)
    one = host_batch(total_q=2, max_q=1)
    assert 296 * 16 * 513 * 4 <= size(dsa.OP_DENSE_MLA, one) <= 296 * 16 * 513 * 4 + 4096
    assert 296 * 32 * 513 * 4 <= size(dsa.OP_DENSE_MLA, host_batch(total_q=4, max_q=2)) <= 296 * 32 * 513 * 4 + 4096
    assert 148 * 128 * 513 * 4 <= size(dsa.OP_DENSE_MLA, flat) <= 148 * 128 * 513 * 4 + 8192
    # the shared prefix adds two whole results per row
    extra = size(dsa.OP_PREFIX_MLA, paged) - size(dsa.OP_DENSE_MLA, paged)
    assert 2 * 160 * 513 * 4 <= extra <= 2 * 160 * 513 * 4 + 4096
    assert size(dsa.OP_PREFIX_MLA, flat) == 0                     # flat caches share nothing
    assert size(dsa.OP_PAGE_TABLES, flat) == 256
    # expanded: only the header, unless few row tiles see a long context
    assert size(dsa.OP_EXPANDED_MLA, flat) == 256
    long = host_batch(B=1, total_q=10, max_q=10, max_kv=8192, total_keys=8192)
    splits = 9                                                    # 148 CTAs / 16
    assert 256 + splits * 160 * 129 * 4 <= size(dsa.OP_EXPANDED_MLA, long) <= 1024 + splits * 160 * 129 * 4
    assert size(dsa.OP_EXPANDED_MLA, paged) == 0
    for op in (dsa.OP_DENSE_MLA, dsa.OP_PREFIX_MLA, dsa.OP_EXPANDED_MLA):
        assert size(op, paged, 0) == 0 and size(op, paged, 129) == 0
        assert size(op, host_batch(B=0, page=64)) == 0


def dense(c, q=FAKE, heads=16, kv=FAKE, scale=0.07, out=FAKE, lse=None, ws=FAKE, n=1 << 40):
    return dsa.library().dsa_dense_mla(ctypes.byref(c), q, heads, kv, scale, out, lse, ws, n, None)


def prefix(c, length, heads=16, ws=FAKE, n=1 << 40):
    return dsa.library().dsa_prefix_mla(ctypes.byref(c), length, FAKE, heads, FAKE, 0.07, FAKE, None, ws, n, None)


def expanded(c, q=FAKE, heads=16, up=FAKE, rope=FAKE, stride=576, scale=0.07, out=FAKE, lse=None, ws=FAKE, n=1 << 40):
    return dsa.library().dsa_expanded_mla(ctypes.byref(c), q, heads, up, rope, stride, scale, out, lse, ws, n, None)


def test_dense_refusals():
    c = host_batch()
    assert dense(c, q=None) == INVALID and dense(c, kv=None) == INVALID and dense(c, out=None) == INVALID
    assert dense(c, q=P(0x10008)) == INVALID and dense(c, kv=P(0x10002)) == INVALID and dense(c, out=P(0x10004)) == INVALID
    assert dense(c, lse=P(0x10002)) == INVALID
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert dense(c, scale=scale) == INVALID
    assert dense(c, heads=0) == UNSUPPORTED and dense(c, heads=129) == UNSUPPORTED
    assert dense(c, ws=None) == INVALID and dense(c, ws=P(0x10008)) == INVALID
    need = dsa.library().dsa_workspace_size(dsa.OP_DENSE_MLA, ctypes.byref(c), 0, 16)
    assert dense(c, n=need - 1) == WORKSPACE
    assert dense(host_batch(B=0)) == INVALID and dense(host_batch(max_q=11)) == INVALID
    assert dense(host_batch(page=96)) == INVALID and dense(host_batch(page=64, blocks=1)) == INVALID
    # nothing to do, also with empty tensors
    assert dense(host_batch(total_q=0, max_q=0)) == 0 and dense(host_batch(total_q=0, max_q=0), q=None, out=None) == 0


def test_prefix_refusals():
    c = host_batch(page=64)
    assert prefix(c, -1) == INVALID and prefix(c, 101) == INVALID
    assert prefix(host_batch(), 10) == UNSUPPORTED                # flat caches
    need = dsa.library().dsa_workspace_size(dsa.OP_PREFIX_MLA, ctypes.byref(c), 0, 16)
    assert prefix(c, 10, n=need - 1) == WORKSPACE
    assert prefix(host_batch(total_q=0, max_q=0, page=64), 10) == 0


def test_expanded_refusals():
    c = host_batch()
    for bad in (dict(q=None), dict(up=None), dict(rope=None), dict(out=None), dict(q=P(0x10008)), dict(up=P(0x10002)),
                dict(rope=P(0x10008)), dict(out=P(0x10004)), dict(lse=P(0x10001)), dict(stride=63), dict(stride=68),
                dict(scale=0.0), dict(ws=None), dict(stride=1 << 31)):
        assert expanded(c, **bad) == INVALID, bad
    assert expanded(c, heads=0) == UNSUPPORTED and expanded(c, heads=129) == UNSUPPORTED
    assert expanded(host_batch(page=64)) == UNSUPPORTED
    assert expanded(c, n=255) == WORKSPACE
    long = host_batch(B=1, total_q=10, max_q=10, max_kv=8192, total_keys=8192)
    assert expanded(long, n=256) == WORKSPACE                     # the split's partial results
    none = host_batch(total_q=0, max_q=0)
    assert expanded(none) == 0 and expanded(none, q=None, up=None, rope=None, out=None) == 0


def tables(n=2, q=0x100000, before=0x200000, free=0x300000, n_free=4, page=64, table=0x400000, blocks=3, tokens=8,
           cu=0x500000, kv=0x600000, pos=0x700000, slots=0x800000, used=0x900000, ws=0xA00000, nbytes=256):
    return dsa.library().dsa_page_tables(n, q, before, free, n_free, page, table, blocks, tokens, cu, kv, pos, slots, used,
                                         ws, nbytes, None)


def test_page_tables_refusals():
    for bad in (dict(n=0), dict(n=65536), dict(n_free=-1), dict(tokens=-1), dict(page=0), dict(page=96), dict(blocks=0),
                dict(q=None), dict(before=None), dict(free=None), dict(table=None), dict(cu=None), dict(kv=None),
                dict(pos=None), dict(slots=None), dict(used=None), dict(ws=None),
                dict(q=0x100002), dict(slots=0x800004), dict(used=0x900001),
                dict(kv=0x200000),                                # kv_len written over kv_before
                dict(cu=0x600000 - 8),                            # cu_q's last entry is kv_len's first
                dict(table=0x300000 + 8),                         # the table over the free pages
                dict(pos=0x800000 + 60)):                         # pos inside slots
        assert tables(**bad) == INVALID, bad
    assert tables(blocks=1 << 25) == UNSUPPORTED                  # 2^31 positions
    assert tables(nbytes=255) == WORKSPACE


def test_bindings_check_shapes_and_devices():
    c = _BatchC()
    cu, kv, start = torch.tensor([0, 2], dtype=torch.int32), torch.tensor([5], dtype=torch.int32), torch.tensor([0])
    b = dsa.Batch(cu, kv, start, 2, 2, 5, 5)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    ws, lse = torch.zeros(256, dtype=torch.uint8), torch.zeros((2, 4))
    with pytest.raises(ValueError):
        dsa.dense_mla(b, bf(2, 4, 512), bf(5, 576), 0.1, bf(2, 4, 512), lse, ws)
    with pytest.raises(ValueError):
        dsa.dense_mla(b, bf(2, 4, 576).float(), bf(5, 576), 0.1, bf(2, 4, 512), lse, ws)
    with pytest.raises(ValueError):
        dsa.dense_mla(b, bf(2, 4, 576), bf(4, 576), 0.1, bf(2, 4, 512), lse, ws)          # fewer rows than total_keys
    with pytest.raises(ValueError):
        dsa.dense_mla(b, bf(2, 4, 576), bf(5, 576), 0.1, bf(3, 4, 512), lse, ws)
    with pytest.raises(ValueError):
        dsa.dense_mla(b, bf(2, 4, 576), bf(5, 576), 0.1, bf(2, 4, 512), lse.double(), ws)
    with pytest.raises(ValueError):
        dsa.prefix_mla(b, 1, bf(2, 4, 576), bf(5, 512), 0.1, bf(2, 4, 512), lse, ws)
    with pytest.raises(ValueError):
        dsa.expanded_mla(b, bf(2, 4, 192), bf(5, 4, 128), bf(5, 64), 0.1, bf(2, 4, 128), lse, ws)
    with pytest.raises(ValueError):
        dsa.expanded_mla(b, bf(2, 4, 192), bf(5, 4, 256), bf(5, 128)[:, ::2], 0.1, bf(2, 4, 128), lse, ws)
    # host tensors never reach the library
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dense_mla(b, bf(2, 4, 576), bf(5, 576), 0.1, bf(2, 4, 512), lse, ws)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.expanded_mla(b, bf(2, 4, 192), bf(5, 4, 256), bf(5, 576)[:, 512:], 0.1, bf(2, 4, 128), lse, ws)
    i = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    args = [i(1), i(0), i(3, 4), 64, i(0, 0).view(1, 2), i(0, 0), i(0), i(0), torch.zeros(1, dtype=torch.int64), i(0), ws]
    with pytest.raises(ValueError, match="CUDA"):
        dsa.page_tables(*args)
    for at, bad in ((0, torch.zeros(1)), (5, i(0)), (8, i(0)), (4, i(0, 0)), (7, i(0, 0))):
        with pytest.raises(ValueError):
            dsa.page_tables(*(args[:at] + [bad] + args[at + 1:]))
    assert c is not None


def test_another_device_becomes_current_for_the_call(monkeypatch):
    # a call whose tensors lie on another device than the current one runs there
    seen = []

    class Guard:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            seen.append(("enter", self.index))

        def __exit__(self, *a):
            seen.append(("exit", self.index))

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(dsa, "_raw_stream", lambda index: 1000 + index)
    calls = []
    dsa._launch(lambda *a: calls.append(a) or 0, "f", 1, None, 7)
    assert calls == [(7, 1001)] and seen == [("enter", 1), ("exit", 1)]
    dsa._launch(lambda *a: calls.append(a) or 0, "f", 0, None, 8)
    assert calls[1] == (8, 1000) and len(seen) == 2
    with pytest.raises(dsa.DSAError):
        dsa._launch(lambda *a: 4, "f", 0, None)
