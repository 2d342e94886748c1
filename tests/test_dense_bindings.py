"""The bindings of the dense attentions and the page tables on the host: which stream and
device a call's memory and work belong to, and arrays that must not reach a kernel."""

import contextlib
import ctypes
import random

import pytest
import torch

import long_context_sparse_lightning_b200 as dsa


def ints(*v):
    return torch.tensor(v, dtype=torch.int32)


def test_from_requests_allocates_on_the_stream_that_writes(monkeypatch):
    # the caching allocator hands memory out in the order of the stream it was asked on: what `stream`
    # writes has to come from its own pool
    inside, seen = [], []

    @contextlib.contextmanager
    def on(stream):
        inside.append(stream)
        yield
        inside.pop()

    empty = torch.empty

    def alloc(*a, **kw):
        seen.append(inside[-1] if inside else None)
        return empty(*a, **kw)

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", alloc)
    launched = []
    monkeypatch.setattr(dsa, "page_tables", lambda *a: launched.append(a[-1]))
    for stream in (None, "side"):
        seen.clear()
        batch, pos, slots, used = dsa.Batch.from_requests(
            ints(2, 1), ints(0, 5), ints(3, 4), 64, torch.zeros((2, 2), dtype=torch.int32),
            torch.zeros(256, dtype=torch.uint8), 4, 2, 6, 320, stream)
        assert seen == [stream] * 5 and launched[-1] == stream and not inside
        assert batch.total_q == 4 and pos.numel() == slots.numel() == 4 and used.numel() == 1


def test_batch_arrays_lie_together():
    # a host array, one on another device, a strided or a short one would be read at the wrong addresses
    cu, kv, start, table = ints(0, 2, 3), ints(5, 9), torch.tensor([0, 5]), torch.zeros((2, 2), dtype=torch.int32)
    make = lambda cu=cu, kv=kv, start=start, table=None: dsa.Batch(cu, kv, start, 3, 2, 9, 128, block_table=table,  # noqa: E731
                                                                  page_size=64 if table is not None else 0)
    make()
    make(start=None, table=table)
    make(cu=ints(0, 2, 3, 0, 0), start=torch.tensor([0, 5, 0]), table=torch.zeros((4, 2), dtype=torch.int32))  # spare entries
    for bad in (dict(kv=kv.to("meta")), dict(start=start.to("meta")), dict(table=table.to("meta")), dict(cu=cu.to("meta")),
                dict(cu=ints(0, 9, 2, 9, 3)[::2]), dict(kv=ints(5, 0, 9, 0)[::2]), dict(start=torch.tensor([0, 9, 5, 9])[::2]),
                dict(cu=ints(0, 2)), dict(start=torch.tensor([0])), dict(table=table[:1])):
        with pytest.raises(ValueError):
            make(**bad)


def test_errors_are_read_behind_the_stream_of_the_workspaces_device(monkeypatch):
    # a call whose tensors lie on another device than the current one runs on that device's stream: so
    # does the wait before its error word is read
    seen = []

    class Guard:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            seen.append(self.index)

        def __exit__(self, *a):
            seen.append(-1)

    class Ws:
        def __init__(self, index):
            self.index = index

        def get_device(self):
            return self.index

        def is_contiguous(self):
            return True

        def data_ptr(self):
            return 4096

    class Lib:
        @staticmethod
        def dsa_check_device_error(ws, stream, site, info):
            seen.append((ws, stream))
            return 0

    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream)
    monkeypatch.setattr(dsa, "_raw_stream", lambda index: 1000 + index)
    monkeypatch.setattr(dsa, "_lib", lambda: Lib)
    dsa.check_device_error(Ws(1))
    assert seen == [1, (4096, 1001), -1]
    del seen[:]
    dsa.check_device_error(Ws(0))
    dsa.check_device_error(Ws(0), Stream)
    assert seen == [(4096, 1000), (4096, 77)]
    with pytest.raises(ValueError, match="CUDA"):
        dsa.check_device_error(torch.zeros(256, dtype=torch.uint8))


def test_a_workspace_serves_every_smaller_batch():
    # a serving loop allocates once, for its bounds: fewer rows over long contexts are split into more parts
    lib, rng = dsa.library(), random.Random(1)

    def size(op, heads, B, total_q, max_q, max_kv):
        c = dsa._BatchC()
        c.num_seqs, c.total_q, c.max_q_per_seq, c.max_kv_len, c.total_keys = B, total_q, max_q, max_kv, 1 << 20
        c.cu_q = c.kv_len = c.block_table = 0x1000
        c.page_size, c.blocks_per_seq = 64, 1 << 14
        if op == dsa.OP_EXPANDED_MLA:
            c.block_table, c.kv_start = None, 0x1000
        return lib.dsa_workspace_size(op, ctypes.byref(c), 0, heads)

    for _ in range(2000):
        heads = rng.choice([1, 2, 16, 20, 70, 128])
        total_q = rng.choice([1, 10, 300, 8192, 40000])
        big = (rng.choice([1, 2, 8, 500]), total_q, rng.randint(1, total_q), 0)
        big = big[:3] + (max(big[2], rng.choice([1, 700, 3000, 100000])),)
        small = (rng.randint(1, big[0]), rng.randint(1, big[1]))
        small += (rng.randint(1, min(small[1], big[2])),)
        small += (rng.randint(small[2], big[3]),)
        for op in (dsa.OP_DENSE_MLA, dsa.OP_PREFIX_MLA, dsa.OP_EXPANDED_MLA):
            need, have = size(op, heads, *small), size(op, heads, *big)
            assert 0 < need <= have, (op, heads, small, big)
            if op == dsa.OP_EXPANDED_MLA:
                assert have <= 20 << 20
