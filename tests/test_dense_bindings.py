"""The bindings of the dense attentions and the page tables on the host: which stream and
device a call's memory and work belong to, and arrays that must not reach a kernel."""

import contextlib

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
        batch, pos, slots, used = dsa.Batch.from_requests(ints(2, 1), ints(0, 5), ints(3, 4), 64, torch.zeros((2, 2), dtype=torch.int32),
                                                          torch.zeros(256, dtype=torch.uint8), 4, 2, 6, 320, stream)
        assert seen == [stream] * 5 and launched[-1] == stream and not inside
        assert batch.total_q == 4 and pos.numel() == slots.numel() == 4 and used.numel() == 1
