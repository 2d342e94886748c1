"""The bindings of the dense attentions and the page tables on a GPU: a batch made on another stream
than the current one, one workspace for steps of different sizes."""

import pytest
import torch

import long_context_sparse_lightning_b200 as dsa
from tests.dense_ref import Case, check
from tests.test_gpu_expanded_mla import Expanded

pytestmark = pytest.mark.gpu


def test_from_requests_on_another_stream_leaves_freed_memory_of_the_current_one():
    # blocks that are free again on the current stream may still be read there by queued work
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    q_len, before, free = i32(2, 1), i32(0, 64), i32(5, 6, 7)
    table, ws = torch.full((2, 3), -1, dtype=torch.int32, device="cuda"), torch.zeros(256, dtype=torch.uint8, device="cuda")
    table[1, 0] = 1
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    olds = [torch.full((n,), 9, dtype=torch.int32, device="cuda") for n in (3, 2, 4, 8, 1) for _ in range(8)]
    torch.cuda._sleep(100_000_000)                    # ~50 ms: the copies below wait behind it
    copies = [x.clone() for x in olds]
    del olds
    batch, pos, slots, used = dsa.Batch.from_requests(q_len, before, free, 64, table, ws, 4, 2, 65, 512, side)
    torch.cuda.synchronize()
    assert all((c == 9).all() for c in copies)
    assert batch.cu_q.tolist() == [0, 2, 3] and batch.kv_len.tolist() == [2, 65] and used.tolist() == [2]
    assert pos.tolist() == [0, 1, 64, 0] and slots.tolist() == [320, 321, 384, -1]
    dsa.check_device_error(ws, side)


def test_expanded_steps_in_one_workspace_of_the_largest():
    # prompts, then few rows over long contexts (split keys), then a step padded far beyond its sequences
    steps = [([700, 300], [700, 900], 0), ([1], [5000], 0), ([40], [2600], 0), ([3, 2], [2000, 900], 700)]
    cases = [Expanded(q, kv, 16, seed=41 + i, pad_rows=pad) for i, (q, kv, pad) in enumerate(steps)]
    bounds = dsa.Batch(cases[0].cu_q, cases[0].kv, cases[0].start, 1000, 700, 5000, 5000)
    ws = dsa.workspace(dsa.OP_EXPANDED_MLA, bounds, n_heads=16)
    for c in cases:
        out, lse = c.outputs(128)
        dsa.expanded_mla(c.batch, c.q.cuda(), c.up.cuda(), c.cache.cuda()[:, 512:], c.scale, out, lse, ws)
        dsa.check_device_error(ws)
        check(out.cpu(), lse.cpu(), c.exact_expanded(), c.rows)


def test_two_captured_graphs_share_a_workspace():
    # one after the other on a stream: nothing in the workspace is kept from one call for the next
    a, b, x = Case([1, 2], [3000, 500], 16, 64, seed=45), Case([3], [900], 40, 0, seed=46), Expanded([20], [2600], 4, seed=47)
    n = max(dsa.workspace_size(dsa.OP_DENSE_MLA, c.batch, 0, c.heads) for c in (a, b))
    n = max(n, dsa.workspace_size(dsa.OP_EXPANDED_MLA, x.batch, 0, 4))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    runs = []
    for c, dim in ((a, 512), (b, 512), (x, 128)):
        q, cache, (out, lse) = c.q.cuda(), c.cache.cuda(), c.outputs(dim)
        if dim == 128:
            up = c.up.cuda()
            call = lambda c=c, q=q, up=up, cache=cache, out=out, lse=lse: dsa.expanded_mla(  # noqa: E731
                c.batch, q, up, cache[:, 512:], c.scale, out, lse, ws)
        else:
            call = lambda c=c, q=q, cache=cache, out=out, lse=lse: dsa.dense_mla(  # noqa: E731
                c.batch, q, cache, c.scale, out, lse, ws)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        # the graph reads q and the caches by address: `call` keeps them (a capture returns freed memory to the device)
        runs.append((g, c, out, lse, c.exact_expanded() if dim == 128 else c.exact_dense(), call))
    for i in (0, 1, 2, 1, 0, 2, 2, 0):
        g, c, out, lse, want, _ = runs[i]
        out.fill_(7.0)
        lse.fill_(7.0)
        g.replay()
        dsa.check_device_error(ws)
        check(out.cpu(), lse.cpu(), want, c.rows)
