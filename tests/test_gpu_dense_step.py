"""Serving steps as a program makes them: page_tables (Batch.from_requests), cache_write,
dense_mla / prefix_mla, step after step on one pool, against 64 bits; the dense
form against the sparse one where the selection holds everything; streams."""

import pytest
import torch

import long_context_sparse_lightning_b200 as dsa

pytestmark = pytest.mark.gpu

PAGE, HEADS, SCALE = 64, 16, 192 ** -0.5


def attend(q, rows, limits):
    """q [n, H, 576] over rows [kv, 576], row i seeing the first limits[i]: [n, H, 512] and lse in 64 bits."""
    outs, zs = [], []
    for i, m in enumerate(limits):
        k = rows[:m].double()
        x = q[i].double() @ k.T * SCALE
        outs.append(torch.softmax(x, -1) @ k[:, :512])
        zs.append(torch.logsumexp(x, -1))
    return torch.stack(outs), torch.stack(zs)


def near(out, lse, want, z):
    assert (out.cpu().double() - want).norm() <= 2.0 ** -8 * want.norm()
    assert (lse.cpu().double() - z).abs().max() <= 1e-3      # scores off by at most 576 * 2^-24 * scale * sum |q c| ~ 1e-3


@pytest.mark.parametrize("pad", [0, 3])
def test_steps_on_one_pool(pad):
    g = torch.Generator().manual_seed(1)
    n, pool = 3, 40 * PAGE
    steps = [[130, 5, 64], [1, 1, 1], [2, 0, 70], [1, 1, 1]]      # prompts, then decode and a chunk
    lat = torch.full((pool, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    k8 = torch.zeros((pool, 128), dtype=torch.uint8, device="cuda")
    ks = torch.zeros(pool, device="cuda")
    table = torch.full((n, 8), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(40, generator=g).to(torch.int32).cuda()
    ws_t = torch.zeros(256, dtype=torch.uint8, device="cuda")
    have = [0] * n
    history = [torch.zeros((0, 576), dtype=torch.bfloat16) for _ in range(n)]
    for q_len in steps:
        total = sum(q_len)
        ql, before = (torch.tensor(x, dtype=torch.int32).cuda() for x in (q_len, have))
        batch, pos, slots, used = dsa.Batch.from_requests(ql, before, free, PAGE, table, ws_t, total + pad,
                                                          max(q_len), 8 * PAGE, pool)
        dsa.check_device_error(ws_t)
        free = free[int(used):]
        new = torch.randn((total + pad, 576), generator=g).to(torch.bfloat16)
        keys = torch.randn((total + pad, 128), generator=g).to(torch.bfloat16)
        ws_c = dsa.workspace(dsa.OP_CACHE_WRITE, batch, 0, 0)
        dsa.cache_write(batch, keys.cuda(), new.cuda(), k8, ks, lat, ws_c)
        dsa.check_device_error(ws_c)
        assert torch.equal(lat[slots[:total]].cpu(), new[:total])       # the slots are where the cache write went
        assert pos[:total].tolist() == [h + i for h, q in zip(have, q_len) for i in range(q)]
        assert slots[total:].tolist() == [-1] * pad
        row = 0
        for b, q in enumerate(q_len):
            history[b] = torch.cat([history[b], new[row:row + q]])
            have[b] += q
            row += q
        q = torch.randn((total + pad, HEADS, 576), generator=g).to(torch.bfloat16)
        out = torch.full((total + pad, HEADS, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((total + pad, HEADS), 7.0, device="cuda")
        ws = dsa.workspace(dsa.OP_DENSE_MLA, batch, n_heads=HEADS)
        dsa.dense_mla(batch, q.cuda(), lat, SCALE, out, lse, ws)
        dsa.check_device_error(ws)
        row = 0
        for b, m in enumerate(q_len):
            if m:
                want, z = attend(q[row:row + m], history[b], [have[b] - m + 1 + i for i in range(m)])
                near(out[row:row + m], lse[row:row + m], want, z)
            row += m
        assert (out[total:] == 7.0).all() and (lse[total:] == 7.0).all()


def test_prefix_over_shared_pages():
    # three requests whose tables begin with the same two pages; the rest comes from page_tables
    g = torch.Generator().manual_seed(2)
    pool, prefix = 20 * PAGE, 2 * PAGE
    lat = torch.randn((pool, 576), generator=g).to(torch.bfloat16).cuda()
    table = torch.full((3, 6), -1, dtype=torch.int32, device="cuda")
    table[:, 0], table[:, 1] = 7, 3
    q_len, before = [2, 1, 3], [prefix, prefix, prefix]
    ws_t = torch.zeros(256, dtype=torch.uint8, device="cuda")
    batch, _, slots, used = dsa.Batch.from_requests(
        torch.tensor(q_len, dtype=torch.int32).cuda(), torch.tensor(before, dtype=torch.int32).cuda(),
        torch.tensor([11, 0, 5, 9], dtype=torch.int32).cuda(), PAGE, table, ws_t, 6, 3, prefix + 3, pool)
    assert int(used) == 3 and slots.tolist() == [11 * PAGE, 11 * PAGE + 1, 0, 5 * PAGE, 5 * PAGE + 1, 5 * PAGE + 2]
    q = torch.randn((6, HEADS, 576), generator=g).to(torch.bfloat16)
    res = []
    for form in ("dense", "prefix"):
        out = torch.empty((6, HEADS, 512), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((6, HEADS), device="cuda")
        ws = dsa.workspace(dsa.OP_DENSE_MLA if form == "dense" else dsa.OP_PREFIX_MLA, batch, n_heads=HEADS)
        if form == "dense":
            dsa.dense_mla(batch, q.cuda(), lat, SCALE, out, lse, ws)
        else:
            dsa.prefix_mla(batch, prefix, q.cuda(), lat, SCALE, out, lse, ws)
        dsa.check_device_error(ws)
        row = 0
        for b, m in enumerate(q_len):
            at = torch.cat([torch.arange(PAGE) + 7 * PAGE, torch.arange(PAGE) + 3 * PAGE, slots[row:row + m].cpu()])
            want, z = attend(q[row:row + m], lat.cpu()[at], [prefix + 1 + i for i in range(m)])
            near(out[row:row + m], lse[row:row + m], want, z)
            row += m
        res.append((out, lse))
    # two roundings of each form: the results differ by at most one bf16 step of the value, or of the sums' size
    assert (res[0][1] - res[1][1]).abs().max() <= 1e-3


def test_equals_the_sparse_form_that_selects_everything():
    g = torch.Generator().manual_seed(3)
    kv = 300
    lat = torch.randn((kv, 576), generator=g).to(torch.bfloat16).cuda()
    q = torch.randn((2, HEADS, 576), generator=g).to(torch.bfloat16).cuda()
    batch = dsa.Batch.from_host([0, 2], [kv], [0])
    idx = torch.full((2, 304), -1, dtype=torch.int32)
    idx[0, :kv - 1] = torch.arange(kv - 1)
    idx[1, :kv] = torch.arange(kv)
    outs = []
    for dense in (True, False):
        out = torch.empty((2, HEADS, 512), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((2, HEADS), device="cuda")
        if dense:
            ws = dsa.workspace(dsa.OP_DENSE_MLA, batch, n_heads=HEADS)
            dsa.dense_mla(batch, q, lat, SCALE, out, lse, ws)
        else:
            ws = dsa.workspace(dsa.OP_SPARSE_MLA, batch, 304, HEADS)
            dsa.sparse_mla(batch, q, lat, idx.cuda(), 304, SCALE, out, lse, ws)
        dsa.check_device_error(ws)
        outs.append((out.double(), lse))
    # bf16 probabilities here, fp16 there: one half step of bf16 each plus the two outputs' roundings
    assert (outs[0][0] - outs[1][0]).norm() <= 2 * 2.0 ** -8 * outs[1][0].norm()
    assert torch.allclose(outs[0][1], outs[1][1], rtol=0, atol=2e-3)


def test_two_streams_with_their_own_workspaces():
    g = torch.Generator().manual_seed(4)
    calls = []
    for kv, heads in ((5000, 16), (3000, 128)):
        batch = dsa.Batch.from_host([0, 1], [kv], [0])
        lat = torch.randn((kv, 576), generator=g).to(torch.bfloat16).cuda()
        q = torch.randn((1, heads, 576), generator=g).to(torch.bfloat16).cuda()
        out = torch.empty((1, heads, 512), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((1, heads), device="cuda")
        calls.append((batch, q, lat, out, lse, dsa.workspace(dsa.OP_DENSE_MLA, batch, n_heads=heads), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for batch, q, lat, out, lse, ws, stream in calls:
            dsa.dense_mla(batch, q, lat, SCALE, out, lse, ws, stream)
    torch.cuda.synchronize()
    for batch, q, lat, out, lse, ws, stream in calls:
        dsa.check_device_error(ws)
        want, z = attend(q.cpu(), lat.cpu(), [lat.shape[0]])
        near(out, lse, want, z)
