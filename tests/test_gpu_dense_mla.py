"""Dense latent attention (dsa_dense_mla) and its shared-prefix form (dsa_prefix_mla)
against their definitions in 64 bits."""

import pytest
import torch

import long_context_sparse_lightning_b200 as dsa
from tests.dense_ref import Case, check

pytestmark = pytest.mark.gpu

CASES = [
    # (q_len, kv_len, heads, page)
    ([1], [1], 16, 0),                                        # one key
    ([1], [64], 16, 0),
    ([1], [65], 1, 64),
    ([1], [1000], 16, 0),
    ([2], [130], 16, 64),                                     # 32 rows
    ([1, 1, 1], [5, 700, 63], 5, 128),
    ([1, 0, 2], [100, 50, 300], 24, 64),                      # a sequence without tokens, ragged counts
    ([3, 1], [3, 260], 128, 0),                               # several row tiles, first tokens see one key
    ([5], [201], 20, 192),                                    # rows that straddle row tiles
    ([1] * 40, [17 * i + 1 for i in range(40)], 16, 64),
    ([70], [70], 16, 0),                                      # prefill: causal inside a tile and across
    ([33, 2], [400, 129], 128, 64),                           # many row tiles, gangs
    ([1], [20000], 128, 64),                                  # one row split over many CTAs
    ([2, 1], [9000, 5], 16, 0),
    # more sequences than a block has threads: the lengths are scanned in chunks
    ([1] * 500, [1 + (37 * i) % 150 for i in range(500)], 4, 64),
    ([(i % 3) for i in range(450)], [2 + (91 * i) % 130 for i in range(450)], 33, 0),
]


@pytest.mark.parametrize("q,kv,heads,page", CASES)
def test_dense_against_64_bits(q, kv, heads, page):
    c = Case(q, kv, heads, page, seed=1)
    out, lse = c.dense()
    check(out, lse, c.exact_dense(), c.rows)


def test_rows_behind_the_last_sequence_are_left():
    c = Case([1, 2], [90, 300], 16, 64, seed=2, pad_rows=5)
    out, lse = c.dense()
    check(out, lse, c.exact_dense(), c.rows)


def test_growing_and_falling_scores():
    # the reference of a row is taken from its first tile and replaced when a
    # score exceeds it by 2^24: scores that climb over hundreds of log2 units along
    # the sequence replace it again and again, falling ones never
    for sign in (1.0, -1.0):
        c = Case([1, 2], [500, 700], 16, 0, seed=3)
        for at, n in zip(c.at, c.kv_len):
            ramp = (sign * torch.arange(n).float() / n * 600).to(torch.bfloat16)
            c.cache[at, 575] = ramp
        c.q[:, :, 575] = 8.0
        out, lse = c.dense()
        # e counts the largest |q k| of any key; here the sums are dominated by one exact product
        check(out, lse, c.exact_dense(), c.rows)


def test_values_at_positions_later_tokens_alone_see():
    # a later token's NaN cache row reaches that token and no earlier one
    c = Case([3], [130], 16, 0, seed=4)
    c.cache[c.at[0][129], 3] = float("nan")
    out, lse = c.dense()
    ref = Case([3], [130], 16, 0, seed=4)
    want, z, A, e = ref.exact_dense()
    assert torch.isnan(out[2].float()).all() and torch.isnan(lse[2]).all()
    assert torch.isfinite(out[:2].float()).all()
    d = (out[:2].double() - want[:2]).abs()
    assert (d <= A[:2] * (2.0 ** -8 + 2 * e[:2, :, None] + 2.0 ** -18) + 2.0 ** -8 * want[:2].abs()).all()


def test_bad_descriptors_are_bounds_errors():
    c = Case([1, 1, 1], [200, 300, 100], 16, 0, seed=5)
    c.start[1] = c.total_keys - 10                        # its rows would lie outside the cache
    out, lse = c.outputs(512)
    ws = dsa.workspace(dsa.OP_DENSE_MLA, c.batch, n_heads=16)
    dsa.dense_mla(c.batch, c.q.cuda(), c.cache.cuda(), c.scale, out, lse, ws)
    with pytest.raises(dsa.DSAError) as e:
        dsa.check_device_error(ws)
    assert e.value.status == 6
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()
    want, z, A, er = c.exact_dense()
    for r in (0, 2):
        assert (out[r].cpu().double() - want[r]).norm() <= 2.0 ** -8 * want[r].norm()


def test_a_page_outside_the_pool_is_skipped():
    c = Case([1], [200], 16, 64, seed=6)
    c.table[0, 1] = 10 ** 6
    out, lse = c.outputs(512)
    ws = dsa.workspace(dsa.OP_DENSE_MLA, c.batch, n_heads=16)
    dsa.dense_mla(c.batch, c.q.cuda(), c.cache.cuda(), c.scale, out, lse, ws)
    with pytest.raises(dsa.DSAError) as e:
        dsa.check_device_error(ws)
    assert e.value.status == 6
    # the other positions' attention
    rows = torch.cat([torch.from_numpy(c.at[0][:64]), torch.from_numpy(c.at[0][128:])])
    k = c.cache[rows].double()
    p = torch.softmax(c.q[0].double() @ k.T * c.scale, -1)
    want = p @ k[:, :512]
    assert (out[0].cpu().double() - want).norm() <= 2.0 ** -8 * want.norm()


PREFIX = [
    # (prefix, q_len, tails, heads, page)
    (64, [1, 1], [1, 1], 16, 64),
    (1000, [1] * 6, [1, 100, 5, 64, 28, 29], 16, 64),
    (5, [1, 2, 3], [3, 3, 70], 5, 64),
    (640, [2] * 5, [2, 50, 200, 3, 129], 128, 128),
    (0, [1, 1], [20, 30], 16, 64),
    (3000, [1] * 33, [1 + 7 * i for i in range(33)], 16, 64),
    (129, [1, 0, 4], [1, 10, 4], 30, 64),
    (200, [1] * 420, [1 + (13 * i) % 90 for i in range(420)], 4, 64),
]


@pytest.mark.parametrize("prefix,q,tails,heads,page", PREFIX)
def test_prefix_against_64_bits(prefix, q, tails, heads, page):
    c = Case(q, [prefix + t for t in tails], heads, page, seed=7, prefix=prefix, pad_rows=2)
    out, lse = c.dense(prefix)
    check(out, lse, c.exact_dense(), c.rows)


def test_prefix_longer_than_a_sequence_is_a_bounds_error():
    c = Case([1, 1], [130, 200], 16, 64, seed=8, prefix=64)
    out, lse = c.outputs(512)
    ws = dsa.workspace(dsa.OP_PREFIX_MLA, c.batch, n_heads=16)
    # sequence 0 holds 130 positions: with a prefix of 130 its query lies inside it
    dsa.prefix_mla(c.batch, 130, c.q.cuda(), c.cache.cuda(), c.scale, out, lse, ws)
    with pytest.raises(dsa.DSAError) as e:
        dsa.check_device_error(ws)
    assert e.value.status == 6
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()
    assert torch.isfinite(lse[1]).all()


def test_one_workspace_for_calls_of_different_shapes():
    big = Case([1] * 9, [900] * 9, 128, 64, seed=9)
    small = Case([1], [3000], 16, 64, seed=10)
    n = max(dsa.workspace_size(dsa.OP_DENSE_MLA, x.batch, 0, x.heads) for x in (big, small))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    for c in (big, small, big, small):
        out, lse = c.dense(ws=ws)
        check(out, lse, c.exact_dense(), c.rows)


def test_captured_and_replayed_with_new_lengths():
    # lengths are read on the device: a captured call replays on grown sequences
    c = Case([1, 1], [700, 900], 16, 64, seed=11)
    q, cache = c.q.cuda(), c.cache.cuda()
    out, lse = c.outputs(512)
    ws = dsa.workspace(dsa.OP_DENSE_MLA, c.batch, n_heads=16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        dsa.dense_mla(c.batch, q, cache, c.scale, out, lse, ws)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.dense_mla(c.batch, q, cache, c.scale, out, lse, ws)
    for kv in ([700, 900], [10, 899], [650, 1]):
        c.kv.copy_(torch.tensor(kv, dtype=torch.int32))
        c.kv_len = kv
        c.at_all = getattr(c, "at_all", c.at)
        c.at = [a[:k] for a, k in zip(c.at_all, kv)]
        out.fill_(7.0)
        g.replay()
        dsa.check_device_error(ws)
        check(out.cpu(), lse.cpu(), c.exact_dense(), c.rows)


def test_same_bits_again_and_without_lse():
    for c, prefix in ((Case([1, 3], [3000, 700], 16, 64, seed=12), None), (Case([2], [5000], 128, 0, seed=13), None),
                      (Case([1, 2, 1], [700, 650, 900], 20, 64, seed=14, prefix=640), 640)):
        first, z = c.dense(prefix)
        again, _ = c.dense(prefix)
        assert torch.equal(first.view(torch.int16), again.view(torch.int16))
        out, _ = c.outputs(512)
        op = dsa.OP_DENSE_MLA if prefix is None else dsa.OP_PREFIX_MLA
        ws = dsa.workspace(op, c.batch, n_heads=c.heads)
        if prefix is None:
            dsa.dense_mla(c.batch, c.q.cuda(), c.cache.cuda(), c.scale, out, None, ws)
        else:
            dsa.prefix_mla(c.batch, prefix, c.q.cuda(), c.cache.cuda(), c.scale, out, None, ws)
        dsa.check_device_error(ws)
        assert torch.equal(first.view(torch.int16), out.cpu().view(torch.int16))


def test_a_row_of_nan_queries_stays_alone():
    c = Case([2, 1], [300, 90], 16, 64, seed=15)
    want = c.exact_dense()
    c.q[1, 5] = float("nan")
    out, lse = c.dense()
    assert torch.isnan(out[1, 5].float()).all() and torch.isnan(lse[1, 5])
    keep = torch.ones((3, 16), dtype=torch.bool)
    keep[1, 5] = False
    d = (out.double() - want[0])[keep]
    assert torch.isfinite(d).all() and d.norm() <= 2.0 ** -8 * want[0][keep].norm()


def test_a_step_without_tokens():
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    bf = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    paged = dsa.Batch(i32(0, 0), i32(70), None, 0, 0, 70, 128, block_table=i32(1, 0).view(1, 2), page_size=64)
    flat = dsa.Batch(i32(0, 0), i32(70), torch.zeros(1, dtype=torch.int64, device="cuda"), 0, 0, 70, 128)
    lse = torch.empty((0, 16), device="cuda")
    for op, call in ((dsa.OP_DENSE_MLA, lambda ws: dsa.dense_mla(paged, bf(0, 16, 576), bf(128, 576), 1.0, bf(0, 16, 512),
                                                                 lse, ws)),
                     (dsa.OP_PREFIX_MLA, lambda ws: dsa.prefix_mla(paged, 64, bf(0, 16, 576), bf(128, 576), 1.0,
                                                                   bf(0, 16, 512), lse, ws)),
                     (dsa.OP_EXPANDED_MLA, lambda ws: dsa.expanded_mla(flat, bf(0, 16, 192), bf(128, 16, 256), bf(128, 64),
                                                                       1.0, bf(0, 16, 128), lse, ws))):
        ws = dsa.workspace(op, flat if op == dsa.OP_EXPANDED_MLA else paged, 0, 16)
        call(ws)
        dsa.check_device_error(ws)
