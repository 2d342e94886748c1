"""Descriptors that are out of range, in every kernel of the dense latent attentions: a bounds error, the
rows of the other sequences right, nothing read or written outside (NaN lies around what may be read)."""

import pytest
import torch

import long_context_sparse_lightning_b200 as dsa
from tests.dense_ref import Case
from tests.test_gpu_expanded_mla import Expanded

pytestmark = pytest.mark.gpu
HEADS = [5, 12, 40]          # with two tokens items of 16 rows, of 32, and of a CTA pair


def failing(c, call, ws):
    call(ws)
    with pytest.raises(dsa.DSAError) as e:
        dsa.check_device_error(ws)
    assert e.value.status == 6
    dsa.check_device_error(ws)          # read and cleared


def dense(c, prefix=None):
    op = dsa.OP_DENSE_MLA if prefix is None else dsa.OP_PREFIX_MLA
    ws = dsa.workspace(op, c.batch, n_heads=c.heads)
    out, lse = c.outputs(512)
    if prefix is None:
        call = lambda w: dsa.dense_mla(c.batch, c.q.cuda(), c.cache.cuda(), c.scale, out, lse, w)  # noqa: E731
    else:
        call = lambda w: dsa.prefix_mla(c.batch, prefix, c.q.cuda(), c.cache.cuda(), c.scale, out, lse, w)  # noqa: E731
    failing(c, call, ws)
    return out.cpu(), lse.cpu()


def expanded(c):
    ws = dsa.workspace(dsa.OP_EXPANDED_MLA, c.batch, n_heads=c.heads)
    out, lse = c.outputs(128)
    failing(c, lambda w: dsa.expanded_mla(c.batch, c.q.cuda(), c.up.cuda(), c.cache.cuda()[:, 512:], c.scale, out, lse, w), ws)
    return out.cpu(), lse.cpu()


def near(got, want):
    assert (got.double() - want).norm() <= 2.0 ** -8 * want.norm()


def attend(c, row, positions):
    k = c.cache[positions].double()
    x = c.q[row].double() @ k.T * c.scale
    return torch.softmax(x, -1) @ k[:, :512], torch.logsumexp(x, -1)


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("kv,block", [(300, 1), (300, 4), (9000, 70)])
def test_positions_of_a_page_outside_the_pool_are_skipped(heads, kv, block):
    for page_id in (10 ** 6, -1):
        c = Case([1, 2], [70, kv], heads, 64, seed=51)
        c.table[1, block] = page_id
        out, lse = dense(c)
        near(out[0], attend(c, 0, torch.from_numpy(c.at[0]))[0])
        for i in (0, 1):
            at = torch.from_numpy(c.at[1][:kv - 1 + i])
            seen = torch.arange(kv - 1 + i)
            want, z = attend(c, 1 + i, at[(seen < 64 * block) | (seen >= 64 * block + 64)])
            near(out[1 + i], want)
            assert (lse[1 + i].double() - z).abs().max() <= 1e-3


@pytest.mark.parametrize("heads", HEADS)
def test_a_page_of_the_shared_prefix_outside_the_pool_is_skipped(heads):
    c = Case([2, 1], [400, 390], heads, 64, seed=52, prefix=300)
    c.table[0, 2] = 10 ** 6              # row 0 names the prefix's pages for all
    out, _ = dense(c, 300)
    for row, b, see in ((0, 0, 399), (1, 0, 400), (2, 1, 390)):
        seen = torch.arange(see)
        near(out[row], attend(c, row, torch.from_numpy(c.at[b][:see])[(seen < 128) | (seen >= 192)])[0])


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("what", ["start", "negative start", "last start", "kv_len", "too long", "negative kv_len"])
def test_a_sequence_outside_the_cache_is_zero(heads, what):
    for make, run, dim in ((lambda: Case([2, 2, 1], [200, 300, 100], heads, 0, seed=53), dense, 512),
                           (lambda: Expanded([2, 2, 1], [200, 300, 100], heads, seed=53), expanded, 128)):
        c = make()
        want = (c.exact_dense() if dim == 512 else c.exact_expanded())[0]
        if what == "start":
            c.start[1] = c.total_keys - 299
        elif what == "negative start":
            c.start[1] = -1
        elif what == "last start":
            c.start[1] = 2 ** 63 - 1         # its sum with a length overflows
        else:
            c.kv[1] = {"kv_len": 1, "too long": 301, "negative kv_len": -5}[what]
        out, lse = run(c)
        assert (out[2:4] == 0).all() and torch.isneginf(lse[2:4]).all()
        for r in (0, 1, 4):
            near(out[r], want[r])


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("cu", [[0, 2, 99, 5], [0, 2, -7, 5], [0, 2, 2 ** 31 - 1, 5], [0, 2, 1, 2 ** 31 - 1]])
def test_offsets_that_do_not_rise(heads, cu):
    # sequence 0 has its rows, the others' descriptors name none: their rows are unspecified, sequence 0's right
    for make, run, dim in ((lambda: Case([2, 2, 1], [200, 300, 100], heads, 0, seed=54), dense, 512),
                           (lambda: Case([2, 2, 1], [264, 300, 265], heads, 64, seed=54, prefix=200), lambda c: dense(c, 200), 512),
                           (lambda: Expanded([2, 2, 1], [200, 300, 100], heads, seed=54), expanded, 128)):
        c = make()
        want = (c.exact_dense() if dim == 512 else c.exact_expanded())[0]
        c.cu_q.copy_(torch.tensor(cu, dtype=torch.int32))
        out, _ = run(c)
        near(out[:2], want[:2])


def test_offsets_that_do_not_rise_where_blocks_look_up_their_row_tile():
    c = Expanded([600] + [3] * 30, [600] + [40] * 30, 2, seed=55)
    want = c.exact_expanded()[0]
    c.cu_q[5] = 10 ** 9                  # sequences 4 and 5 have no rows
    out, _ = expanded(c)
    keep = [r for r in range(c.rows) if not 600 + 3 * 3 <= r < 600 + 5 * 3]
    near(out[:c.rows][keep], want[keep])


def test_a_first_row_whose_sum_with_the_length_overflows():
    # the same descriptor in the library's other calls: an error, and not an address far outside
    c = Case([2, 2], [200, 300], 16, 0, seed=56)
    c.start[0] = 2 ** 63 - 1
    ws = dsa.workspace(dsa.OP_FORWARD, c.batch, 64, 16)
    idx = torch.arange(64, dtype=torch.int32, device="cuda").repeat(4, 1)
    out, lse = c.outputs(512)
    failing(c, lambda w: dsa.sparse_mla(c.batch, c.q.cuda(), c.cache.cuda(), idx, 64, c.scale, out, lse, w), ws)
    assert (out[:2] == 0).all() and torch.isneginf(lse[:2]).all() and torch.isfinite(lse[2:]).all()
    k8, ks = torch.zeros((c.total_keys, 128), dtype=torch.uint8, device="cuda"), torch.ones(c.total_keys, device="cuda")
    q8, qs = torch.zeros((4, 64, 128), dtype=torch.uint8, device="cuda"), torch.ones((4, 64), device="cuda")
    scores = torch.full((4, 300), 7.0, device="cuda")
    failing(c, lambda w: dsa.indexer_scores(c.batch, q8, qs, qs, k8, ks, scores, w), ws)
    assert (scores[:2] == 7.0).all() and (scores[2, :299] == 0).all() and (scores[3] == 0).all()
    cache, before = c.cache.cuda(), c.cache.cuda()
    new = torch.zeros((4, 576), dtype=torch.bfloat16, device="cuda")
    failing(c, lambda w: dsa.cache_write(c.batch, new[:, :128].contiguous(), new, k8, ks, cache, w), ws)
    changed = (cache.view(torch.int16) != before.view(torch.int16)).any(1).nonzero().flatten().tolist()
    assert changed == c.at[1][298:].tolist()
