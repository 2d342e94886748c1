"""Latent attention in the expanded form (dsa_expanded_mla) against its definition in 64 bits."""

import pytest
import torch

import long_context_sparse_lightning_b200 as dsa
from tests.dense_ref import Case, check

pytestmark = pytest.mark.gpu


class Expanded(Case):
    """Case with per-head keys and values; rows that no sequence owns are NaN."""

    def __init__(self, q_len, kv_len, heads, seed=0, **kw):
        super().__init__(q_len, kv_len, heads, 0, seed=seed, q_dim=192, **kw)
        self.up = torch.full((self.total_keys, heads, 256), float("nan"), dtype=torch.bfloat16)
        self.up[self.used] = torch.randn((len(self.used), heads, 256), generator=self.g).to(torch.bfloat16)

    def run(self, check=True, contiguous_rope=False):
        out, lse = self.outputs(128)
        ws = dsa.workspace(dsa.OP_EXPANDED_MLA, self.batch, n_heads=self.heads)
        rope = self.cache.cuda()[:, 512:]
        if contiguous_rope:
            rope = rope.contiguous()
        dsa.expanded_mla(self.batch, self.q.cuda(), self.up.cuda(), rope, self.scale, out, lse, ws)
        if check:
            dsa.check_device_error(ws)
        return out.cpu(), lse.cpu()

    def exact_expanded(self):
        def kv(b):
            up = self.up[self.at[b]].double()
            r = self.cache[self.at[b], 512:].double()[:, None, :].expand(-1, self.heads, -1)
            return torch.cat([up[..., :128], r], -1), up[..., 128:]
        return self.exact(kv)


CASES = [
    # (q_len, kv_len, heads)
    ([1], [1], 1),
    ([1], [129], 3),
    ([128], [128], 2),
    ([129], [129], 2),
    ([256], [256], 1),
    ([257, 3], [300, 1000], 2),
    ([5, 0, 130], [5, 40, 200], 3),
    ([700], [1500], 2),
    ([100, 300, 1, 513], [100, 333, 513, 640], 4),
    ([64], [2000], 16),
    ([30], [30], 128),
    # long prompts, short sequences among them
    ([1024], [1024], 19),
    ([1100, 5, 257, 600], [1300, 5, 400, 601], 16),
    ([1025, 0, 1], [1700, 9, 128], 25),
    # few rows, long contexts: the keys are split
    ([1], [5000], 2),
    ([200], [3001], 3),
    ([256, 7], [2600, 400], 1),                   # parts that end before the other sequence's, or hold none of its keys
    ([300], [2049], 1),
]


@pytest.mark.parametrize("q,kv,heads", CASES)
def test_expanded_against_64_bits(q, kv, heads):
    c = Expanded(q, kv, heads, seed=1, pad_rows=3)
    out, lse = c.run(contiguous_rope=heads % 2 == 0)
    check(out, lse, c.exact_expanded(), c.rows)


def test_growing_scores():
    for sign, n, kv, heads in ((1.0, 300, 900, 2), (-1.0, 300, 900, 2), (1.0, 1030, 1100, 25), (-1.0, 1030, 1100, 25)):
        c = Expanded([n], [kv], heads, seed=2)
        c.up[c.at[0], :, 5] = (sign * torch.arange(kv).float() / kv * 600).to(torch.bfloat16)[:, None]
        c.q[:, :, 5] = 8.0
        out, lse = c.run()
        check(out, lse, c.exact_expanded(), c.rows)


@pytest.mark.parametrize("n,heads,at,dim", [(300, 1, 200, 9), (1030, 25, 200, 9), (1030, 25, 700, 73), (1030, 25, 1026, 127)])
def test_values_at_positions_later_tokens_alone_see(n, heads, at, dim):
    c = Expanded([n], [n], heads, seed=3)
    want = c.exact_expanded()
    row = c.at[0][at]
    c.up[row, 0, 128 + dim] = float("nan")        # a value of position `at`
    if at + 50 < n:
        c.up[row + 50, 0, 3] = float("inf")       # a key of a later one
    out, _ = c.run()
    got = out[:n, 0].float()
    assert torch.isfinite(got[:at]).all()
    assert torch.isnan(got[at:, dim]).all()
    assert torch.isfinite(got[at:at + 50][:, [d for d in range(128) if d != dim]]).all()
    d = (got[:at].double() - want[0][:at, 0]).abs()
    A, e = want[2][:at, 0], want[3][:at, 0]
    assert (d <= A * (2.0 ** -8 + 2 * e[:, None] + 2.0 ** -18) + 2.0 ** -8 * want[0][:at, 0].abs()).all()
    for h in range(1, heads):                     # the other heads' values are theirs
        assert (out[:n, h].double() - want[0][:, h]).norm() <= 2.0 ** -8 * want[0][:, h].norm()


def test_bad_descriptors_are_bounds_errors():
    c = Expanded([10, 10], [50, 60], 2, seed=4)
    want = c.exact_expanded()
    c.start[1] = c.total_keys - 5
    out, lse = c.outputs(128)
    ws = dsa.workspace(dsa.OP_EXPANDED_MLA, c.batch, n_heads=2)
    dsa.expanded_mla(c.batch, c.q.cuda(), c.up.cuda(), c.cache.cuda()[:, 512:], c.scale, out, lse, ws)
    with pytest.raises(dsa.DSAError) as e:
        dsa.check_device_error(ws)
    assert e.value.status == 6
    assert (out[10:20] == 0).all() and torch.isneginf(lse[10:20]).all()
    assert (out[:10].cpu().double() - want[0][:10]).norm() <= 2.0 ** -8 * want[0][:10].norm()


def test_equals_the_absorbed_form():
    # keys and values made from the latent rows by up-projections, and the same
    # projections absorbed into q and applied to the absorbed output
    heads, n = 4, 200
    c = Case([n], [n], heads, 0, seed=5, q_dim=192)
    g = torch.Generator().manual_seed(6)
    wk = torch.randn((heads, 128, 512), generator=g) / 512 ** 0.5
    wv = torch.randn((heads, 128, 512), generator=g) / 512 ** 0.5
    lat = c.cache.nan_to_num().double()
    up = torch.cat([torch.einsum("hdc,sc->shd", wk.double(), lat[:, :512]),
                    torch.einsum("hdc,sc->shd", wv.double(), lat[:, :512])], -1).to(torch.bfloat16)
    qa = torch.cat([torch.einsum("ihd,hdc->ihc", c.q[..., :128].double(), wk.double()), c.q[..., 128:].double()], -1)
    out, lse = c.outputs(128)
    ws = dsa.workspace(dsa.OP_EXPANDED_MLA, c.batch, n_heads=heads)
    dsa.expanded_mla(c.batch, c.q.cuda(), up.cuda(), c.cache.cuda()[:, 512:], c.scale, out, lse, ws)
    dsa.check_device_error(ws)
    oa, la = c.outputs(512)
    ws = dsa.workspace(dsa.OP_DENSE_MLA, c.batch, n_heads=heads)
    dsa.dense_mla(c.batch, qa.to(torch.bfloat16).cuda(), c.cache.cuda(), c.scale, oa, la, ws)
    dsa.check_device_error(ws)
    o2 = torch.einsum("ihc,hdc->ihd", oa.cpu().double(), wv.double())
    # per form: the operands' rounding (keys, values or absorbed q: 2^-8 each, which moves a score of size
    # |q||k| scale ~ 1 by as much), the probabilities' and the output's: six half steps in all, in the 2-norm
    assert (out.cpu().double() - o2).norm() <= 6 * 2.0 ** -8 * o2.norm()


def test_more_tokens_than_the_host_said_is_a_bounds_error():
    c = Expanded([300, 10], [300, 40], 1, seed=7)
    want = c.exact_expanded()
    c.batch.c.max_q_per_seq = 256                    # sizes the grid: sequence 0's last rows have no block
    out, lse = c.outputs(128)
    ws = dsa.workspace(dsa.OP_EXPANDED_MLA, c.batch, n_heads=1)
    dsa.expanded_mla(c.batch, c.q.cuda(), c.up.cuda(), c.cache.cuda()[:, 512:], c.scale, out, lse, ws)
    with pytest.raises(dsa.DSAError) as e:
        dsa.check_device_error(ws)
    assert e.value.status == 6
    assert (out[:256] == 0).all() and torch.isneginf(lse[:256]).all()
    assert (out[300:310].cpu().double() - want[0][300:]).norm() <= 2.0 ** -8 * want[0][300:].norm()


@pytest.mark.parametrize("q,kv,heads", [
    ([700] + [3] * 20, [900] + [5 + i for i in range(20)], 2),                   # most blocks look up their row tile
    ([3] * 400 + [600, 0, 257] + [1] * 30, [4] * 400 + [600, 3, 300] + [9] * 30, 1),     # more sequences than threads
    ([600, 2, 0, 5, 1, 1], [6000, 4000, 7, 900, 3000, 1], 1),                    # and the keys are split
])
def test_one_long_sequence_among_short_ones(q, kv, heads):
    c = Expanded(q, kv, heads, seed=12)
    out, lse = c.run()
    check(out, lse, c.exact_expanded(), c.rows)


@pytest.mark.parametrize("q,kv,heads", [
    ([100] * 4, [100, 129, 700, 257], 128),                   # two heads a block, 1 to 6 key tiles of each
    ([3, 128, 1, 0, 128, 60], [300, 128, 1, 9, 500, 60], 127),   # the last head alone
    ([257, 40, 128, 129], [300, 40, 640, 1000], 128),         # blocks of one and of two heads
    ([300] + [5] * 40, [300] + [140 + i for i in range(40)], 33),
    ([700] + [3] * 20, [900] + [5 + i for i in range(20)], 17),  # and the blocks look up their row tile
])
def test_two_heads_per_block(q, kv, heads):
    c = Expanded(q, kv, heads, seed=14)
    out, lse = c.run()
    check(out, lse, c.exact_expanded(), c.rows)


def test_a_bad_descriptor_of_two_heads_per_block():
    c = Expanded([40] * 4, [50, 60, 40, 300], 127, seed=16)
    want = c.exact_expanded()
    c.start[1] = c.total_keys - 5
    out, lse = c.outputs(128)
    ws = dsa.workspace(dsa.OP_EXPANDED_MLA, c.batch, n_heads=127)
    dsa.expanded_mla(c.batch, c.q.cuda(), c.up.cuda(), c.cache.cuda()[:, 512:], c.scale, out, lse, ws)
    with pytest.raises(dsa.DSAError) as e:
        dsa.check_device_error(ws)
    assert e.value.status == 6
    assert (out[40:80] == 0).all() and torch.isneginf(lse[40:80]).all()
    keep = [r for r in range(160) if not 40 <= r < 80]
    assert (out.cpu().double() - want[0])[keep].norm() <= 2.0 ** -8 * want[0][keep].norm()


def test_values_that_are_not_finite_stay_with_their_head_and_rows():
    # of two heads in a block, at a position that later rows alone see
    c = Expanded([90, 70, 5], [220, 70, 5], 128, seed=15)
    want = c.exact_expanded()
    at, head = 60, 41
    c.up[c.at[0][130 + at], head, 128 + 7] = float("inf")
    out, lse = c.run()
    bad = torch.isnan(out.float())
    assert bad[at:90, head, 7].all() and int(bad.sum()) == 90 - at
    d = (out.double() - want[0])[~bad]
    assert d.norm() <= 2.0 ** -8 * want[0][~bad].norm()


def test_rows_of_too_many_tokens_are_zero():
    # the grid's last row tile of the sequence takes the rows behind it, whichever way the blocks find their tiles
    for q, kv, max_q in (([600, 10], [600, 40], 256), ([900] + [4] * 12, [900] + [30] * 12, 600), ([300], [5000], 200)):
        c = Expanded(q, kv, 1, seed=13)
        want = c.exact_expanded()
        c.batch.c.max_q_per_seq = max_q
        out, lse = c.outputs(128)
        ws = dsa.workspace(dsa.OP_EXPANDED_MLA, c.batch, n_heads=1)
        dsa.expanded_mla(c.batch, c.q.cuda(), c.up.cuda(), c.cache.cuda()[:, 512:], c.scale, out, lse, ws)
        with pytest.raises(dsa.DSAError) as e:
            dsa.check_device_error(ws)
        assert e.value.status == 6
        n = q[0]
        assert (out[:n] == 0).all() and torch.isneginf(lse[:n]).all()
        assert (out[n:c.rows].cpu().double() - want[0][n:]).norm() <= 2.0 ** -8 * want[0][n:].norm()


def test_same_bits_again_and_without_lse():
    for q, kv, heads in (([300, 5], [700, 40], 3), ([1100], [1200], 30), ([40], [4000], 2)):
        c = Expanded(q, kv, heads, seed=8)
        first, _ = c.run()
        again, _ = c.run()
        assert torch.equal(first.view(torch.int16), again.view(torch.int16))
        out, _ = c.outputs(128)
        ws = dsa.workspace(dsa.OP_EXPANDED_MLA, c.batch, n_heads=heads)
        dsa.expanded_mla(c.batch, c.q.cuda(), c.up.cuda(), c.cache.cuda()[:, 512:], c.scale, out, None, ws)
        dsa.check_device_error(ws)
        assert torch.equal(first.view(torch.int16), out.cpu().view(torch.int16))


def test_nan_and_infinite_scores_stay_in_their_rows():
    c = Expanded([200], [500], 2, seed=9)
    want = c.exact_expanded()
    c.q[7, 1] = float("nan")
    c.q[150, 0, 3] = float("inf")                   # scores of +-inf: NaN by the definition
    out, lse = c.run()
    for r, h in ((7, 1), (150, 0)):
        assert torch.isnan(out[r, h].float()).all() and torch.isnan(lse[r, h])
    keep = torch.ones((200, 2), dtype=torch.bool)
    keep[7, 1] = keep[150, 0] = False
    d = (out.double() - want[0])[keep]
    assert torch.isfinite(d).all() and d.norm() <= 2.0 ** -8 * want[0][keep].norm()


def test_captured_and_replayed_with_new_lengths():
    c = Expanded([100, 60], [400, 200], 2, seed=10)
    q, up, cache = c.q.cuda(), c.up.cuda(), c.cache.cuda()
    out, lse = c.outputs(128)
    ws = dsa.workspace(dsa.OP_EXPANDED_MLA, c.batch, n_heads=2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        dsa.expanded_mla(c.batch, q, up, cache[:, 512:], c.scale, out, lse, ws)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.expanded_mla(c.batch, q, up, cache[:, 512:], c.scale, out, lse, ws)
    whole = c.at
    for kv in ([400, 200], [130, 60], [257, 199]):
        c.kv.copy_(torch.tensor(kv, dtype=torch.int32))
        c.kv_len = kv
        c.at = [a[:k] for a, k in zip(whole, kv)]
        out.fill_(7.0)
        g.replay()
        dsa.check_device_error(ws)
        check(out.cpu(), lse.cpu(), c.exact_expanded(), c.rows)
