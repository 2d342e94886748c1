"""Infinities that a query does see, in the dense latent attentions: by the definition a key of score -inf
has weight 0, and 0 x an infinite value is NaN in that dim, wherever the tiles, the items and the pieces of a
split end.  A value that is not finite makes the output NaN in its dim (dsa.h); a NaN or a score of +inf the whole row."""

import pytest
import torch

from tests.dense_ref import Case, compare_nonfinite

pytestmark = pytest.mark.gpu
INF = float("inf")


def latent(c):
    rows = [c.cache[at].double() for at in c.at]
    return lambda b, h: (rows[b], rows[b][:, :512])


DENSE = [
    # (q_len, kv_len, heads, page, bad positions of the last sequence)
    ([3], [130], 5, 0, [129]),                       # 15, 30, 48 rows; only the last token sees it
    ([3], [130], 10, 64, [128, 129]),
    ([3], [130], 16, 0, [128, 129]),
    ([1, 2], [70, 200], 64, 64, [199]),
    ([2], [500], 8, 0, [100]),                       # in a tile that all rows see
    ([2], [500], 40, 0, [100]),
    ([2], [2562], 8, 64, range(2432, 2562)),         # whole pieces of a split hold nothing else
    ([2], [4098], 40, 0, range(3900, 4098)),
    ([4], [2050], 33, 64, range(2046, 2050)),
]


@pytest.mark.parametrize("dim", [7, 300, 540])
@pytest.mark.parametrize("q,kv,heads,page,bad", DENSE)
def test_infinite_cache_values_that_are_seen(q, kv, heads, page, bad, dim):
    for sign in (1.0, -1.0):
        c = Case(q, kv, heads, page, seed=21)
        c.cache[c.at[-1][list(bad)], dim] = sign * INF
        out, lse = c.dense()
        nan_dims = compare_nonfinite(c, out, lse, latent(c))
        assert nan_dims > 0


@pytest.mark.parametrize("heads", [4, 40])
def test_infinite_values_behind_a_shared_prefix(heads):
    c = Case([2, 1, 3], [72, 75, 290], heads, 64, seed=22, prefix=70)
    for b, at in ((0, 70), (1, 74), (2, 289), (2, 200)):
        c.cache[c.at[b][at], 11] = INF
    c.cache[c.at[1][10], 500] = -INF                 # in the prefix: a copy of sequence 0's row, so all of them
    c.cache[c.at[0][10], 500] = c.cache[c.at[2][10], 500] = -INF
    out, lse = c.dense(70)
    compare_nonfinite(c, out, lse, latent(c))


@pytest.mark.parametrize("heads,kv", [(8, 100), (8, 3000), (40, 100), (40, 3000)])
def test_rows_whose_scores_are_all_minus_infinity(heads, kv):
    # no key has a weight: 0 and -inf as for a row without keys, and NaN where a value is not finite
    c = Case([2], [kv], heads, 0, seed=23)
    c.cache[c.at[0], 7] = INF
    c.q[:, :, 7] = -1.0
    out, lse = c.dense()
    assert torch.isneginf(lse[:2]).all()
    assert torch.isnan(out[:2, :, 7].float()).all()
    rest = torch.cat([out[:2, :, :7], out[:2, :, 8:]], -1)
    assert (rest == 0).all()


def test_infinite_values_among_many_items_of_a_pair():
    # items without keys (sequences out of range) among those that the pairs walk, infinities in most others
    n, heads = 400, 64
    c = Case([2] * n, [40 + (37 * i) % 300 for i in range(n)], heads, 64, seed=27)
    clean = c.exact_dense()[0]
    bad = [i % 5 != 0 and i % 3 == 0 for i in range(n)]          # kv_len out of range
    for i in range(n):
        if i % 4 != 3:
            c.cache[c.at[i][-1], (13 * i) % 512] = INF           # the last token alone sees it
        if bad[i]:
            c.kv[i] = 1
    out, lse = c.dense(check=False)
    for i in range(n):
        a, b = out[2 * i].double(), out[2 * i + 1].double()
        if bad[i]:
            assert (a == 0).all() and (b == 0).all() and torch.isneginf(lse[2 * i:2 * i + 2]).all()
            continue
        assert (a - clean[2 * i]).norm() <= 2.0 ** -8 * clean[2 * i].norm()
        if i % 4 == 3:
            assert (b - clean[2 * i + 1]).norm() <= 2.0 ** -8 * clean[2 * i + 1].norm()
        else:
            down = c.q[2 * i + 1, :, (13 * i) % 512] < 0         # the score is -inf, or +inf
            assert torch.isnan(b[~down]).all() and torch.isfinite(lse[2 * i + 1][down]).all()
            want = torch.zeros((heads, 512), dtype=torch.bool)
            want[:, (13 * i) % 512] = True
            assert torch.equal(torch.isnan(b)[down], want[down])
