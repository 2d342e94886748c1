"""Infinities that a query does see, in the expanded latent attention: a key of score -inf has weight 0, a
value that is not finite makes the output NaN in its dim (dsa.h), wherever the tiles, the blocks and the parts
of a split end."""

import pytest
import torch

from tests.dense_ref import compare_nonfinite
from tests.test_gpu_expanded_mla import Expanded

pytestmark = pytest.mark.gpu
INF = float("inf")


def expanded(c):
    def kv(b, h):
        up = c.up[c.at[b], h].double()
        return torch.cat([up[:, :128], c.cache[c.at[b], 512:].double()], -1), up[:, 128:]
    return kv


EXPANDED = [
    # (q_len, kv_len, heads): blocks of one head, of two, and split keys
    ([300], [300], 1),
    ([100] * 4, [300, 130, 100, 260], 96),
    ([20], [3000], 2),
    ([270], [1300], 1),
]


@pytest.mark.parametrize("q,kv,heads", EXPANDED)
@pytest.mark.parametrize("kind", ["inf", "-inf", "both", "nan"])
def test_values_that_are_not_finite_are_nan_in_every_tile(q, kv, heads, kind):
    c = Expanded(q, kv, heads, seed=24)
    want = c.exact_expanded()[0]
    h, n, first = heads - 1, q[0], kv[0] - q[0]
    at = c.at[0]
    values = {"inf": (INF, INF), "-inf": (-INF, -INF), "both": (INF, -INF), "nan": (float("nan"), INF)}[kind]
    c.up[at[10], h, 128 + 4] = values[0]             # a tile that some rows' blocks have in their inside, some on the border
    c.up[at[-3], h, 128 + 70] = values[0]            # the border of the last rows
    c.up[at[40], h, 128 + 4] = values[1]
    out, lse = c.run()
    bad = torch.zeros(out.shape, dtype=torch.bool)
    for i in range(n):
        bad[i, h, 4] = first + i >= 10
        bad[i, h, 70] = first + i >= kv[0] - 3
    assert torch.equal(torch.isnan(out.float()), bad)
    assert torch.isfinite(out[~bad].float()).all() and torch.isfinite(lse[:c.rows]).all()
    d = (out.double() - want)[~bad]
    assert d.norm() <= 2.0 ** -8 * want[~bad].norm()


@pytest.mark.parametrize("q,kv,heads,bad", [([10], [400], 1, range(0, 256)), ([30], [3000], 2, range(2000, 2900)),
                                            ([100] * 4, [300] * 4, 96, range(0, 128)), ([5], [2000], 1, [1998])])
def test_keys_of_score_minus_infinity_have_no_weight(q, kv, heads, bad):
    c = Expanded(q, kv, heads, seed=25)
    h = heads - 1
    c.up[c.at[0][list(bad)], h, 5] = INF
    c.q[:q[0], h, 5] = -1.0
    out, lse = c.run()
    c.q_len, c.kv_len, c.q = q[:1], kv[:1], c.q[:q[0], h:]
    full, c.heads = expanded(c), 1
    assert compare_nonfinite(c, out[:q[0], h:], lse[:q[0], h:], lambda b, _: full(b, h)) == 0


@pytest.mark.parametrize("n,kv", [(10, 400), (10, 100), (10, 3000), (300, 900)])
def test_expanded_rows_whose_scores_are_all_minus_infinity(n, kv):
    c = Expanded([n], [kv], 1, seed=26)
    c.up[c.at[0], :, 5] = INF
    c.q[:, :, 5] = -1.0
    c.up[c.at[0][3], 0, 128 + 9] = INF
    out, lse = c.run()
    assert torch.isneginf(lse[:n]).all()
    seen = torch.arange(n) + kv - n >= 3
    assert torch.equal(torch.isnan(out[:n, 0, 9].float()), seen)
    rest = torch.cat([out[:n, 0, :9], out[:n, 0, 10:]], -1)
    assert (rest == 0).all()
