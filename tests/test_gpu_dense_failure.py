"""The device error path of the dense latent attentions, without faulting or hanging the GPU: as
in test_gpu_failure.py one plain thread arrival is withheld (DSA_TEST_SKIP_ARRIVAL; no TMA, bulk copy or tensor-core
operation completes that barrier) under a short wait budget.  The bounded waits run out, every copy and
product in flight is waited for, the host reads DSA_ERR_DEVICE_TIMEOUT, and the next call is right."""

import pytest
import torch

import long_context_sparse_lightning_b200 as dsa
from tests.dense_ref import Case, check
from tests.test_gpu_expanded_mla import Expanded

pytestmark = pytest.mark.gpu


def withheld(monkeypatch, call, ws, sites):
    monkeypatch.setenv("DSA_WAIT_BUDGET_CYCLES", "20000000")     # ~10 ms per bounded wait
    monkeypatch.setenv("DSA_TEST_SKIP_ARRIVAL", "0")
    call()
    with pytest.raises(dsa.DSAError) as e:
        dsa.check_device_error(ws)
    assert e.value.status == 5                                   # DSA_ERR_DEVICE_TIMEOUT
    assert e.value.site in sites
    dsa.check_device_error(ws)                                   # read and cleared; the context is usable
    monkeypatch.delenv("DSA_TEST_SKIP_ARRIVAL")
    monkeypatch.delenv("DSA_WAIT_BUDGET_CYCLES")


@pytest.mark.parametrize("seqs,heads,sites", [
    (500, 16, range(510, 536)),                                  # items of 16 rows, of 32, and of a CTA pair
    (500, 24, range(510, 536)),
    (200, 64, range(550, 589)),
])
def test_a_wait_that_runs_out_in_the_absorbed_form(monkeypatch, seqs, heads, sites):
    # more items than CTAs (pairs): the first one's second product waits for the withheld release
    c = Case([1] * seqs, [100 + i % 90 for i in range(seqs)], heads, 64, seed=31)
    ws = dsa.workspace(dsa.OP_DENSE_MLA, c.batch, n_heads=heads)
    withheld(monkeypatch, lambda: c.dense(ws=ws, check=False), ws, sites)
    out, lse = c.dense(ws=ws)
    check(out, lse, c.exact_dense(), c.rows)


@pytest.mark.parametrize("q,kv,heads", [
    ([300], [700], 4),                                           # split keys, two row tiles, two heads a block
    ([1000], [1000], 3),
    ([100] * 4, [500] * 4, 128),
])
def test_a_wait_that_runs_out_in_the_expanded_form(monkeypatch, q, kv, heads):
    c = Expanded(q, kv, heads, seed=32)
    args = c.q.cuda(), c.up.cuda(), c.cache.cuda()[:, 512:]
    out, lse = c.outputs(128)
    ws = dsa.workspace(dsa.OP_EXPANDED_MLA, c.batch, n_heads=heads)
    call = lambda: dsa.expanded_mla(c.batch, *args, c.scale, out, lse, ws)  # noqa: E731
    withheld(monkeypatch, call, ws, range(610, 644))
    call()
    dsa.check_device_error(ws)
    check(out.cpu(), lse.cpu(), c.exact_expanded(), c.rows)
