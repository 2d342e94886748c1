"""Block tables, offsets, positions and slots built on the device (dsa_page_tables)
against plain loops."""

import numpy as np
import pytest
import torch

import long_context_sparse_lightning_b200 as dsa

pytestmark = pytest.mark.gpu


def plain(q, before, free, page, table, cap):
    table, free = table.copy(), list(free)
    cu, pos, slots, used = [0], [], [], 0
    for b, (n, pre) in enumerate(zip(q, before)):
        for p in range(pre, pre + n):
            if p % page == 0:
                table[b][p // page] = free[used]
                used += 1
            pos.append(p)
            slots.append(int(table[b][p // page]) * page + p % page)
        cu.append(cu[-1] + n)
    pos += [0] * (cap - len(pos))
    slots += [-1] * (cap - len(slots))
    return table, cu, [n + p for n, p in zip(q, before)], pos, slots, used


def setup(q, before, page, pad, seed, extra_blocks=1):
    rng = np.random.default_rng(seed)
    n = len(q)
    have = [-(-x // page) for x in before]
    blocks = max(-(-(x + y) // page) for x, y in zip(q, before)) + extra_blocks
    need = sum(-(-(x + y) // page) - h for x, y, h in zip(q, before, have))
    ids = rng.permutation(sum(have) + need + 4).astype(np.int32)
    table = np.full((n, blocks), -1, np.int32)
    k = 0
    for b in range(n):
        table[b, :have[b]] = ids[k:k + have[b]]
        k += have[b]
    return table, ids[k:], sum(q) + pad


class Call:
    def __init__(self, q, before, page, table, free, cap):
        i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        n = len(q)
        self.q, self.before, self.free, self.page = i(q), i(before), i(free), page
        self.table = torch.from_numpy(table.copy()).cuda()
        self.cu, self.kv, self.used = i([-9] * (n + 1)), i([-9] * n), i([-9])
        self.pos = i([-9] * cap)
        self.slots = torch.full((cap,), -9, dtype=torch.int64, device="cuda")
        self.ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def run(self):
        dsa.page_tables(self.q, self.before, self.free, self.page, self.table, self.cu, self.kv, self.pos, self.slots,
                        self.used, self.ws)
        return self


CASES = [
    ([1], [0], 64, 0),
    ([0], [0], 64, 3),
    ([1, 1, 1], [63, 64, 65], 64, 2),
    ([200, 0, 1, 130], [5, 64, 0, 62], 64, 0),
    ([1] * 300, [i * 37 for i in range(300)], 128, 12),
    ([3] * 255 + [9000, 1], [i for i in range(257)], 64, 100),
    ([(i * 7) % 5 for i in range(1000)], [(i * 131) % 3000 for i in range(1000)], 256, 0),
]


@pytest.mark.parametrize("q,before,page,pad", CASES)
def test_against_plain_loops(q, before, page, pad):
    table, free, cap = setup(q, before, page, pad, seed=1)
    c = Call(q, before, page, table, free, cap).run()
    dsa.check_device_error(c.ws)
    t, cu, kv, pos, slots, used = plain(q, before, free, page, table, cap)
    assert np.array_equal(c.table.cpu().numpy(), t)
    assert c.cu.tolist() == cu and c.kv.tolist() == kv
    assert c.pos.tolist() == pos and c.slots.tolist() == slots
    assert c.used.tolist() == [used]


def test_too_few_pages():
    q, before, page = [100, 200], [0, 30], 64
    table, free, cap = setup(q, before, page, 0, seed=2)
    c = Call(q, before, page, table, free[:3], cap).run()
    with pytest.raises(dsa.DSAError) as e:
        dsa.check_device_error(c.ws)
    assert e.value.status == 6
    t, cu, kv, pos, slots, used = plain(q, before, free, page, table, cap)
    assert c.cu.tolist() == cu and c.pos.tolist() == pos and c.used.tolist() == [3]
    # sequence 0 takes two pages, sequence 1 the third, and has no page from position 128 on
    assert c.slots.tolist()[:100 + 98] == slots[:198]
    assert c.slots.tolist()[198:] == [-1] * (cap - 198)


def test_bad_lengths_take_no_tokens():
    q, before, page = [2, -3, 5, 10 ** 9], [1, 4, 6, 2 ** 31 - 5], 64
    table = np.full((4, 3), 0, np.int32)
    c = Call(q, before, page, table, [7, 8], 10).run()
    with pytest.raises(dsa.DSAError) as e:
        dsa.check_device_error(c.ws)
    assert e.value.status == 6
    assert c.cu.tolist() == [0, 2, 2, 7, 7]
    assert c.pos.tolist() == [1, 2, 6, 7, 8, 9, 10, 0, 0, 0]
    assert c.slots.tolist() == [1, 2, 6, 7, 8, 9, 10, -1, -1, -1]
    assert np.array_equal(c.table.cpu().numpy(), table)


def test_more_tokens_than_rows():
    q, before, page = [5, 6], [0, 0], 64
    table, free, cap = setup(q, before, page, 0, seed=3)
    c = Call(q, before, page, table, free, 8).run()
    with pytest.raises(dsa.DSAError):
        dsa.check_device_error(c.ws)
    assert c.cu.tolist() == [0, 5, 8] and c.pos.tolist() == [0, 1, 2, 3, 4, 0, 1, 2]


def test_no_rows_at_all():
    table, free, cap = setup([0, 0], [70, 3], 64, 0, seed=4)
    c = Call([0, 0], [70, 3], 64, table, free, 0).run()
    dsa.check_device_error(c.ws)
    assert c.cu.tolist() == [0, 0, 0] and c.kv.tolist() == [70, 3] and c.used.tolist() == [0]
