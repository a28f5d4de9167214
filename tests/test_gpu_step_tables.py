"""The tables of a serving step against the same built request by request.
Whole numbers: everything has to be equal."""
import numpy as np
import pytest

from layer_oracle import step_tables_plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import gated_deltanet_dual_amd as g
    g.lib()
    return g


def dev(x):
    import torch
    return torch.tensor(x, dtype=torch.int32).cuda()


def make(seed, R, held, new, page):
    rng = np.random.default_rng(seed)
    h, n = rng.integers(0, held + 1, R), rng.integers(0, new + 1, R)
    width = max(1, -(-(held + new) // page))
    ids = rng.permutation(R * width * 2 + 9).astype(np.int32)
    return h, n, ids[:R * width].reshape(R, width).copy(), ids[R * width:].copy()


@pytest.mark.parametrize("R,held,new,page,offset", [(1, 0, 1, 16, 0), (1, 5, 0, 4, 7), (7, 40, 9, 16, 100), (300, 200, 4, 64, 0),
                                                    (513, 0, 70, 1, 3), (64, 33, 33, 33, 0), (5, 0, 2900, 256, 0), (8192, 3, 2, 2, 0)])
def test_tables(g, R, held, new, page, offset):
    import torch
    h, n, table, free = make(R + page, R, held, new, page)
    total = int(n.sum())
    for pad in (0, 1, 1500):
        M = total + pad
        want = step_tables_plain(h, n, table, free, 2, page, M, offset)
        bt = dev(table)
        lens = dev(h)
        got = g.step_tables(lens, dev(n), bt, dev(free), dev([2]), page, M, position_offset=offset)
        torch.cuda.synchronize()
        assert int(got["status"]) == g.TABLES_OK
        for name in ("cu_new", "positions", "slots", "seq_lens", "pages_used"):
            assert got[name].cpu().tolist() == want[name], name
        assert bt.cpu().tolist() == want["block_table"]
        assert lens.cpu().tolist() == list(h)


def test_no_requests(g):
    got = g.step_tables(dev([]), dev([]), dev(np.zeros((0, 4), np.int32)), dev([]), dev([0]), 16, 5)
    assert got["cu_new"].cpu().tolist() == [0] and got["slots"].cpu().tolist() == [-1] * 5 and int(got["status"]) == 0


def refused(g, why, h, n, table, free, used, page, M):
    """Status `why`; nothing allocated, nothing changed, every slot -1."""
    bt = dev(table)
    got = g.step_tables(dev(h), dev(n), bt, dev(free), dev([used]), page, M)
    assert int(got["status"]) == why
    assert got["cu_new"].cpu().tolist() == [0] * (len(h) + 1)
    assert got["slots"].cpu().tolist() == [-1] * M and got["positions"].cpu().tolist() == [0] * M
    assert got["seq_lens"].cpu().tolist() == list(h) and int(got["pages_used"]) == used
    assert bt.cpu().tolist() == np.asarray(table).tolist()


def test_refused_steps_change_nothing(g):
    table = np.arange(8).reshape(2, 4)
    free = np.arange(100, 110)
    refused(g, g.TABLES_NO_PAGES, [3, 4], [2, 1], table, free, 9, 4, 8)     # two pages opened, one free
    refused(g, g.TABLES_TOO_MANY_TOKENS, [3, 4], [5, 4], table, free, 0, 4, 8)
    refused(g, g.TABLES_TOO_LONG, [3, 14], [1, 3], table, free, 0, 4, 8)
    refused(g, g.TABLES_TOO_LONG, [2 ** 31 - 1, 0], [2 ** 31 - 1, 1], table, free, 0, 4, 8)
    refused(g, g.TABLES_BAD_LENGTH, [3, -1], [1, 3], table, free, 0, 4, 8)
    refused(g, g.TABLES_BAD_LENGTH, [3, 1], [-2 ** 31, 3], table, free, 0, 4, 8)
    refused(g, g.TABLES_BAD_LENGTH, [3, 1], [1, 1], table, free, -1, 4, 8)
    refused(g, g.TABLES_NO_PAGES, [3, 1], [2, 1], table, free, 2 ** 31 - 1, 4, 8)


def test_steps_in_a_row(g):
    """A serving loop: each step's lengths and pages_used feed the next; every
    live token of every request keeps a slot of its own."""
    import torch
    R, page, width = 9, 8, 12
    lens, used, bt = dev([0] * R), dev([0]), dev(np.full((R, width), -7))
    free = dev(np.random.default_rng(1).permutation(R * width))
    seen = {}
    for step in range(6):
        n = [(r * 5 + step * 3) % 11 for r in range(R)]
        t = g.step_tables(lens, dev(n), bt, free, used, page, 128)
        assert int(t["status"]) == 0
        cu, slots, pos = (t[k].cpu().tolist() for k in ("cu_new", "slots", "positions"))
        for r in range(R):
            for i in range(cu[r], cu[r + 1]):
                assert slots[i] not in seen.values()
                seen[(r, pos[i])] = slots[i]
        lens, used = t["seq_lens"], t["pages_used"]
    table = bt.cpu().tolist()
    assert all(table[r][p // page] * page + p % page == s for (r, p), s in seen.items())
    assert len(seen) == int(lens.sum()) and torch.equal(used, dev([sum(-(-int(x) // page) for x in lens.cpu())]))
