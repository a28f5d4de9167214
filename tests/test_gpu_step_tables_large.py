"""Serving-step tables of so many rows that a workgroup passes its share of them
more than once (more than 2048 rows a workgroup), against the same built request
by request.  Whole numbers: everything has to be equal."""
import numpy as np
import pytest

from layer_oracle import step_tables_plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import gated_deltanet_dual_amd as g
    g.lib()
    return g


@pytest.mark.parametrize("page,longest,pad", [(16, 60000, 1), (1, 2000, 513), (48, 60000, 400000)])
def test_tables_of_more_than_a_million_rows(g, page, longest, pad):
    import torch
    rng = np.random.default_rng(page)
    R = 1300
    held, new = rng.integers(0, 100, R), rng.integers(0, 2000, R)
    new[::9] = 0            # requests that add nothing
    new[333] = longest      # one that fills many workgroups alone
    held[5], new[5] = 0, 0
    width = int((-(-(held + new) // page)).max())
    ids = rng.permutation(3 * 10 ** 6)[:int((-(-(held + new) // page)).sum()) + 5].astype(np.int32)
    table = np.full((R, width), -3, np.int32)
    at = 0
    for r in range(R):
        have = -(-int(held[r]) // page)
        table[r, :have] = ids[at:at + have]
        at += have
    M = int(new.sum()) + pad
    assert M > 1100000
    dev = lambda x: torch.from_numpy(np.asarray(x, np.int32)).cuda()  # noqa: E731
    bt = dev(table)
    got = g.step_tables(dev(held), dev(new), bt, dev(ids[at:]), dev([2]), page, M, position_offset=7)
    assert int(got["status"]) == g.TABLES_OK
    want = step_tables_plain(held, new, table, ids[at:], 2, page, M, 7)
    for name in ("cu_new", "positions", "slots", "seq_lens", "pages_used"):
        assert np.array_equal(got[name].cpu().numpy(), np.asarray(want[name])), name
    assert np.array_equal(bt.cpu().numpy(), np.asarray(want["block_table"]))
