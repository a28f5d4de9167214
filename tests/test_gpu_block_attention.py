"""The block attention over pages and a shared prefix against softmax sums in
64 bits.  Tolerances, per output: its last rounding (half a bf16 step of it); the
weights p are rounded to bf16 before the second product, half a step each, which
moves the output by at most 2^-8 * sum p |v| / sum p (the reference gives that sum);
scores are exact bf16 products summed in fp32 over d <= 256 channels, of size <=
16 here, so p is off by at most 16 * 256 * 2^-24 = 2.5e-4 of itself at the very worst,
and its exponential and the sums by far less: 4e-4 of the same sum for all of it."""
import math

import numpy as np
import pytest

from layer_oracle import attention64, close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import gated_deltanet_dual_amd as g
    g.lib()
    return g


def make(seed, R, B, Hk, G, d, page, lens, prefix, fill=float("nan"), kscale=1.0):
    """Caches whose rows behind the lengths hold `fill`, and unreached table
    entries that name no page."""
    import torch
    gen = torch.Generator().manual_seed(seed)
    width = max(1, max(-(-n // page) for n in lens)) + 1
    shared = -(-prefix // page)
    need = [-(-max(0, n) // page) for n in lens]
    pages = sum(need) + shared + 2
    ids = torch.randperm(pages, generator=gen).tolist()
    kc = torch.randn(pages, Hk, page, d, generator=gen) * kscale
    vc = torch.randn(pages, Hk, page, d, generator=gen)
    bt = torch.full((R, width), 2 ** 30, dtype=torch.int32)
    used = torch.zeros(pages, page, dtype=torch.bool)
    pt = torch.tensor([ids.pop() for _ in range(shared)], dtype=torch.int32)
    for j in range(prefix):
        used[int(pt[j // page]), j % page] = True
    for r, n in enumerate(lens):
        for p in range(need[r]):
            bt[r, p] = ids.pop()
        for j in range(max(0, n)):
            used[int(bt[r, j // page]), j % page] = True
    dead = ~used
    kc.transpose(1, 2)[dead] = fill
    vc.transpose(1, 2)[dead] = fill
    q = torch.randn(R, B, Hk * G, d, generator=gen)
    bf = lambda t: t.to(torch.bfloat16).cuda()  # noqa: E731
    return bf(q), bf(kc), bf(vc), bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), pt.cuda()


def check(g, args, prefix, causal, **more):
    import torch
    q, kc, vc, bt, lens, pt = args
    o, lse = g.block_attention(q, kc, vc, bt, lens, prefix_table=pt, prefix_len=prefix, causal=causal, want_lse=True, **more)
    torch.cuda.synchronize()
    ro, rl, size = attention64(q, kc, vc, bt, lens, pt, prefix, causal, more.get("scale"))
    close(o, ro, torch.bfloat16, (2.0 ** -8 + 4e-4) * size, "o")
    fin = torch.isfinite(rl)
    assert torch.equal(torch.isfinite(lse.cpu()), fin) and (lse.cpu()[~fin] == -math.inf).all()
    assert float((lse.cpu().double() - rl)[fin].abs().max() if fin.any() else 0) <= 5e-4
    return o, lse


CASES = [
    # R, B, Hk, G, d, page, lens, prefix
    (1, 1, 1, 1, 64, 16, [1], 0),
    (1, 1, 1, 1, 128, 16, [17], 0),
    (1, 1, 4, 4, 128, 64, [700], 0),
    (3, 4, 2, 4, 128, 64, [0, 5, 200], 0),
    (3, 4, 2, 4, 128, 16, [1, 33, 130], 77),
    (4, 1, 1, 8, 256, 32, [15, 16, 31, 32], 1),
    (2, 7, 2, 8, 256, 16, [9, 300], 250),
    (5, 3, 1, 5, 64, 128, [3, 64, 127, 128, 129], 129),
    (2, 16, 1, 8, 64, 32, [16, 47], 40),
    (2, 32, 2, 1, 128, 32, [32, 90], 0),
    (6, 2, 1, 2, 128, 16, [0, 0, 2, 0, 1, 40], 513),
    (2, 1, 1, 1, 64, 16, [0, 0], 0),
    (2, 2, 1, 3, 128, 16, [0, 0], 30),
    (1, 1, 1, 2, 64, 16, [4500], 0),
    (40, 2, 1, 2, 64, 32, [(i * 37) % 90 for i in range(40)], 300),
    # prefixes long and wide enough for shared tiles, in one part and in several, ending inside a tile and a page
    (40, 2, 2, 2, 128, 16, [(i * 11) % 50 for i in range(40)], 333),
    (9, 8, 1, 3, 128, 64, [8 + i for i in range(9)], 64),
    (9, 8, 1, 3, 128, 64, [8 + i for i in range(9)], 1),
    (30, 4, 1, 2, 128, 32, [4] * 30, 1500),
    (33, 2, 1, 2, 256, 16, [(i * 7) % 40 for i in range(33)], 700),
    (64, 1, 1, 1, 64, 16, [0] * 64, 1000),
    (13, 1, 1, 8, 128, 128, [0] * 13, 200),
    # prefixes too long for one part with the own keys: shared by the requests' rows, few and many, parts joined
    (3, 2, 2, 2, 128, 16, [0, 33, 70], 4100),
    (9, 8, 1, 3, 128, 64, [8 + 9 * i for i in range(9)], 4200),
    (20, 2, 1, 4, 64, 32, [(i * 17) % 60 for i in range(20)], 4300),
    (5, 4, 1, 4, 256, 16, [4, 0, 16, 37, 300], 2100),
    (2, 20, 1, 8, 128, 32, [20, 131], 5000),
    (1, 1, 1, 1, 64, 16, [1], 4097),
]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_attention(g, i, causal):
    R, B, Hk, G, d, page, lens, prefix = CASES[i]
    check(g, make(i, R, B, Hk, G, d, page, lens, prefix), prefix, causal)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,Hk,prefix", [(64, 2, 0), (64, 2, 200), (128, 2, 77), (128, 2, 4130), (128, 1, 0)])
def test_many_requests_with_many_rows(g, d, Hk, prefix, causal):
    """Enough rows in all that a wave takes two tiles of them (Hk = 2: 260 workgroups of
    80 rows; Hk = 1: one below), own keys from none to several tiles."""
    R, B, G = 130, 20, 4
    check(g, make(11, R, B, Hk, G, d, 16, [(i * 29) % 150 for i in range(R)], prefix), prefix, causal)


def test_sharp_scores_and_scale(g):
    """Scores far apart (the running maximum moves, weights vanish) and a scale of
    the caller's own."""
    args = make(3, 2, 2, 1, 2, 64, 16, [100, 333], 70, kscale=6.0)
    check(g, args, 70, False)
    check(g, args, 70, True, scale=0.03125)


def test_rows_beyond_the_bound_are_cut(g):
    """max_seq_len bounds the lengths: longer ones are read up to it."""
    import torch
    args = make(4, 3, 2, 1, 2, 64, 16, [40, 20, 64], 0)
    o = g.block_attention(*args[:5], max_seq_len=32)
    cut = list(args)
    cut[4] = args[4].clamp(max=32)
    ro, _, size = attention64(*cut[:5], None, 0, False)
    close(o, ro, torch.bfloat16, (2.0 ** -8 + 4e-4) * size, "o")
    zero = g.block_attention(*args[:5], max_seq_len=0)
    assert (zero == 0).all()


def test_result_does_not_depend_on_the_batch(g):
    """A request alone and in a batch with another bound: the parts differ, the
    result by rounding only."""
    import torch
    args = make(5, 3, 4, 2, 4, 128, 32, [500, 61, 7], 90)
    q, kc, vc, bt, lens, pt = args
    whole = g.block_attention(q, kc, vc, bt, lens, prefix_table=pt, prefix_len=90)
    for r in range(3):
        one = g.block_attention(q[r:r + 1], kc, vc, bt[r:r + 1].contiguous(), lens[r:r + 1], prefix_table=pt, prefix_len=90)
        assert torch.allclose(one.float(), whole[r:r + 1].float(), rtol=2.0 ** -6, atol=2.0 ** -7)
    again = g.block_attention(q, kc, vc, bt, lens, prefix_table=pt, prefix_len=90)
    assert torch.equal(whole, again)


def test_values_that_are_not_finite(g):
    """Infinities and NaN in a value row reach exactly the queries that see its
    key: a later token of the block does not reach the earlier ones."""
    import torch
    for d, B, G in [(64, 5, 2), (128, 5, 4), (128, 20, 8), (256, 4, 1)]:
        args = make(7, 2, B, 1, G, d, 16, [40 + B, B], 70)
        q, kc, vc, bt, lens, pt = args
        clean = g.block_attention(q, kc, vc, bt, lens, prefix_table=pt, prefix_len=70, causal=True)
        bad = vc.clone()
        for r, n in enumerate([40 + B, B]):
            for back, value in ((1, float("inf")), (2, float("nan")), (3, float("-inf"))):
                j = n - back  # seen by the last `back` tokens of the block
                bad[int(bt[r, j // 16]), 0, j % 16, back] = value
        o = g.block_attention(q, kc, bad, bt, lens, prefix_table=pt, prefix_len=70, causal=True)
        for b in range(B):
            back = B - b  # this token sees keys up to n - back + 1
            for ch, value in ((1, math.inf), (2, None), (3, -math.inf)):
                got = o[:, b, :, ch]
                if ch < back:  # key n - ch lies behind this token's view
                    assert torch.equal(got, clean[:, b, :, ch]), (d, b, ch)
                elif value is None:
                    assert torch.isnan(got).all(), (d, b, ch)
                else:
                    assert (got == value).all(), (d, b, ch)
        assert torch.equal(o[..., 4:], clean[..., 4:]) and torch.equal(o[..., 0], clean[..., 0])


def test_extreme_scales(g):
    """A scale so small that all weights are equal, and one so large that the
    largest score takes all."""
    import torch
    q, kc, vc, bt, lens, pt = args = make(8, 2, 2, 1, 2, 64, 16, [50, 33], 20)
    o = g.block_attention(q, kc, vc, bt, lens, prefix_table=pt, prefix_len=20, scale=1e-36)
    ro, _, size = attention64(*args, 20, False, 1e-36)
    close(o, ro, torch.bfloat16, (2.0 ** -8 + 4e-4) * size, "o")
    o = g.block_attention(q, kc, vc, bt, lens, prefix_table=pt, prefix_len=20, scale=1e4)
    ro, _, size = attention64(*args, 20, False, 1e4)
    close(o, ro, torch.bfloat16, (2.0 ** -8 + 4e-4) * size, "o")


def test_table_entries_that_name_no_page_stay_inside(g):
    """Ids outside the cache read some page of it: finite numbers, no fault, and
    the other requests' results are untouched."""
    import torch
    q, kc, vc, bt, lens, pt = make(9, 3, 1, 2, 2, 128, 16, [40, 40, 40], 0, fill=0.0)
    want = g.block_attention(q, kc, vc, bt, lens)
    bt[1, 1] = -5
    bt[1, 2] = 2 ** 31 - 1
    o = g.block_attention(q, kc, vc, bt, lens)
    assert torch.isfinite(o.float()).all() and torch.equal(o[0], want[0]) and torch.equal(o[2], want[2])
