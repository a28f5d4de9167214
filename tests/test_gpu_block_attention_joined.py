"""Block attention whose parts are joined by the second launch: captured and replayed,
on two streams at once, pages that several requests share, and keys by the hundred
thousand.  Tolerances as derived for the block attention; sums of more keys only add
fp32 steps of the sum's own size (2^17 keys in parts of at most 4096: chains of at most
512 tiles and 32 parts, 544 * 2^-24 < 4e-5, inside the 4e-4 allowed)."""
import math

import pytest

from layer_oracle import attention64, close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import gated_deltanet_dual_amd as g
    g.lib()
    return g


def make(seed, R, B, Hk, G, d, page, lens, prefix, pages=None):
    """Every request's pages and the prefix's taken from a cache of `pages` (default:
    as many as all need), one after the other and round again."""
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    wide, shared = max(-(-n // page) for n in lens) + 1, -(-prefix // page)
    pages = pages or R * wide + shared
    ids = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    ids = ids.repeat(-(-(R * wide + shared) // pages))
    return (rnd(R, B, Hk * G, d), rnd(pages, Hk, page, d), rnd(pages, Hk, page, d),
            ids[shared:shared + R * wide].reshape(R, wide).contiguous(), torch.tensor(lens, dtype=torch.int32).cuda(),
            ids[:shared].contiguous())


def check(g, args, prefix, causal):
    import torch
    q, kc, vc, bt, lens, pt = args
    o = g.block_attention(q, kc, vc, bt, lens, prefix_table=pt, prefix_len=prefix, causal=causal)
    torch.cuda.synchronize()
    ro, _, size = attention64(q, kc, vc, bt, lens, pt, prefix, causal)
    close(o, ro, torch.bfloat16, (2.0 ** -8 + 4e-4) * size, "o")


SHAPES = [(6, 4, 2, 4, 128, 16, [40, 0, 300, 4, 1000, 77], 4500), (3, 7, 1, 8, 256, 32, [700, 7, 60], 3000),
          (2, 1, 4, 4, 64, 64, [5000, 1], 0)]


@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_captured_and_replayed(g, i):
    """Every replay, on new inputs and lengths and with eager work between, gives the
    eager call's bits; so do two graphs that share a memory pool, one after the other."""
    import torch
    R, B, Hk, G, d, page, lens, prefix = SHAPES[i]
    assert g.block_attention_workspace_bytes(R, B, Hk * G, Hk, d, page, (max(-(-n // page) for n in lens) + 1) * page, prefix) > 0
    static = make(1, *SHAPES[i])
    call = lambda a, causal: g.block_attention(*a[:5], prefix_table=a[5], prefix_len=prefix, causal=causal, want_lse=True)  # noqa: E731
    call(static, False)
    torch.cuda.synchronize()
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        got1 = call(static, False)
    with torch.cuda.graph(second, pool=first.pool()):
        got2 = call(static, True)
    for rep in range(4):
        new = list(make(10 + rep, *SHAPES[i]))
        new[4] = new[4].roll(rep)  # the lengths' order; every table row is as wide
        for a, b in zip(static, new):
            a.copy_(b)
        want1, want2 = call(static, False), call(static, True)
        junk = torch.randn(1 << 18, device="cuda").sum()
        torch.cuda.synchronize()
        first.replay()
        second.replay()
        torch.cuda.synchronize()
        assert float(junk) == float(junk)
        for got, want in ((got2, want2), (got1, want1)):
            assert all(torch.equal(a, b) for a, b in zip(got, want)), rep


def test_two_streams_at_once(g):
    """Calls under way together, each with its own workspace, give the bits of one after
    the other."""
    import torch
    sets = [make(20 + i, *s) for i, s in enumerate(SHAPES[:2])]
    pre = [s[-1] for s in SHAPES[:2]]
    call = lambda k: g.block_attention(*sets[k][:5], prefix_table=sets[k][5], prefix_len=pre[k], causal=True)  # noqa: E731
    want = [call(0), call(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [[], []]
        for _ in range(6):
            for k, s in enumerate(streams):
                with torch.cuda.stream(s):
                    got[k].append(call(k))
        torch.cuda.synchronize()
        assert all(torch.equal(o, want[k]) for k in range(2) for o in got[k])


@pytest.mark.parametrize("causal", [False, True])
def test_pages_that_requests_share(g, causal):
    """Requests that forked from one another, the prefix too: the same pages in several
    rows of the table."""
    check(g, make(30, 5, 3, 2, 2, 128, 16, [200, 90, 0, 333, 33], 1000, pages=40), 1000, causal)


@pytest.mark.parametrize("d,prefix,lens", [(64, 131072, [3, 700]), (128, 40001, [70000]), (256, 0, [33333, 5])])
def test_many_keys(g, d, prefix, lens):
    """Against sums in 64 bits on the GPU."""
    import torch
    R, B, Hk, G, page = len(lens), 2, 1, 2, 64
    q, kc, vc, bt, sl, pt = make(40, R, B, Hk, G, d, page, lens, prefix)
    o, lse = g.block_attention(q, kc, vc, bt, sl, prefix_table=pt, prefix_len=prefix, causal=True, want_lse=True)
    rows = lambda c, t, n: c[t.long()].transpose(1, 2).reshape(-1, d)[:n].double()  # noqa: E731  (one kv head)
    for r, n in enumerate(lens):
        k, v = (torch.cat([rows(c, pt, prefix), rows(c, bt[r], n)]) for c in (kc, vc))
        for b in range(B):
            m = prefix + max(0, n - (B - 1 - b))
            for h in range(G):
                s = (k[:m] * q[r, b, h].double()).sum(1) / math.sqrt(d)
                p = torch.softmax(s, 0)[:, None]
                close(o[r, b, h], (p * v[:m]).sum(0).cpu(), torch.bfloat16, (2.0 ** -8 + 4e-4) * (p * v[:m].abs()).sum(0).cpu(),
                      "request %d query %d head %d" % (r, b, h))
                assert abs(float(lse[r, b, h]) - float(torch.logsumexp(s, 0))) <= 5e-4
