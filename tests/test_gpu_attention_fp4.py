"""The block attention over a cache in 4 bits against softmax sums in 64 bits over the
values that the codes stand for.  Tolerances, per output: its last rounding (half a bf16
step of it); the weights p are rounded to bf16 before the second product, half a step
each, which moves the output by at most 2^-8 * sum p |v| / sum p (the reference gives that
sum); keys and values are bf16 exactly, so scores are exact products summed in fp32 over
d <= 256 channels, of size <= 16 here: p is off by at most 16 * 256 * 2^-24 = 2.5e-4 of
itself at the very worst, and its exponential and the sums by far less: 4e-4 of the same
sum for all of it, 5e-4 for the logarithm of the sum."""
import math

import pytest

from layer_oracle import attention64, close
from softmax_oracle import cache_values, fp4_nearest, leaf, norm_rotary64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import gated_deltanet_dual_amd as g
    g.lib()
    return g


def to_cache(x, gen):
    """x [pages, heads, page, d] of the values that 4 bits hold, as (codes, scales); NaN
    where it is NaN: groups of any codes under a scale of 255."""
    import torch
    d = x.shape[-1]
    gx = x.reshape(*x.shape[:-1], d // 32, 32)
    top = gx.abs().amax(-1)
    fine = torch.isfinite(top)
    e = torch.frexp(torch.where(fine & (top > 0), top, 2.0 ** -126).double())[1].long() - 3
    e = (e + (top.nan_to_num() > 7 * torch.exp2(e.double()))).clamp(-126, 125)
    z = gx.double().abs() * torch.exp2(-e.double())[..., None]
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    code = torch.bucketize(z.nan_to_num(), mids) + 8 * (gx < 0)
    code = torch.where(fine[..., None], code, torch.randint(0, 16, code.shape, generator=gen)).flatten(-2)
    codes = (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)
    scales = torch.where(fine, e + 127, 255).to(torch.uint8).transpose(2, 3).contiguous()
    return codes.cuda(), scales.cuda()


def make(seed, R, B, Hk, G, d, page, lens, prefix, dead=True, kscale=1.0, values=None):
    """Caches whose rows behind the lengths are NaN (dead), and unreached table entries that
    name no page."""
    import torch
    gen = torch.Generator().manual_seed(seed)
    width = max(1, max(-(-n // page) for n in lens)) + 1
    shared = -(-prefix // page)
    need = [-(-max(0, n) // page) for n in lens]
    pages = sum(need) + shared + 2
    ids = torch.randperm(pages, generator=gen).tolist()
    kc = torch.randn(pages, Hk, page, d, generator=gen) * kscale
    vc = torch.randn(pages, Hk, page, d, generator=gen) * torch.exp2(torch.randint(-3, 3, (pages, Hk, page, 1), generator=gen))
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
    if dead:
        kc.transpose(1, 2)[~used] = math.nan
        vc.transpose(1, 2)[~used] = math.nan
    q = torch.randn(R, B, Hk * G, d, generator=gen)
    return (q.to(torch.bfloat16).cuda(), to_cache(kc, gen), to_cache(vc, gen), bt.cuda(),
            torch.tensor(lens, dtype=torch.int32).cuda(), pt.cuda())


def check(g, args, prefix, causal, **more):
    import torch
    q, kc, vc, bt, lens, pt = args
    o, lse = g.block_attention_fp4(q, kc, vc, bt, lens, prefix_table=pt, prefix_len=prefix, causal=causal, want_lse=True, **more)
    torch.cuda.synchronize()
    ro, rl, size = attention64(q, cache_values(*kc), cache_values(*vc), bt, lens, pt, prefix, causal, more.get("scale"))
    close(o, ro, torch.bfloat16, (2.0 ** -8 + 4e-4) * size, "o")
    fin = torch.isfinite(rl)
    assert torch.equal(torch.isfinite(lse.cpu()), fin) and (lse.cpu()[~fin] == -math.inf).all()
    assert float((lse.cpu().double() - rl)[fin].abs().max() if fin.any() else 0) <= 5e-4
    return o, lse


CASES = [
    # R, B, Hk, G, d, page, lens, prefix
    (1, 1, 1, 1, 64, 16, [1], 0),
    (1, 1, 1, 1, 128, 16, [17], 0),
    (1, 1, 1, 1, 256, 16, [33], 0),
    (1, 1, 4, 4, 128, 64, [700], 0),
    (3, 4, 2, 4, 128, 64, [0, 5, 200], 0),
    (3, 4, 2, 4, 128, 16, [1, 33, 130], 77),
    (4, 1, 1, 8, 256, 32, [15, 16, 31, 32], 1),
    (2, 7, 2, 8, 256, 16, [9, 300], 250),
    (5, 3, 1, 5, 64, 128, [3, 64, 127, 128, 129], 129),
    (2, 16, 1, 8, 64, 32, [16, 47], 40),
    (2, 32, 2, 1, 128, 32, [32, 90], 0),
    (2, 9, 2, 2, 128, 16, [9, 90], 31),
    (6, 2, 1, 2, 128, 16, [0, 0, 2, 0, 1, 40], 513),
    (2, 1, 1, 1, 64, 16, [0, 0], 0),
    (2, 2, 1, 3, 128, 16, [0, 0], 30),
    (1, 1, 1, 2, 64, 16, [4500], 0),
    (2, 5, 1, 5, 64, 16, [200, 3], 0),
    (40, 2, 1, 2, 64, 32, [(i * 37) % 90 for i in range(40)], 300),
    (40, 2, 2, 2, 128, 16, [(i * 11) % 50 for i in range(40)], 333),
    (9, 8, 1, 3, 128, 64, [8 + i for i in range(9)], 64),
    (9, 8, 1, 3, 128, 64, [8 + i for i in range(9)], 1),
    (30, 4, 1, 2, 128, 32, [4] * 30, 1500),
    (33, 2, 1, 2, 256, 16, [(i * 7) % 40 for i in range(33)], 700),
    (64, 1, 1, 1, 64, 16, [0] * 64, 1000),
    # prefixes too long for one part with the own keys: shared by the requests' rows, few and many, parts joined
    (1, 1, 1, 4, 128, 16, [70], 4200),
    (3, 2, 2, 2, 128, 16, [0, 33, 70], 4100),
    (2, 3, 1, 4, 256, 16, [70, 5], 4100),
    (9, 8, 1, 3, 128, 64, [8 + 9 * i for i in range(9)], 4200),
    (20, 2, 1, 4, 64, 32, [(i * 17) % 60 for i in range(20)], 4300),
    (5, 4, 1, 4, 256, 16, [4, 0, 16, 37, 300], 4100),
    (2, 20, 1, 8, 128, 32, [20, 131], 5000),
    (3, 9, 1, 3, 64, 32, [20, 0, 131], 4500),
    (1, 1, 1, 1, 64, 16, [1], 4097),
    # a short prefix before more own keys than a part of shared tiles holds
    (40, 1, 1, 2, 256, 64, [2500] + [40] * 39, 100),
    (40, 1, 1, 2, 128, 64, [3900] + [40] * 39, 100),
    (3, 40, 1, 1, 128, 64, [3900, 40, 41], 150),
    (3, 40, 1, 1, 256, 64, [1900, 40, 41], 100),
]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_attention(g, i, causal):
    R, B, Hk, G, d, page, lens, prefix = CASES[i]
    check(g, make(i, R, B, Hk, G, d, page, lens, prefix), prefix, causal)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,Hk,prefix", [(64, 2, 0), (64, 2, 200), (128, 2, 77), (128, 2, 4130), (128, 1, 0), (256, 1, 50)])
def test_many_requests_with_many_rows(g, d, Hk, prefix, causal):
    R, B, G = 130, 20, 4
    check(g, make(11, R, B, Hk, G, d, 16, [(i * 29) % 150 for i in range(R)], prefix), prefix, causal)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("R,B,Hk,G,d,prefix", [(210, 2, 2, 4, 64, 4500), (70, 4, 2, 5, 64, 4500), (260, 4, 2, 2, 128, 4300),
                                               (140, 4, 2, 5, 128, 4300), (50, 2, 1, 8, 256, 4200)])
def test_prefix_of_many_requests_with_few_rows(g, R, B, Hk, G, d, prefix, causal):
    """Tiles of the prefix shared by the rows of many requests, their own keys' by none."""
    check(g, make(12, R, B, Hk, G, d, 16, [(i * 29) % 70 for i in range(R)], prefix), prefix, causal)


def test_sharp_scores_and_scale(g):
    """Scores far apart (the running maximum moves, weights vanish) and a scale of the
    caller's own."""
    args = make(3, 2, 2, 1, 2, 64, 16, [100, 333], 70, kscale=6.0)
    check(g, args, 70, False)
    check(g, args, 70, True, scale=0.03125)


def test_extreme_scales(g):
    import torch
    q, kc, vc, bt, lens, pt = args = make(8, 2, 2, 1, 2, 64, 16, [50, 33], 20)
    for scale in (1e-36, 1e4):
        o = g.block_attention_fp4(q, kc, vc, bt, lens, prefix_table=pt, prefix_len=20, scale=scale)
        ro, _, size = attention64(q, cache_values(*kc), cache_values(*vc), bt, lens, pt, 20, False, scale)
        close(o, ro, torch.bfloat16, (2.0 ** -8 + 4e-4) * size, "o")


def test_rows_beyond_the_bound_are_cut(g):
    import torch
    args = make(4, 3, 2, 1, 2, 64, 16, [40, 20, 64], 0)
    o = g.block_attention_fp4(*args[:5], max_seq_len=32)
    want = g.block_attention_fp4(*args[:4], args[4].clamp(max=32), max_seq_len=32)
    assert torch.equal(o, want)
    assert (g.block_attention_fp4(*args[:5], max_seq_len=0) == 0).all()


def test_result_does_not_depend_on_the_batch(g):
    import torch
    q, kc, vc, bt, lens, pt = make(5, 3, 4, 2, 4, 128, 32, [500, 61, 7], 90)
    whole = g.block_attention_fp4(q, kc, vc, bt, lens, prefix_table=pt, prefix_len=90)
    for r in range(3):
        one = g.block_attention_fp4(q[r:r + 1], kc, vc, bt[r:r + 1].contiguous(), lens[r:r + 1], prefix_table=pt, prefix_len=90)
        assert torch.allclose(one.float(), whole[r:r + 1].float(), rtol=2.0 ** -6, atol=2.0 ** -7)
    assert torch.equal(whole, g.block_attention_fp4(q, kc, vc, bt, lens, prefix_table=pt, prefix_len=90))


@pytest.mark.parametrize("d,B,G", [(64, 5, 2), (128, 5, 4), (128, 20, 8), (128, 9, 2), (256, 4, 1), (256, 9, 2)])
def test_values_that_are_not_finite(g, d, B, G):
    """Groups of NaN, and of values that no float holds, reach exactly the queries that see
    their key: a later token of the block does not reach the earlier ones."""
    import torch
    q, kc, vc, bt, lens, pt = make(7, 2, B, 1, G, d, 16, [40 + B, B], 70, kscale=0.5)
    call = lambda v: g.block_attention_fp4(q, kc, v, bt, lens, prefix_table=pt, prefix_len=70, causal=True)  # noqa: E731
    clean = call(vc)
    codes, scales = (t.clone() for t in vc)
    for r, n in enumerate([40 + B, B]):
        j = n - 1  # seen by the last token of the block: NaN in its first group
        scales[int(bt[r, j // 16]), 0, 0, j % 16] = 255
        j = n - 2  # by the last two: infinities of both signs in the second
        scales[int(bt[r, j // 16]), 0, 1, j % 16] = 254
        codes[int(bt[r, j // 16]), 0, j % 16, 16:32] = 0xF7
    o = call((codes, scales))
    for b in range(B):
        first, second = o[:, b, :, :32], o[:, b, :, 32:64]
        assert torch.isnan(first).all() if b == B - 1 else torch.equal(first, clean[:, b, :, :32]), b
        if b >= B - 2:
            assert (second[..., 0::2] == math.inf).all() and (second[..., 1::2] == -math.inf).all(), b
        else:
            assert torch.equal(second, clean[:, b, :, 32:64]), b
    assert torch.equal(o[..., 64:], clean[..., 64:])
    # scales of 253 whose codes are small enough to be finite: their weight's share, in every row that sees them
    j = 39 + B
    codes.copy_(vc[0]), scales.copy_(vc[1])
    scales[int(bt[0, j // 16]), 0, 0, j % 16] = 253
    codes[int(bt[0, j // 16]), 0, j % 16, :16] = 0x22
    o, lse = g.block_attention_fp4(q, kc, (codes, scales), bt, lens, prefix_table=pt, prefix_len=70, causal=True, want_lse=True)
    ro, _, size = attention64(q, cache_values(*kc), cache_values(codes, scales), bt, lens, pt, 70, True)
    close(o, ro, torch.bfloat16, (2.0 ** -8 + 4e-4) * size, "o")


def test_scores_that_are_not_finite(g):
    """A key of NaN makes the rows that see it NaN and no others."""
    import torch
    q, kc, vc, bt, lens, pt = make(9, 2, 4, 1, 2, 128, 16, [44, 20], 0)
    clean = g.block_attention_fp4(q, kc, vc, bt, lens, causal=True)
    scales = kc[1].clone()
    j = 43 - 1  # seen by the last two tokens of the first request
    scales[int(bt[0, j // 16]), 0, 2, j % 16] = 255
    o = g.block_attention_fp4(q, (kc[0], scales), vc, bt, lens, causal=True)
    assert torch.isnan(o[0, 2:]).all() and torch.equal(o[0, :2], clean[0, :2]) and torch.equal(o[1], clean[1])
    # a query of NaN or infinity: its own rows
    q2 = q.clone()
    q2[1, 3, 0, 5], q2[1, 1, 1, 100] = math.nan, math.inf
    o = g.block_attention_fp4(q2, kc, vc, bt, lens, causal=True)
    hit = torch.zeros(2, 4, 2, dtype=torch.bool, device="cuda")
    hit[1, 3, 0] = hit[1, 1, 1] = True
    assert torch.isnan(o[hit]).all() and torch.equal(o[~hit], clean[~hit])


def test_table_entries_that_name_no_page_stay_inside(g):
    import torch
    q, kc, vc, bt, lens, pt = make(9, 3, 1, 2, 2, 128, 16, [40, 40, 40], 0, dead=False)
    want = g.block_attention_fp4(q, kc, vc, bt, lens)
    bt[1, 1], bt[1, 2] = -5, 2 ** 31 - 1
    o = g.block_attention_fp4(q, kc, vc, bt, lens)
    assert torch.isfinite(o.float()).all() and torch.equal(o[0], want[0]) and torch.equal(o[2], want[2])


SHAPES = [(6, 4, 2, 4, 128, 16, [40, 0, 300, 4, 1000, 77], 4500), (3, 7, 1, 8, 256, 32, [700, 7, 60], 5000),
          (2, 1, 4, 4, 64, 64, [5000, 1], 0)]


def random_set(g, seed, R, B, Hk, G, d, page, lens, prefix, pages=None):
    """Random codes under scales that make normal-sized values, tables round and round the
    pages."""
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    wide, shared = max(-(-n // page) for n in lens) + 1, -(-prefix // page)
    pages = pages or R * wide + shared
    ids = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    ids = ids.repeat(-(-(R * wide + shared) // pages))

    def cache():
        codes, scales = g.cache_fp4(pages, Hk, page, d)
        codes.random_(0, 256, generator=gen)
        scales.random_(122, 127, generator=gen)
        return codes, scales
    q = torch.randn(R, B, Hk * G, d, generator=gen, device="cuda").to(torch.bfloat16)
    return [q, cache(), cache(), ids[shared:shared + R * wide].reshape(R, wide).contiguous(),
            torch.tensor(lens, dtype=torch.int32).cuda(), ids[:shared].contiguous()]


def flat(args):
    return [t for a in args for t in (a if isinstance(a, tuple) else (a,))]


@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_captured_and_replayed(g, i):
    """Every replay, on new inputs and lengths and with eager work between, gives the eager
    call's bits; so do two graphs that share a memory pool, one after the other."""
    import torch
    R, B, Hk, G, d, page, lens, prefix = SHAPES[i]
    assert g.block_attention_fp4_workspace_bytes(R, B, Hk * G, Hk, d, page, (max(-(-n // page) for n in lens) + 1) * page, prefix) > 0
    static = random_set(g, 1, *SHAPES[i])
    call = lambda a, causal: g.block_attention_fp4(*a[:5], prefix_table=a[5], prefix_len=prefix, causal=causal, want_lse=True)  # noqa: E731
    call(static, False)
    torch.cuda.synchronize()
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        got1 = call(static, False)
    with torch.cuda.graph(second, pool=first.pool()):
        got2 = call(static, True)
    for rep in range(4):
        new = random_set(g, 10 + rep, *SHAPES[i])
        new[4] = new[4].roll(rep)
        for a, b in zip(flat(static), flat(new)):
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
    import torch
    sets = [random_set(g, 20 + i, *s) for i, s in enumerate(SHAPES[:2])]
    pre = [s[-1] for s in SHAPES[:2]]
    call = lambda k: g.block_attention_fp4(*sets[k][:5], prefix_table=sets[k][5], prefix_len=pre[k], causal=True)  # noqa: E731
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
    check(g, random_set(g, 30, 5, 3, 2, 2, 128, 16, [200, 90, 0, 333, 33], 1000, pages=40), 1000, causal)


def key_rows(cache, table, n, d):
    """The first n keys of a table's pages in 64 bits, on the GPU (one kv head)."""
    import torch
    codes, scales = (t[table.long()] for t in cache)
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    value = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    v = torch.where(c >= 8, -1.0, 1.0) * value[(c & 7).long()]
    unit = torch.exp2(scales.double() - 127).transpose(2, 3).repeat_interleave(32, -1)
    return (v * unit).transpose(1, 2).reshape(-1, d)[:n]


@pytest.mark.parametrize("d,prefix,lens", [(64, 131072, [3, 700]), (128, 40001, [70000]), (256, 0, [33333, 5])])
def test_many_keys(g, d, prefix, lens):
    """Against sums in 64 bits on the GPU."""
    import torch
    R, B, Hk, G, page = len(lens), 2, 1, 2, 64
    q, kc, vc, bt, sl, pt = random_set(g, 40, R, B, Hk, G, d, page, lens, prefix)
    o, lse = g.block_attention_fp4(q, kc, vc, bt, sl, prefix_table=pt, prefix_len=prefix, causal=True, want_lse=True)
    for r, n in enumerate(lens):
        k, v = (torch.cat([key_rows(c, pt, prefix, d), key_rows(c, bt[r], n, d)]) for c in (kc, vc))
        for b in range(B):
            m = prefix + max(0, n - (B - 1 - b))
            for h in range(G):
                s = (k[:m] * q[r, b, h].double()).sum(1) / math.sqrt(d)
                p = torch.softmax(s, 0)[:, None]
                close(o[r, b, h], (p * v[:m]).sum(0).cpu(), torch.bfloat16, (2.0 ** -8 + 4e-4) * (p * v[:m].abs()).sum(0).cpu(),
                      "request %d query %d head %d" % (r, b, h))
                assert abs(float(lse[r, b, h]) - float(torch.logsumexp(s, 0))) <= 5e-4


def test_offsets_beyond_32_bits(g):
    """A cache of 4.6 GB of codes whose last pages are read."""
    import torch
    pages, Hk, page, d = 70000, 8, 64, 256
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    ids = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32, device="cuda")

    def cache():
        codes = torch.empty((pages, Hk, page, d // 2), dtype=torch.uint8, device="cuda")
        scales = torch.empty((pages, Hk, d // 32, page), dtype=torch.uint8, device="cuda")
        for p in ids[0].tolist():
            codes[p].random_(0, 256, generator=gen)
            scales[p].random_(122, 127, generator=gen)
        return codes, scales
    kc, vc = cache(), cache()
    assert kc[0].numel() > 2 ** 32
    q = torch.randn(1, 2, Hk * 2, d, generator=gen, device="cuda").to(torch.bfloat16)
    lens = torch.tensor([170], dtype=torch.int32, device="cuda")
    o = g.block_attention_fp4(q, kc, vc, ids, lens, causal=True)
    at = ids[0].long()
    small = [tuple(t[at] for t in c) for c in (kc, vc)]
    bt = torch.arange(3, dtype=torch.int32, device="cuda")[None]
    ro, _, size = attention64(q, cache_values(*small[0]), cache_values(*small[1]), bt, lens, None, 0, True)
    close(o, ro, torch.bfloat16, (2.0 ** -8 + 4e-4) * size, "o")


def test_a_layer_served_from_4_bits(g):
    """Step tables, q/k norms and rotary positions into the cache, and the attention over a
    shared prefix, for a prompt and three blocks: keys and values as 64 bits round them from
    the same inputs, the outputs those of a softmax over them."""
    import torch
    R, B, Hq, Hk, d, page, prefix = 5, 4, 8, 2, 128, 16, 50
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    freqs, m = g.rotary_frequencies(d, scaling="yarn", factor=4.0, original_length=64)
    qw, kw = 1 + 0.2 * rnd(d), 1 + 0.2 * rnd(d)
    pages, width = 64, 6
    kc, vc = g.cache_fp4(pages, Hk, page, d), g.cache_fp4(pages, Hk, page, d)
    free = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    shared = -(-prefix // page)
    pt = free[:shared].contiguous()
    rows64 = [torch.zeros(pages * page, Hk, d, dtype=torch.float64) for _ in range(2)]

    def put(x, pos, slots):
        q, k, v = x.split([Hq, Hk, Hk], 1)
        y = g.qk_norm_rotary_cache_fp4(pos, freqs, q, k, v, slots, kc, vc, qw, kw, mscale=m)
        live = slots.cpu() >= 0
        k64 = norm_rotary64(leaf(k).detach(), leaf(kw).detach(), pos, freqs, False, m, 1e-6)
        rows64[0][slots.cpu()[live]] = fp4_nearest(k64)[live]
        rows64[1][slots.cpu()[live]] = fp4_nearest(v)[live]
        return y

    at = torch.arange(prefix, device="cuda")
    put(rnd(prefix, Hq + 2 * Hk, d).bfloat16(), at.int(), pt[at // page].long() * page + at % page)
    lens, table = torch.zeros(R, dtype=torch.int32, device="cuda"), torch.zeros(R, width, dtype=torch.int32, device="cuda")
    used = torch.full((1,), shared, dtype=torch.int32, device="cuda")
    for step, new in enumerate([[7, 0, 20, 16, 33], [B] * R, [B] * R, [B] * R]):
        new = torch.tensor(new, dtype=torch.int32, device="cuda")
        total = int(new.sum())
        t = g.step_tables(lens, new, table, free, used, page, total + 3, position_offset=prefix)
        assert int(t["status"]) == 0
        y = put(rnd(total + 3, Hq + 2 * Hk, d).bfloat16(), t["positions"], t["slots"])
        lens, used = t["seq_lens"], t["pages_used"]
        if step == 0:
            continue
        q = y[:total].reshape(R, B, Hq, d)
        for causal in (False, True):
            o = g.block_attention_fp4(q, kc, vc, table, lens, prefix_table=pt, prefix_len=prefix, causal=causal)
            pages64 = [r.reshape(pages, page, Hk, d).transpose(1, 2) for r in rows64]
            ro, _, size = attention64(q, *pages64, table, lens, pt, prefix, causal)
            close(o, ro, torch.bfloat16, (2.0 ** -8 + 4e-4) * size, "step %d" % step)
        # and a softmax over the same rows moved into a cache of bf16
        every = torch.arange(pages * page, device="cuda")
        rk, rv = g.cache_fp4_rows(every, kc, vc)
        as16 = [r.reshape(pages, page, Hk, d).transpose(1, 2).contiguous() for r in (rk, rv)]
        b16 = g.block_attention(q, *as16, table, lens, prefix_table=pt, prefix_len=prefix, causal=True)
        assert torch.allclose(o.float(), b16.float(), rtol=2.0 ** -6, atol=2.0 ** -7)


def test_calls_allocate_only_what_they_return(g):
    import torch
    q, kc, vc, bt, lens, pt = random_set(g, 3, *SHAPES[0])
    o, lse = g.block_attention_fp4(q, kc, vc, bt, lens, prefix_table=pt, prefix_len=4500, want_lse=True)
    n = g.block_attention_fp4_workspace_bytes(6, 4, 8, 2, 128, 16, bt.shape[1] * 16, 4500)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    g.block_attention_fp4(q, kc, vc, bt, lens, prefix_table=pt, prefix_len=4500, out=o, lse=lse, workspace=ws)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before


def test_refusals(g):
    import torch
    q, kc, vc, bt, lens, pt = make(1, 2, 2, 1, 2, 64, 16, [40, 20], 30)
    ok = lambda **m: g.block_attention_fp4(**{**dict(q=q, k_cache=kc, v_cache=vc, block_table=bt, seq_lens=lens), **m})  # noqa: E731
    ok()
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(q=q[..., :32].contiguous()), dict(k_cache=kc[0]), dict(k_cache=vc[0], v_cache=vc[0]),
                dict(v_cache=(vc[0][:1], vc[1][:1])), dict(v_cache=(vc[0], vc[1][:, :, :1])), dict(block_table=bt.long()),
                dict(block_table=bt[0]), dict(seq_lens=lens[:1]), dict(prefix_len=17, prefix_table=pt[:1]), dict(prefix_len=-1),
                dict(max_seq_len=10 ** 6), dict(scale=math.inf), dict(out=q[:1].clone()), dict(workspace=torch.empty(1, device="cuda"), prefix_len=30, prefix_table=pt.cpu())):
        with pytest.raises(g.FlareError):
            ok(**bad)
    odd = torch.empty(vc[0].numel() + 8, dtype=torch.uint8, device="cuda")[8:].reshape(vc[0].shape)
    with pytest.raises(g.FlareError):
        ok(v_cache=(odd, vc[1]))


FEW_AND_MANY_ROWS = [
    (1, 1, 4, 4, 128, 64, [700], 0), (3, 4, 2, 4, 128, 16, [1, 33, 130], 77), (4, 1, 1, 8, 256, 32, [15, 16, 31, 32], 1),
    (2, 16, 1, 2, 64, 32, [16, 47], 40), (5, 3, 1, 5, 64, 128, [3, 64, 127, 128, 129], 129), (1, 1, 1, 2, 64, 16, [4500], 0),
    (1, 1, 1, 4, 128, 16, [70], 4200), (3, 2, 2, 2, 128, 16, [0, 33, 70], 4100), (2, 8, 1, 4, 128, 16, [8, 90], 20),
    # tiles that four waves share: of own keys, with a prefix before them, of a prefix alone
    (2, 16, 1, 8, 64, 32, [16, 47], 40), (2, 20, 1, 8, 128, 32, [20, 131], 70), (2, 9, 1, 8, 256, 16, [9, 90], 31),
    (2, 32, 2, 2, 128, 32, [32, 190], 0), (3, 9, 1, 5, 64, 32, [20, 0, 131], 4500), (140, 4, 2, 2, 128, 16, [(i * 29) % 70 for i in range(140)], 4300),
    (50, 2, 1, 8, 256, 16, [(i * 29) % 70 for i in range(50)], 4200), (130, 20, 1, 4, 128, 16, [(i * 29) % 90 for i in range(130)], 77)]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("i", range(len(FEW_AND_MANY_ROWS)))
def test_weights_keep_16_bits(g, i, causal):
    """The weights go into the second product in two bf16 halves.  The first is cut, so that up to
    2^-7 of a weight is left, the second rounds that by 2^-8 of itself, and 2^-20 are added: 2^-15 +
    2^-20 of sum p |v| / sum p in place of 2^-8.  Scores, exponentials and sums as above."""
    import torch
    R, B, Hk, G, d, page, lens, prefix = FEW_AND_MANY_ROWS[i]
    q, kc, vc, bt, sl, pt = make(50 + i, R, B, Hk, G, d, page, lens, prefix)
    o = g.block_attention_fp4(q, kc, vc, bt, sl, prefix_table=pt, prefix_len=prefix, causal=causal)
    ro, _, size = attention64(q, cache_values(*kc), cache_values(*vc), bt, sl, pt, prefix, causal)
    close(o, ro, torch.bfloat16, (2.0 ** -15 + 2.0 ** -20 + 4e-4) * size, "o")


@pytest.mark.parametrize("d,B,G,R", [(64, 5, 2, 2), (128, 1, 4, 2), (128, 8, 4, 2), (256, 4, 1, 2), (128, 20, 8, 2), (256, 9, 2, 2)])
def test_infinite_values_that_every_row_sees(g, d, B, G, R):
    """A value that no float holds times a weight above 0 is infinite, of the value's sign,
    whatever the weight's bits: also where one key has all the weight, which is then 1 exactly."""
    import torch
    for own, prefix in ((1, 0), (40, 0), (90, 70)):
        q, kc, vc, bt, lens, pt = make(60, R, B, 1, G, d, 16, [own] * R, prefix, kscale=0.5)
        clean = g.block_attention_fp4(q, kc, vc, bt, lens, prefix_table=pt, prefix_len=prefix)
        codes, scales = (t.clone() for t in vc)
        for r in range(R):
            page = int(bt[r, 0])
            scales[page, 0, 1, 0] = 254
            codes[page, 0, 0, 16:32] = 0xF7
        o = g.block_attention_fp4(q, kc, (codes, scales), bt, lens, prefix_table=pt, prefix_len=prefix)
        assert (o[..., 32:64:2] == math.inf).all() and (o[..., 33:64:2] == -math.inf).all()
        assert torch.equal(o[..., :32], clean[..., :32]) and torch.equal(o[..., 64:], clean[..., 64:])
