"""The norms of queries and keys with rotary positions, their reverse mode, the forms into
a paged cache of the inputs' type and in 4 bits, and rows read back from one, against
64-bit definitions.

Tolerances, relative to the size of the terms a value is formed of (|a| + |b| of a turned
pair, scaled): the sum of squares is off by at most as many half steps of fp32 as its
chain is long (48 products of a lane and 6 joins at most, half of it in the root), root,
quotient and the two products by 4, the coefficients by 4 each (the angle's rest in turns
is rounded once, pi half steps, the sine by 2) and the rotation's products and sum by 3:
48 half steps in all.  Then the output's own rounding.  The reverse mode forms two such
sums and two more products: 96."""
import math

import pytest

from layer_oracle import HALF_STEP, close
from softmax_oracle import (STEP, cache_values, fp4_nearest, leaf, norm_rotary64, norm_rotary_size, rotary_leaf, same)

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def g():
    import gated_deltanet_dual_amd as g
    g.lib()
    return g


def make(seed, T, Hq, Hk, d, rot, io, norm="qk", far=4096, wide=True):
    """q, k, v as slices of one projection's rows (wide), positions, frequencies, weights."""
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    rows = rnd(T, (Hq + 2 * Hk) * d + 3).to(io)
    cut = lambda a, n: rows[:, a * d + 3:(a + n) * d + 3].unflatten(1, (n, d))  # noqa: E731
    q, k, v = cut(0, Hq), cut(Hq, Hk), cut(Hq + Hk, Hk)
    if not wide:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pos = torch.randint(0, far, (T,), generator=gen, device="cuda", dtype=torch.int32)
    freqs = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64, device="cuda") / max(rot // 2, 1))
    w = {n: 1 + 0.2 * rnd(d) if n in norm else None for n in "qk"}
    return q, k, v, pos, freqs, w["q"], w["k"], rnd


def check_forward(y, x, w, pos, freqs, inter, mscale, io, where):
    x64, w64 = leaf(x).detach(), None if w is None else leaf(w).detach()
    size = norm_rotary_size(x64, w64, freqs, inter, mscale, EPS)
    close(y, norm_rotary64(x64, w64, pos, freqs, inter, mscale, EPS), io, 48 * STEP * size, where)


# T, q heads, k heads, d, turned, interleaved, io, normed: one token to many, heads of every width class, odd ones,
# nothing and everything turned, vectors that end inside a row
SIZES = [(1, 16, 4, 128, 128, False, "bf16", "qk"), (5, 3, 1, 64, 64, True, "bf16", "qk"), (33, 6, 3, 80, 50, True, "f32", "qk"),
         (7, 1, 1, 2, 2, False, "f32", "qk"), (70, 2, 2, 100, 34, False, "bf16", "q"), (70, 2, 5, 100, 34, True, "f32", "k"),
         (300, 5, 2, 96, 0, False, "bf16", "qk"), (65, 4, 2, 256, 128, False, "f32", "qk"), (9, 2, 1, 1024, 514, False, "f32", "qk"),
         (9, 2, 1, 1023, 77, True, "bf16", "qk"), (2500, 16, 4, 128, 32, False, "bf16", "qk"), (40, 2, 1, 1, 0, False, "f32", "qk"),
         (3000, 1, 1, 64, 64, False, "bf16", "")]


def types(io):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[io]


@pytest.mark.parametrize("T,Hq,Hk,d,rot,inter,io,norm", SIZES)
def test_forward(g, T, Hq, Hk, d, rot, inter, io, norm):
    io = types(io)
    for wide in (False, True):
        q, k, _, pos, freqs, qw, kw, _ = make(T + d, T, Hq, Hk, d, rot, io, norm, wide=wide)
        y, z = g.qk_norm_rotary(pos, freqs, q, k, qw, kw, eps=EPS, interleaved=inter, mscale=1.25)
        check_forward(y, q, qw, pos, freqs, inter, 1.25, io, "q")
        check_forward(z, k, kw, pos, freqs, inter, 1.25, io, "k")
    alone, none = g.qk_norm_rotary(pos, freqs, q, None, qw, interleaved=inter, mscale=1.25, eps=EPS)
    assert none is None
    same(alone, y.cpu().double())


# heads that 64 lanes do not hold at a time, in whole vectors and short ones; vectors of 4 and of 8; heads narrower than a
# vector; workgroups of many tokens, the last one's fewer
FORMS = [(6, 2, 1, 1020, 600, False, "bf16", "qk"), (6, 2, 1, 1021, 14, False, "bf16", "qk"), (6, 1, 2, 1024, 1024, True, "bf16", "qk"),
         (6, 1, 2, 1020, 600, True, "f32", "qk"), (11, 3, 2, 132, 64, True, "bf16", "qk"), (11, 3, 2, 132, 132, False, "bf16", "k"),
         (9, 5, 3, 3, 2, True, "bf16", "qk"), (9, 5, 3, 3, 2, False, "f32", "qk"), (9, 2, 2, 2, 2, True, "bf16", "qk"),
         (70001, 1, 1, 16, 16, False, "bf16", "qk"), (3083, 2, 3, 20, 10, True, "bf16", "qk")]


@pytest.mark.parametrize("T,Hq,Hk,d,rot,inter,io,norm", FORMS)
def test_forms(g, T, Hq, Hk, d, rot, inter, io, norm):
    import torch
    io = types(io)
    q, k, v, pos, freqs, qw, kw, rnd = make(T + d, T, Hq, Hk, d, rot, io, norm)
    y, z = g.qk_norm_rotary(pos, freqs, q, k, qw, kw, eps=EPS, interleaved=inter)
    check_forward(y, q, qw, pos, freqs, inter, 1.0, io, "q")
    check_forward(z, k, kw, pos, freqs, inter, 1.0, io, "k")
    dq, dk = rnd(T, Hq, d).to(io), rnd(T, Hk, d).to(io)
    out = g.qk_norm_rotary_bwd(pos, freqs, q, k, dq, dk, qw, kw, eps=EPS, interleaved=inter)
    chain = 256 + 64 + max(Hq, Hk) * (1 + T // 256)
    check_reverse(out, "q", q, qw, dq, pos, freqs, inter, 1.0, io, chain)
    check_reverse(out, "k", k, kw, dk, pos, freqs, inter, 1.0, io, chain)
    pages = -(-T // 16) + 1
    kc, vc = rnd(pages, Hk, 16, d).to(io), rnd(pages, Hk, 16, d).to(io)
    slots = torch.randperm(pages * 16, device="cuda")[:T]
    y2 = g.qk_norm_rotary_cache(pos, freqs, q, k, v, slots, kc, vc, qw, kw, eps=EPS, interleaved=inter)
    flat = lambda c: c.transpose(1, 2).flatten(0, 1)[slots]  # noqa: E731
    assert y2.equal(y) and flat(kc).equal(z) and flat(vc).equal(v)


def gradients64(x, w, dy, pos, freqs, inter, mscale):
    """(dx, dw) and the size of the terms that each is formed of."""
    import torch
    x, w, dy = leaf(x), leaf(w), dy.detach().cpu().double()
    norm_rotary64(x, w, pos, freqs, inter, mscale, EPS).backward(dy)
    with torch.no_grad():
        du = norm_rotary_size(dy, None, freqs, inter, mscale, EPS)
        if w is None:
            return x.grad, None, du, None
        r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
        n = (x * r).abs()
        dn = du * w.abs()
        return x.grad, w.grad, r * (dn + n * (dn * n).mean(-1, keepdim=True)), (du * n).sum((0, 1))


def check_reverse(grads, side, x, w, dy, pos, freqs, inter, mscale, io, chain):
    dx, dw, dx_size, dw_size = gradients64(x, w, dy, pos, freqs, inter, mscale)
    close(grads["d" + side], dx, io, 96 * STEP * dx_size, "d" + side)
    if w is None:
        assert grads["d%s_weight" % side] is None
    else:
        # a thread's rows in turn, the teams of a workgroup, the workgroups: `chain` joins at most
        close(grads["d%s_weight" % side], dw, types("f32"), (96 + chain) * STEP * dw_size, "d%s_weight" % side)


@pytest.mark.parametrize("T,Hq,Hk,d,rot,inter,io,norm", SIZES)
def test_reverse(g, T, Hq, Hk, d, rot, inter, io, norm):
    io = types(io)
    q, k, _, pos, freqs, qw, kw, rnd = make(T + d + 1, T, Hq, Hk, d, rot, io, norm)
    dq, dk = rnd(T, Hq + Hk, d).to(io).split([Hq, Hk], 1)  # slices of wider rows
    out = g.qk_norm_rotary_bwd(pos, freqs, q, k, dq, dk, qw, kw, eps=EPS, interleaved=inter, mscale=0.75)
    # at most 1024 workgroups of up to 256 teams: no thread passes more than T * heads / teams + heads rows
    chain = 256 + 64 + max(Hq, Hk) * (1 + T // 256)
    check_reverse(out, "q", q, qw, dq, pos, freqs, inter, 0.75, io, chain)
    check_reverse(out, "k", k, kw, dk, pos, freqs, inter, 0.75, io, chain)
    again = g.qk_norm_rotary_bwd(pos, freqs, q, k, dq, dk, qw, kw, eps=EPS, interleaved=inter, mscale=0.75)
    for name, t in out.items():
        assert t is None or t.equal(again[name]), name
    # queries alone
    alone = g.qk_norm_rotary_bwd(pos, freqs, q, None, dq, None, qw, eps=EPS, interleaved=inter, mscale=0.75)
    assert alone["dk"] is None and alone["dk_weight"] is None and alone["dq"].equal(out["dq"])


def test_reverse_of_many_rows(g):
    """Workgroups that pass several tokens' rounds, and weights' sums over 10^5 rows."""
    import torch
    T, Hq, Hk, d = 20011, 8, 2, 64
    q, k, _, pos, freqs, qw, kw, rnd = make(3, T, Hq, Hk, d, 64, torch.bfloat16)
    dq, dk = rnd(T, Hq, d).bfloat16(), rnd(T, Hk, d).bfloat16()
    out = g.qk_norm_rotary_bwd(pos, freqs, q, k, dq, dk, qw, kw, eps=EPS)
    chain = 256 + 64 + Hq * (1 + T // 256)
    check_reverse(out, "q", q, qw, dq, pos, freqs, False, 1.0, torch.bfloat16, chain)
    check_reverse(out, "k", k, kw, dk, pos, freqs, False, 1.0, torch.bfloat16, chain)


@pytest.mark.parametrize("inter", [False, True])
def test_reverse_against_differences(g, inter):
    """(L(x + h v) - L(x - h v)) / 2 h of L = <dy, y> through the kernel, in fp32: what the
    same quotient is in 64 bits, off by the outputs' error over h; and that quotient nears
    <dx, v> as h^2."""
    import torch
    T, Hq, Hk, d, h = 6, 3, 2, 40, 2.0 ** -6
    q, k, _, pos, freqs, qw, kw, rnd = make(5, T, Hq, Hk, d, 24, torch.float32, wide=False)
    dq, dk = rnd(T, Hq, d), rnd(T, Hk, d)
    grads = g.qk_norm_rotary_bwd(pos, freqs, q, k, dq, dk, qw, kw, eps=EPS, interleaved=inter)
    for side, x, w, dy in (("q", q, qw, dq), ("k", k, kw, dk)):
        vx, vw = (rnd(*x.shape) * 8).round() / 8, (rnd(*w.shape) * 8).round() / 8
        at = lambda s: ((x.double() + s * vx.double()).float(), (w.double() + s * vw.double()).float())  # noqa: E731
        y = {s: g.qk_norm_rotary(pos, freqs, *((at(s)[0], None, at(s)[1]) if side == "q" else (x, at(s)[0], None, at(s)[1])),
                                 eps=EPS, interleaved=inter)[side == "k"] for s in (h, -h)}
        L = lambda t: float((t.cpu().double() * dy.cpu().double()).sum())  # noqa: E731
        y64 = lambda s: norm_rotary64(*(t.cpu().double() for t in at(s)), pos, freqs, inter, 1.0, EPS)  # noqa: E731
        got, want = (L(y[h]) - L(y[-h])) / (2 * h), (L(y64(h)) - L(y64(-h))) / (2 * h)
        size = norm_rotary_size(x.cpu().double(), w.cpu().double(), freqs, inter, 1.0, EPS)
        noise = 49 * STEP * float((1.5 * size * dy.cpu().double().abs()).sum()) / h
        assert abs(got - want) <= noise
        slope = float((grads["d" + side].double() * vx.double()).sum() + (grads["d%s_weight" % side].double() * vw.double()).sum())
        half = (L(y64(h / 2)) - L(y64(-h / 2))) / h
        assert abs(half - slope) <= 0.3 * abs(want - slope) + 1e-4 * float((size * dy.cpu().double().abs()).sum())


def page_slots(T, pages, page, seed):
    """Distinct slots of a cache, some rows padded."""
    import torch
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(seed))[:T]
    slots[3::11] = -1
    if T > 7:
        slots[7] = pages * page  # of no page either
    return slots.cuda()


@pytest.mark.parametrize("T,Hq,Hk,d,rot,inter,io,norm,page", [
    (1, 16, 4, 128, 128, False, "bf16", "qk", 64), (70, 3, 2, 100, 34, True, "f32", "qk", 1), (300, 4, 2, 64, 16, False, "bf16", "k", 16),
    (40, 2, 9, 72, 72, True, "bf16", "", 7), (2300, 2, 1, 64, 64, False, "bf16", "qk", 128)])
def test_cache(g, T, Hq, Hk, d, rot, inter, io, norm, page):
    import torch
    io = types(io)
    q, k, v, pos, freqs, qw, kw, rnd = make(T, T, Hq, Hk, d, rot, io, norm)
    pages = -(-T // page) + 3
    kc, vc = rnd(pages, Hk, page, d).to(io), rnd(pages, Hk, page, d).to(io)
    k0, v0, slots = kc.clone(), vc.clone(), page_slots(T, pages, page, 1)
    y = g.qk_norm_rotary_cache(pos, freqs, q, k, v, slots, kc, vc, qw, kw, eps=EPS, interleaved=inter, mscale=1.5)
    packed = g.qk_norm_rotary(pos, freqs, q, k, qw, kw, eps=EPS, interleaved=inter, mscale=1.5)
    assert y.equal(packed[0])  # tested above
    live = torch.nonzero((slots >= 0) & (slots < pages * page))[:, 0]
    at, off = slots[live] // page, slots[live] % page
    k0[at, :, off], v0[at, :, off] = packed[1][live], v[live]
    assert kc.equal(k0) and vc.equal(v0)


# d and Hk of one round of keys through the workgroup's buffer and of several
FP4_SIZES = [(1, 16, 4, 128, 128, False, "bf16", "qk", 64), (70, 3, 2, 96, 34, True, "f32", "qk", 1), (300, 4, 2, 64, 16, False, "bf16", "k", 16),
             (40, 1, 9, 256, 256, True, "bf16", "qk", 32), (33, 2, 3, 1024, 100, False, "f32", "qk", 16), (9, 2, 40, 32, 0, False, "bf16", "", 7),
             (2300, 2, 1, 64, 64, False, "bf16", "q", 128), (2100, 1, 8, 160, 160, False, "f32", "qk", 64),
             # heads that 64 lanes do not hold at a time; workgroups of many tokens of one key head
             (5, 1, 2, 1024, 1024, False, "bf16", "qk", 16), (5, 1, 2, 992, 50, True, "f32", "qk", 16),
             (66000, 1, 1, 32, 32, True, "bf16", "qk", 64), (50, 3, 2, 128, 120, False, "bf16", "qk", 16)]


def fill(g, pages, heads, page, d, seed):
    """A cache in 4 bits of random codes and scales."""
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    codes, scales = g.cache_fp4(pages, heads, page, d)
    codes.random_(0, 256, generator=gen)
    scales.random_(100, 140, generator=gen)
    return codes, scales


@pytest.mark.parametrize("T,Hq,Hk,d,rot,inter,io,norm,page", FP4_SIZES)
def test_cache_fp4(g, T, Hq, Hk, d, rot, inter, io, norm, page):
    import torch
    io = types(io)
    q, k, v, pos, freqs, qw, kw, _ = make(T, T, Hq, Hk, d, rot, io, norm, far=1000000)
    pages = -(-T // page) + 3
    kc, vc = fill(g, pages, Hk, page, d, 1), fill(g, pages, Hk, page, d, 2)
    want = [cache_values(*c).transpose(1, 2).flatten(0, 1) for c in (kc, vc)]  # by slot
    slots = page_slots(T, pages, page, 2)
    y = g.qk_norm_rotary_cache_fp4(pos, freqs, q, k, v, slots, kc, vc, qw, kw, eps=EPS, interleaved=inter, mscale=1.5)
    check_forward(y, q, qw, pos, freqs, inter, 1.5, io, "q")
    live = torch.nonzero((slots.cpu() >= 0) & (slots.cpu() < pages * page))[:, 0]
    k64 = norm_rotary64(leaf(k).detach(), None if kw is None else leaf(kw).detach(), pos, freqs, inter, 1.5, EPS)
    want[0][slots.cpu()[live]] = fp4_nearest(k64)[live]
    want[1][slots.cpu()[live]] = fp4_nearest(v)[live]
    for got, w in zip((kc, vc), want):
        same(cache_values(*got).transpose(1, 2).flatten(0, 1), w)
    # and all rows read back, by their slots
    every = torch.arange(pages * page, device="cuda")
    for t in (torch.bfloat16, torch.float32):
        rk, rv = g.cache_fp4_rows(every, kc, vc, dtype=t)
        same(rk, want[0])
        same(rv, want[1])


def exact_rows():
    """Rows of 64 channels, each value of two groups: halfway between codes, next to it by
    a step of bf16 or fp32, the scales' borders, extremes, infinities and NaN."""
    import torch
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]
    rows = []
    for top in (6.0, 7.0, 7.03125, 4.0, 7.96875, 5.0):
        for e in (-20, 0, 3, 100):
            rows.append([s * m * 2.0 ** e for s in (1, -1) for m in mids] + [top * 2.0 ** e] + [0.0] * 15)
            rows.append([s * m * (1 + b * 2.0 ** -7) * 2.0 ** e for s in (1, -1) for m in mids for b in (1, -0.5)][:31] + [top * 2.0 ** e])
    rows += [[0.0] * 32, [-0.0] * 32, [2.0 ** -133] * 32, [2.0 ** -126, -2.0 ** -127] * 16, [2.0 ** -130] + [0.0] * 31,
             [3.3895e38] + [1e38] * 31, [2.9e38, 2.97e38, 3.0e38] + [2.5e38] * 29, [math.inf] + [1.0] * 31, [1.0] * 31 + [-math.inf],
             [math.nan] + [2.0] * 31, [math.inf, math.nan] + [0.0] * 30]
    x = torch.tensor(rows, dtype=torch.float64)
    return torch.cat([x, x.roll(5, 0)], -1)  # each group beside another


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_rounding_of_4_bits(g, io):
    """Keys that are neither normed nor turned go by the 64-bit path, values by the other:
    both to the value that the search finds."""
    import torch
    from softmax_oracle import fp4_values
    io = types(io)
    x = exact_rows().to(io)[:, None].cuda()
    T = x.shape[0]
    kc, vc = fill(g, 4, 1, 32, 64, 1), fill(g, 4, 1, 32, 64, 2)
    pos, freqs = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.float64, device="cuda")
    slots = torch.arange(T, device="cuda")
    g.qk_norm_rotary_cache_fp4(pos, freqs, x, x, x, slots, kc, vc)
    want = fp4_values(x)
    for t in (torch.float32, torch.bfloat16):
        k, v = g.cache_fp4_rows(slots, kc, vc, dtype=t)
        same(k, want)
        same(v, want)
    bytes_ = kc[1].transpose(2, 3).reshape(-1, 2)[:T].cpu()
    assert bytes_.equal(vc[1].transpose(2, 3).reshape(-1, 2)[:T].cpu())
    assert ((bytes_ >= 1) & (bytes_ <= 252) | (bytes_ == 255)).all()


def test_every_code_and_scale_reads_back(g):
    """All 256 bytes of codes under all 256 scales, as both types."""
    import torch
    codes, scales = g.cache_fp4(16, 1, 16, 512)
    codes.copy_(torch.arange(256, dtype=torch.uint8, device="cuda").expand(16, 1, 16, 256))
    scales.copy_(torch.arange(256, dtype=torch.uint8, device="cuda").reshape(16, 1, 1, 16).expand(16, 1, 16, 16))
    slots = torch.arange(256, device="cuda")
    want = cache_values(codes, scales).transpose(1, 2).flatten(0, 1)
    big = want.abs() >= 2.0 ** 128  # what neither type holds: infinities
    want = torch.where(big, torch.sign(want) * math.inf, want)
    for t in (torch.float32, torch.bfloat16):
        same(g.cache_fp4_rows(slots, (codes, scales), dtype=t), want, str(t))


def test_rows_of_no_slot_and_twice(g):
    import torch
    c = fill(g, 3, 2, 16, 96, 1)
    slots = torch.tensor([5, -1, 47, 48, 5, 2 ** 40, -(2 ** 62), 0], device="cuda")
    out = torch.full((8, 2, 96), 7.0, dtype=torch.bfloat16, device="cuda")
    got = g.cache_fp4_rows(slots, c, out=out)
    assert got is out
    want = cache_values(*c).transpose(1, 2).flatten(0, 1)
    for i, s in enumerate(slots.tolist()):
        same(got[i], want[s] if 0 <= s < 48 else torch.zeros(2, 96))
    assert g.cache_fp4_rows(slots[:0], c).shape == (0, 2, 96)


def test_infinities_and_nan_stay_in_their_rows(g):
    import torch
    q, k, v, pos, freqs, qw, kw, rnd = make(1, 12, 2, 2, 64, 32, torch.bfloat16, wide=False)
    clean = g.qk_norm_rotary(pos, freqs, q, k, qw, kw)
    q[3, 1, 7], k[5, 0, 40], v[6, 1, 33] = math.nan, math.inf, math.nan
    y, z = g.qk_norm_rotary(pos, freqs, q, k, qw, kw)
    for got, ref, (t, h) in ((y, clean[0], (3, 1)), (z, clean[1], (5, 0))):
        hit = torch.zeros(12, 2, dtype=torch.bool, device="cuda")
        hit[t, h] = True
        assert got[~hit].equal(ref[~hit]) and torch.isnan(got[hit]).any() and not torch.isfinite(got[hit]).all()
    kc, vc = g.cache_fp4(1, 2, 16, 64), g.cache_fp4(1, 2, 16, 64)
    slots = torch.arange(12, device="cuda")
    g.qk_norm_rotary_cache_fp4(pos, freqs, q, k, v, slots, kc, vc, qw, kw)
    rk, rv = g.cache_fp4_rows(slots, kc, vc)
    same(rv, fp4_nearest(v))
    assert torch.isnan(rv[6, 1, 32:]).all() and not torch.isnan(rv[6, 1, :32]).any()  # the group of 32
    bad = torch.isnan(rk)
    assert bad[5, 0].any() and int(bad.sum()) == int(bad[5, 0].sum())
    grads = g.qk_norm_rotary_bwd(pos, freqs, q, k, clean[0], clean[1], qw, kw)
    assert torch.isnan(grads["dq"][3, 1]).all() and int(torch.isnan(grads["dq"]).sum()) == 64


def test_no_tokens(g):
    import torch
    q, k, v, pos, freqs, qw, kw, _ = make(1, 0, 4, 2, 64, 32, torch.bfloat16, wide=False)
    y, z = g.qk_norm_rotary(pos, freqs, q, k, qw, kw)
    assert y.shape == (0, 4, 64) and z.shape == (0, 2, 64)
    out = {"dq_weight": torch.full((64,), 3.0, device="cuda"), "dk_weight": torch.full((64,), 3.0, device="cuda")}
    got = g.qk_norm_rotary_bwd(pos, freqs, q, k, y, z, qw, kw, out=out)
    assert got["dq_weight"] is out["dq_weight"] and not got["dq_weight"].any() and not got["dk_weight"].any()
    c = g.cache_fp4(2, 2, 16, 64)
    g.qk_norm_rotary_cache_fp4(pos, freqs, q, k, v, pos.long(), c, c, qw, kw)
    # a cache of no pages takes nothing
    q, k, v, pos, freqs, qw, kw, _ = make(1, 3, 4, 2, 64, 32, torch.bfloat16)
    none = g.cache_fp4(0, 2, 16, 64)
    same(g.qk_norm_rotary_cache_fp4(pos, freqs, q, k, v, pos.long(), none, none, qw, kw), g.qk_norm_rotary(pos, freqs, q, k, qw, kw)[0].cpu().double())
    assert not g.cache_fp4_rows(pos.long(), none).any()


def test_offsets_beyond_32_bits(g):
    """A cache of 4.5 GB of codes: slots behind 2^32 bytes, written and read back."""
    import torch
    pages, Hk, page, d = 70000, 8, 64, 256
    T = 40
    q, k, v, pos, freqs, _, kw, _ = make(2, T, 1, Hk, d, 64, torch.bfloat16)
    kc, vc = ((torch.empty((pages, Hk, page, d // 2), dtype=torch.uint8, device="cuda"),
               torch.empty((pages, Hk, d // 32, page), dtype=torch.uint8, device="cuda")) for _ in range(2))
    assert kc[0].numel() > 2 ** 32
    slots = pages * page - 1 - 3 * torch.arange(T, device="cuda")
    slots[0] = 0
    g.qk_norm_rotary_cache_fp4(pos, freqs, q, k, v, slots, kc, vc, None, kw)
    rk, rv = g.cache_fp4_rows(slots, kc, vc)
    same(rv, fp4_nearest(v))
    same(rk, fp4_nearest(norm_rotary64(leaf(k).detach(), leaf(kw).detach(), pos, freqs, False, 1.0, EPS)))


def test_captured_on_another_stream_and_replayed(g):
    """Forward, reverse mode and the cache's forms in one graph, replayed with eager work
    between: each replay as the eager calls on the same inputs."""
    import torch
    T = 50
    q, k, v, pos, freqs, qw, kw, rnd = make(4, T, 4, 2, 64, 64, torch.bfloat16, wide=False)
    dq, dk = rnd(T, 4, 64).bfloat16(), rnd(T, 2, 64).bfloat16()
    kc, vc, slots = g.cache_fp4(5, 2, 16, 64), g.cache_fp4(5, 2, 16, 64), page_slots(T, 5, 16, 3)

    def calls(kc, vc):
        y, z = g.qk_norm_rotary(pos, freqs, q, k, qw, kw)
        grads = g.qk_norm_rotary_bwd(pos, freqs, q, k, dq, dk, qw, kw)
        y4 = g.qk_norm_rotary_cache_fp4(pos, freqs, q, k, v, slots, kc, vc, qw, kw)
        return [y, z, y4, *grads.values(), *g.cache_fp4_rows(slots, kc, vc)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        calls(kc, vc)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = calls(kc, vc)
    for i in range(3):
        q.copy_(rnd(*q.shape))
        k.copy_(rnd(*k.shape))
        v.copy_(rnd(*v.shape))
        graph.replay()
        torch.cuda.synchronize()
        want = calls(g.cache_fp4(5, 2, 16, 64), g.cache_fp4(5, 2, 16, 64))
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert a.equal(b)


def test_autograd(g):
    """The differentiable form's gradients are the reverse mode's; broadcast and transposed
    inputs and gradients are taken; an unused output counts as zero."""
    import torch
    from gated_deltanet_dual_amd import autograd
    q, k, _, pos, freqs, qw, kw, rnd = make(6, 30, 4, 2, 64, 32, torch.bfloat16, wide=False)
    leaves = [t.detach().requires_grad_() for t in (q, k, qw, kw)]
    y, z = autograd.qk_norm_rotary(pos, freqs, *leaves)
    dy, dz = rnd(30, 4, 64).bfloat16(), rnd(30, 2, 64).bfloat16()
    torch.autograd.backward([y, z], [dy, dz])
    want = g.qk_norm_rotary_bwd(pos, freqs, q, k, dy, dz, qw, kw)
    for t, name in zip(leaves, ("dq", "dk", "dq_weight", "dk_weight")):
        assert t.grad.equal(want[name]), name
    # a gradient that is one number for all, a query that is the same for all heads
    one = rnd(30, 1, 64).bfloat16().requires_grad_()
    y, z = autograd.qk_norm_rotary(pos, freqs, one.expand(30, 4, 64), leaves[1], leaves[2], leaves[3])
    for t in leaves:
        t.grad = None
    y.float().sum().backward()
    want = g.qk_norm_rotary_bwd(pos, freqs, one.detach().expand(30, 4, 64).contiguous(), k, torch.ones_like(q), torch.zeros_like(k), qw, kw)
    assert leaves[1].grad.equal(want["dk"]) and not leaves[1].grad.any() and leaves[2].grad.equal(want["dq_weight"])
    close(one.grad, want["dq"].cpu().double().sum(1, keepdim=True), torch.bfloat16, 2.0 ** -7 * want["dq"].cpu().double().abs().sum(1, keepdim=True))
    # queries alone, not normed
    x = q.detach().requires_grad_()
    y, none = autograd.qk_norm_rotary(pos, freqs, x)
    y.backward(dy)
    assert none is None and x.grad.equal(g.rotary(pos, freqs, dy, inverse=True)[0])


def test_refusals(g):
    import torch
    q, k, v, pos, freqs, qw, kw, _ = make(1, 6, 4, 2, 64, 32, torch.bfloat16, wide=False)
    c, slots = g.cache_fp4(2, 2, 16, 64), torch.arange(6, device="cuda")
    for bad in (lambda: g.qk_norm_rotary(pos, freqs, q, None, qw, kw), lambda: g.qk_norm_rotary(pos, freqs, q, k, qw[:32], kw),
                lambda: g.qk_norm_rotary(pos, freqs, q, k, qw.double(), kw), lambda: g.qk_norm_rotary(pos, freqs, q, k, qw, kw, eps=-1.0),
                lambda: g.qk_norm_rotary(pos, freqs, q, k.float(), qw, kw), lambda: g.qk_norm_rotary(pos[:5], freqs, q, k, qw, kw),
                lambda: g.qk_norm_rotary(pos, freqs, q.transpose(1, 2), None, qw),
                lambda: g.qk_norm_rotary_bwd(pos, freqs, q, k, q, None, qw, kw), lambda: g.qk_norm_rotary_bwd(pos, freqs, q, None, q, k, qw),
                lambda: g.qk_norm_rotary_bwd(pos, freqs, q, k, q, k, qw, kw, workspace=torch.empty(10, dtype=torch.uint8, device="cuda")),
                lambda: g.qk_norm_rotary_cache(pos, freqs, q, k, None, slots, q, q), lambda: g.qk_norm_rotary_cache(pos, freqs, q, k, v, slots, c, c),
                lambda: g.qk_norm_rotary_cache_fp4(pos, freqs, q, k, v, slots, c[0], c[0]),
                lambda: g.qk_norm_rotary_cache_fp4(pos, freqs, q, k, v, slots.int(), c, c),
                lambda: g.qk_norm_rotary_cache_fp4(pos, freqs, q, k, v, slots, c, g.cache_fp4(3, 2, 16, 64)),
                lambda: g.qk_norm_rotary_cache_fp4(pos, freqs, q, k, v, slots, c, tuple(t.cpu() for t in c)),
                lambda: g.qk_norm_rotary_cache_fp4(pos, freqs, q[..., :48].contiguous(), k[..., :48].contiguous(), v[..., :48].contiguous(), slots, c, c),
                lambda: g.cache_fp4_rows(slots, c[0]), lambda: g.cache_fp4_rows(slots, c, dtype=torch.float16),
                lambda: g.cache_fp4_rows(slots, c, g.cache_fp4(2, 2, 32, 64)), lambda: g.cache_fp4_rows(slots[None], c)):
        with pytest.raises(g.FlareError):
            bad()


def test_two_streams_at_once(g):
    """Calls under way together, each with its own workspace and cache, give the bits of one
    after the other."""
    import torch
    sets = []
    for seed, T, Hq, Hk, d, rot, io in ((7, 3000, 8, 2, 128, 64, torch.bfloat16), (8, 700, 3, 2, 96, 34, torch.float32)):
        q, k, v, pos, freqs, qw, kw, rnd = make(seed, T, Hq, Hk, d, rot, io)
        sets.append((pos, freqs, q, k, v, qw, kw, rnd(T, Hq, d).to(io), rnd(T, Hk, d).to(io), torch.randperm(4096, device="cuda")[:T]))

    def calls(i):
        pos, freqs, q, k, v, qw, kw, dq, dk, slots = sets[i]
        kc, vc = g.cache_fp4(64, k.shape[1], 64, k.shape[2]), g.cache_fp4(64, k.shape[1], 64, k.shape[2])
        grads = g.qk_norm_rotary_bwd(pos, freqs, q, k, dq, dk, qw, kw)
        return [*g.qk_norm_rotary(pos, freqs, q, k, qw, kw), *grads.values(),
                g.qk_norm_rotary_cache_fp4(pos, freqs, q, k, v, slots, kc, vc, qw, kw), *kc, *vc, *g.cache_fp4_rows(slots, kc, vc)]

    want = [calls(0), calls(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        got = [[], []]
        for _ in range(4):
            for i, s in enumerate(streams):
                with torch.cuda.stream(s):
                    got[i].append(calls(i))
        torch.cuda.synchronize()
        assert all(a.equal(b) for i in range(2) for one in got[i] for a, b in zip(one, want[i]))


@pytest.mark.parametrize("half", [4, 36, 252, 508])
def test_interleaved_heads_of_an_item_more_than_lanes(g, half):
    """bf16 heads of 1024 whose turned part and whose rest both end in half an item of two
    vectors of 8: 65 items for 64 lanes."""
    test_forms(g, 6, 2, 1, 1024, 2 * half, True, "bf16", "qk")
    test_cache_fp4(g, 9, 3, 2, 1024, 2 * half, True, "bf16", "qk", 16)


@pytest.mark.parametrize("inter", [False, True])
def test_coefficients_of_fp32_rows(g, inter):
    """Rows whose pairs are (1, 0) come out as the cosine and sine themselves, in reverse as the
    cosine and the negative sine: off by 4 half steps (two units of the functions) and one of the
    last sum, relative to the value also where it is near 0; what 64 bits leave of 4096 radians
    is 4e-12."""
    import torch
    T, d = 4096, 64
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    freqs = 10000.0 ** (-torch.arange(d // 2, dtype=torch.float64, device="cuda") / (d // 2))
    re = torch.arange(d // 2, device="cuda") * (2 if inter else 1)
    im = re + (1 if inter else d // 2)
    x = torch.zeros(T, 1, d, device="cuda")
    x[..., re] = 1.0
    angle = pos.cpu().double()[:, None] * freqs.cpu()
    c, s = torch.cos(angle), torch.sin(angle)
    y, z = g.qk_norm_rotary(pos, freqs, x, x, interleaved=inter)
    back = g.qk_norm_rotary_bwd(pos, freqs, x, x, x, x, interleaved=inter)
    for got, sign in ((y, 1), (z, 1), (back["dq"], -1), (back["dk"], -1)):
        for at, want in ((re, c), (im, sign * s)):
            off = (got[:, 0, at].cpu().double() - want).abs()
            assert (off <= 5 * STEP * want.abs() + 4e-12).all(), float((off / want.abs().clamp(min=1e-9)).max() / STEP)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_weights_sums_of_many_teams(g, io):
    """256 heads of 8 channels of one token, a team of a workgroup each: gradients whose sum in
    32 bits would lose the small ones beside two large ones of either sign.  Rows of ones have a
    norm of 1, so that every term is a gradient itself."""
    import torch
    io = types(io)
    H, d = 256, 8
    x = torch.ones(1, H, d, device="cuda").to(io)
    dy = torch.ones(1, H, d, device="cuda").to(io)
    dy[0, 0], dy[0, H - 1] = 2.0 ** 25, -2.0 ** 25
    dy[0, 1] = torch.arange(d).to(io)
    pos, freqs = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.float64, device="cuda")
    w = torch.ones(d, device="cuda")
    out = g.qk_norm_rotary_bwd(pos, freqs, x, None, dy, None, w, eps=0.0)
    assert out["dq_weight"].tolist() == [H - 3.0 + i for i in range(d)]
