"""Rotary positions and their serving form against complex products in 64
bits.  Tolerances: the last rounding is half a step; before it the coefficients
are off by at most 4 * 2^-24 (angle in turns to fp32, 2 pi * 2^-25, and 2 steps of
sin / cos) and the two products and their sum by 3 * 2^-24, of the pair's size:
8e-7 * sqrt(2) * |x| * mscale, bounded below by 1.2e-6 of the largest input."""
import pytest

from layer_oracle import close, rotary64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import gated_deltanet_dual_amd as g
    g.lib()
    return g


def rnd(seed, *shape, io="bf16"):
    import torch
    t = torch.randn(shape, generator=torch.Generator().manual_seed(seed))
    return t.to(torch.bfloat16 if io == "bf16" else torch.float32).cuda()


def slack(x, m):
    return 1.2e-6 * float(x.abs().max()) * m if x.numel() else 0.0


# (T, Hq, Hk, d, rot): whole heads, part of a head, none of it, odd channel
# counts, halves that are no multiple of a vector, no k heads, no tokens
SHAPES = [(1, 1, 1, 64, 64), (5, 4, 2, 128, 32), (37, 3, 1, 80, 20), (9, 2, 2, 66, 22), (3, 2, 1, 7, 4), (4, 2, 1, 64, 0),
          (6, 5, 0, 128, 128), (0, 2, 1, 64, 64), (9000, 2, 1, 64, 16), (2, 1, 1, 1024, 1024)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,d,rot", SHAPES)
def test_rotary(g, T, Hq, Hk, d, rot, inter, io):
    import torch
    freqs, m = g.rotary_frequencies(rot, scaling="yarn", factor=4.0, original_length=4096)
    pos = torch.randint(0, 2 ** 31 - 1, (T,), generator=torch.Generator().manual_seed(1), dtype=torch.int64).to(torch.int32).cuda()
    if T > 2:
        pos[0], pos[1] = 0, -5
    rows = rnd(2, T, (Hq + 2 * Hk) * d, io=io)
    q, k = rows[:, :Hq * d].unflatten(1, (Hq, d)), rows[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d)) if Hk else None
    for sign in (1.0, -1.0):
        qo, ko = g.rotary(pos, freqs, q, k, interleaved=inter, mscale=m, inverse=sign < 0)
        torch.cuda.synchronize()
        close(qo, rotary64(q, pos, freqs, inter, m, sign), q.dtype, slack(q, m), "q")
        assert torch.equal(qo[..., rot:], q[..., rot:])
        if Hk:
            close(ko, rotary64(k, pos, freqs, inter, m, sign), q.dtype, slack(k, m), "k")
        else:
            assert ko is None


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("page", [1, 16, 48])
def test_rotary_cache(g, page, inter, io):
    """Live rows land in their slots as rotary() gives them; padded rows and slots
    beyond the cache write nothing; everything else in the pages is left as it was."""
    import torch
    T, Hq, Hk, d, rot = 41, 4, 2, 64, 32
    freqs, m = g.rotary_frequencies(rot)
    pages = -(-T // page) + 3
    perm = torch.randperm(pages * page, generator=torch.Generator().manual_seed(3))[:T].cuda()
    perm[5], perm[11], perm[40] = -1, pages * page, -2 ** 40
    pos = torch.arange(T, dtype=torch.int32).cuda() + 100000
    q, k, v = rnd(1, T, Hq, d, io=io), rnd(2, T, Hk, d, io=io), rnd(3, T, 2 * Hk * d, io=io)[:, 8:8 + Hk * d].unflatten(1, (Hk, d))
    kc, vc = rnd(4, pages, Hk, page, d, io=io), rnd(5, pages, Hk, page, d, io=io)
    wk, wv = kc.clone(), vc.clone()
    qo = g.rotary_cache(pos, freqs, q, k, v, perm, kc, vc, interleaved=inter, mscale=m)
    qr, kr = g.rotary(pos, freqs, q, k, interleaved=inter, mscale=m)
    for t in range(T):
        s = int(perm[t])
        if 0 <= s < pages * page:
            wk[s // page, :, s % page], wv[s // page, :, s % page] = kr[t], v[t]
    assert torch.equal(qo, qr) and torch.equal(kc, wk) and torch.equal(vc, wv)


def test_rotary_keeps_relative_positions(g):
    """q.k of turned rows depends on the distance of their positions alone."""
    import torch
    freqs, _ = g.rotary_frequencies(64)
    q, k = rnd(1, 1, 1, 64, io="f32").expand(4, 1, 64).contiguous(), rnd(2, 1, 1, 64, io="f32").expand(4, 1, 64).contiguous()
    pq = torch.tensor([10, 1010, 1000010, 5], dtype=torch.int32).cuda()
    qo, _ = g.rotary(pq, freqs, q)
    ko, _ = g.rotary(pq - 7, freqs, k)
    dots = (qo.double() * ko.double()).sum((1, 2)).cpu()
    # each coefficient off by 4 * 2^-24 of values up to 4, over 64 channels
    assert float((dots - dots[0]).abs().max()) <= 64 * 16 * 8 * 2.0 ** -24
