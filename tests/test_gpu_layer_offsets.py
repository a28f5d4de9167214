"""Places beyond 32 bits: token strides, rows and cache pages whose offset passes
2^31 and 2^32 elements give, bit for bit, what the same numbers give close to the
start of a small buffer (a row's arithmetic does not depend on where it lies)."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import gated_deltanet_dual_amd as g
    g.lib()
    return g


def rnd(seed, *shape, io="bf16"):
    import torch
    t = torch.randn(*shape, generator=torch.Generator().manual_seed(seed))
    return t.to(torch.bfloat16 if io == "bf16" else torch.float32).cuda()


def far(t, stride):
    """t [T, ...] with `stride` elements between its tokens."""
    import torch
    row = t[0].numel()
    buf = torch.empty((t.shape[0] - 1) * stride + row, dtype=t.dtype, device=t.device)
    view = buf.as_strided(t.shape, (stride,) + t.stride()[1:])
    view.copy_(t)
    return view


def test_token_strides(g):
    import torch
    x, gate, w = rnd(1, 3, 2, 64), rnd(2, 3, 2, 64), rnd(3, 64, io="f32")
    fx, fg = far(x, 2 ** 30 + 8), far(gate, 2 ** 30 + 3)
    y, rstd = g.gated_norm(x, w, gate, want_rstd=True)
    fy, frstd = g.gated_norm(fx, w, fg, want_rstd=True)
    assert torch.equal(y, fy) and torch.equal(rstd, frstd)
    dy = rnd(4, 3, 2, 64)
    for a, b in zip(g.gated_norm_bwd(x, w, gate, dy, rstd), g.gated_norm_bwd(fx, w, fg, far(dy, 2 ** 30 + 1), rstd)):
        assert torch.equal(a, b)
    freqs, _ = g.rotary_frequencies(32)
    pos = torch.tensor([0, 70000, 2 ** 31 - 1], dtype=torch.int32).cuda()
    for a, b in zip(g.rotary(pos, freqs, x, gate), g.rotary(pos, freqs, fx, fg)):
        assert torch.equal(a, b)


def test_many_rows(g):
    import torch
    C, n = 16384, 3
    T = 2 ** 31 // C + n  # the last three rows lie behind 2^31 elements
    parts = {k: rnd(i, n, C, io=io) for i, (k, io) in enumerate([("x", "bf16"), ("res", "f32"), ("dy", "bf16"), ("dh", "f32")])}
    big = {}
    for k, v in parts.items():
        big[k] = torch.zeros(T, C, dtype=v.dtype, device="cuda")
        big[k][-n:] = v
    w = rnd(9, C, io="f32")
    h, y, rstd = g.residual_norm(parts["x"], parts["res"], w, w_post=w, want_rstd=True)
    bh, by, brstd = g.residual_norm(big["x"], big["res"], w, w_post=w, want_rstd=True)
    assert torch.equal(h, bh[-n:]) and torch.equal(y, by[-n:]) and torch.equal(rstd, brstd[-n:])
    del bh, by
    a = g.residual_norm_bwd(parts["x"], parts["res"], w, parts["dy"], parts["dh"], rstd, w_post=w)
    b = g.residual_norm_bwd(big["x"], big["res"], w, big["dy"], big["dh"], brstd, w_post=w)
    for k in ("dx", "dresidual"):
        assert torch.equal(a[k], b[k][-n:]), k


@pytest.mark.parametrize("d", [64, 128, 256])
def test_cache_pages(g, d):
    """Pages at the end of a cache of more than 2^32 elements, written and read."""
    import torch
    Hk, page, R, B, n = 8, 64, 2, 3, 100
    pages = 2 ** 32 // (Hk * page * d) + 6
    table = torch.tensor([[0, 2], [3, 1]], dtype=torch.int32).cuda()
    shared = torch.tensor([5, 4], dtype=torch.int32).cuda()
    lens = torch.tensor([n, 70], dtype=torch.int32).cuda()
    freqs, _ = g.rotary_frequencies(d)
    q = rnd(1, R * B, 2 * Hk, d)
    out = []
    for first, size in ((0, 6), (pages - 6, pages)):
        kc, vc = (torch.empty(size, Hk, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        k, v = rnd(2, 6 * page, Hk, d), rnd(3, 6 * page, Hk, d)
        slots = torch.arange(6 * page, device="cuda") + first * page
        pos = torch.arange(6 * page, dtype=torch.int32, device="cuda")
        g.rotary_cache(pos, freqs, rnd(4, 6 * page, 1, d), k, v, slots, kc, vc)
        for causal in (False, True):
            out.append(g.block_attention(q.view(R, B, 2 * Hk, d), kc, vc, table + first, lens, prefix_table=shared + first,
                                         prefix_len=90, causal=causal))
        assert torch.equal(vc[first:].transpose(1, 2).reshape(6 * page, Hk, d), v)
        del kc, vc
    assert torch.equal(out[0], out[2]) and torch.equal(out[1], out[3]) and bool(torch.isfinite(out[0].float()).all())


def test_bounds_beyond_32_bits_are_refused(g):
    import torch
    page = 2 ** 14
    cache = torch.zeros(1, 1, page, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(1, 2 ** 18, dtype=torch.int32, device="cuda")  # holds 2^32 keys
    lens = torch.tensor([5], dtype=torch.int32).cuda()
    q = rnd(1, 1, 1, 1, 64)
    with pytest.raises(g.FlareError, match="beyond 32 bits"):
        g.block_attention(q, cache, cache, table, lens)
    assert bool((g.block_attention(q, cache, cache, table, lens, max_seq_len=5) == 0).all())
    with pytest.raises(g.FlareError, match="beyond 32 bits"):
        g.block_attention(q, cache, cache, table, lens, max_seq_len=5, prefix_len=2 ** 32)
    with pytest.raises(g.FlareError, match="beyond 32 bits"):
        g.step_tables(lens, lens.clone(), table, table[0], torch.zeros(1, dtype=torch.int32).cuda(), 2 ** 32 + 16, 4)
