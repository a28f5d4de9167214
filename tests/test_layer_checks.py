"""Refusals of the operators around the GDN step, on the CPU: the C entry points
validate before anything is launched (device pointers are dummies, never
dereferenced), the binding refuses host tensors, and the workspace sizes and
rotary frequencies are what their formulas say."""
import ctypes
import math

import numpy as np
import pytest
import torch

import gated_deltanet_dual_amd as g

FAKE = 0x7F0000001000


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(g.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return g.lib()


def gated(L, tokens=4, heads=2, dim=64, io=g.BF16, x=FAKE, xs=128, gate=FAKE, gs=128, w=FAKE, act=1, eps=1e-6, y=FAKE):
    return L.flare_gated_norm(tokens, heads, dim, io, x, xs, gate, gs, w, act, eps, y, None, None)


def test_gated_norm(L):
    assert gated(L, tokens=-1) == 2 and gated(L, heads=0) == 2 and gated(L, dim=0) == 2
    assert gated(L, dim=16385, xs=40000, gs=40000) == 4 and gated(L, io=2) == 4 and gated(L, act=3) == 4
    assert gated(L, tokens=2 ** 31) == 4 and gated(L, tokens=2 ** 30, heads=4, xs=256, gs=256) == 4
    assert gated(L, xs=127) == 2 and gated(L, gs=127) == 2
    assert gated(L, x=None) == 1 and gated(L, w=None) == 1 and gated(L, y=None) == 1
    assert gated(L, eps=-1.0) == 2 and gated(L, eps=math.nan) == 2 and gated(L, eps=math.inf) == 2
    assert gated(L, tokens=0, x=None, w=None, y=None) == 0  # nothing to do
    # without a gate its stride and activation are not looked at, its row is
    assert gated(L, gate=None, gs=0, act=9, y=None) == 1
    assert b"y is NULL" in L.flare_last_error()


def gated_bwd(L, tokens=4, ws=FAKE & ~255, nbytes=1 << 30, dw=FAKE, rstd=FAKE, dg=FAKE, ds=128):
    return L.flare_gated_norm_bwd(tokens, 2, 64, g.BF16, FAKE, 128, FAKE, 128, FAKE, 1, rstd, FAKE, ds, FAKE, dg, dw,
                                  ws, nbytes, None)


def test_gated_norm_bwd(L):
    need = g.gated_norm_bwd_workspace_bytes(4, 2, 64)
    assert need == 8 * 64 * 4 + 256
    assert g.gated_norm_bwd_workspace_bytes(1 << 20, 16, 128) == 1536 * 128 * 4 + 256
    assert g.gated_norm_bwd_workspace_bytes(1 << 20, 1, 2048) == 768 * 2048 * 4 + 256
    assert g.gated_norm_bwd_workspace_bytes(-1, 2, 64) == 0 and g.gated_norm_bwd_workspace_bytes(4, 0, 64) == 0
    assert gated_bwd(L, nbytes=need - 1) == 5 and gated_bwd(L, ws=None) == 5 and gated_bwd(L, ws=(FAKE & ~255) + 16) == 5
    assert gated_bwd(L, dw=None) == 1 and gated_bwd(L, rstd=None) == 1 and gated_bwd(L, dg=None) == 1
    assert gated_bwd(L, ds=127) == 2


def residual(L, tokens=4, dim=64, io=g.BF16, res=g.F32, xs=64, r=FAKE, gs=64, act=1, w=FAKE, h=FAKE, eps=1e-6):
    return L.flare_residual_norm(tokens, dim, io, res, FAKE, xs, r, FAKE, gs, w, None, None, act, eps, h, FAKE, None, None)


def test_residual_norm(L):
    assert residual(L, tokens=-1) == 2 and residual(L, dim=0) == 2 and residual(L, xs=63) == 2 and residual(L, gs=63) == 2
    assert residual(L, io=g.F32, res=g.BF16) == 4 and residual(L, res=5) == 4 and residual(L, act=-2) == 4
    assert residual(L, dim=20000, xs=20000, gs=20000) == 4 and residual(L, tokens=2 ** 31) == 4
    assert residual(L, r=None) == 1 and residual(L, w=None) == 1 and residual(L, h=None) == 1
    assert residual(L, eps=-1e-3) == 2 and residual(L, tokens=0, r=None) == 0
    assert g.residual_norm_bwd_workspace_bytes(4, 64) == 3 * 4 * 64 * 4 + 256
    bwd = lambda dwp=FAKE, post=None, dpost=None, n=1 << 30: L.flare_residual_norm_bwd(  # noqa: E731
        4, 64, g.BF16, g.F32, FAKE, 64, FAKE, None, 0, FAKE, post, None, 0, FAKE, FAKE, None, FAKE, FAKE, None, dwp, dpost,
        None, FAKE & ~255, n, None)
    assert bwd(dwp=None) == 1 and bwd(post=FAKE) == 1 and bwd(n=100) == 5


def rotary(L, tokens=4, qh=2, kh=1, dim=64, half=16, io=g.BF16, inter=0, pos=FAKE, freqs=FAKE, qs=128, ks=64, inv=0, ko=FAKE):
    s = g.RotaryShape(qh, kh, dim, half, io, inter, 1.0)
    return L.flare_rotary(tokens, ctypes.byref(s), pos, freqs, FAKE, qs, FAKE, ks, inv, FAKE, ko, None)


def test_rotary(L):
    assert rotary(L, tokens=-1) == 2 and rotary(L, qh=0) == 2 and rotary(L, kh=-1) == 2 and rotary(L, dim=0) == 2
    assert rotary(L, half=33) == 2 and rotary(L, half=-1) == 2 and rotary(L, qs=127) == 2 and rotary(L, ks=63) == 2
    assert rotary(L, dim=2048, qs=4096, ks=2048) == 4 and rotary(L, io=7) == 4 and rotary(L, inter=2) == 4
    assert rotary(L, inv=2) == 4 and rotary(L, tokens=2 ** 31) == 4
    assert rotary(L, pos=None) == 1 and rotary(L, freqs=None) == 1 and rotary(L, ko=None) == 1
    assert rotary(L, tokens=0, pos=None, freqs=None, ko=None) == 0
    assert L.flare_rotary(4, None, FAKE, FAKE, FAKE, 128, FAKE, 64, 0, FAKE, FAKE, None) == 1
    s = g.RotaryShape(2, 1, 64, 16, g.BF16, 0, 1.0)
    cache = lambda s=s, vs=64, slots=FAKE, kc=FAKE, pages=8, page=16: L.flare_rotary_cache(  # noqa: E731
        4, ctypes.byref(s), FAKE, FAKE, FAKE, 128, FAKE, 64, FAKE, vs, slots, FAKE, kc, FAKE, pages, page, None)
    assert cache(vs=63) == 2 and cache(slots=None) == 1 and cache(kc=None) == 1
    assert cache(pages=-1) == 2 and cache(page=0) == 2 and cache(s=g.RotaryShape(2, 0, 64, 16, g.BF16, 0, 1.0)) == 2


def tables(L, R=2, lens=FAKE, new=FAKE + 64, bt=FAKE, wide=4, free=FAKE, F=10, used=FAKE, page=16, off=0, M=8, pos=FAKE,
           lens_out=FAKE + 128, used_out=FAKE + 192, status=FAKE):
    return L.flare_step_tables(R, lens, new, bt, wide, free, F, used, page, off, M, FAKE, pos, FAKE, lens_out, used_out,
                               status, None)


def test_step_tables(L):
    for bad in (dict(R=-1), dict(wide=-1), dict(F=-1), dict(M=-1), dict(off=-1), dict(page=0)):
        assert tables(L, **bad) == 2, bad
    assert tables(L, R=8193) == 4 and tables(L, F=2 ** 31) == 4 and tables(L, M=2 ** 31) == 4
    for bad in ("lens", "new", "bt", "free", "used", "pos", "lens_out", "used_out", "status"):
        assert tables(L, **{bad: None}) == 1, bad
    # an output that is its own input
    assert tables(L, lens_out=FAKE) == 2 and tables(L, used_out=FAKE) == 2


def attention(L, R=2, block=4, qh=8, kh=2, d=128, page=64, io=g.BF16, causal=0, scale=0.0, q=FAKE, pages=100, bt=FAKE, wide=8,
              lens=FAKE, most=512, pt=FAKE, n=5000, ws=FAKE & ~255, nbytes=1 << 40):
    s = g.AttentionShape(block, qh, kh, d, page, io, causal, scale)
    return L.flare_block_attention(R, ctypes.byref(s), q, FAKE, FAKE, pages, bt, wide, lens, most, pt, n, FAKE, None, ws,
                                   nbytes, None)


def test_block_attention(L):
    for bad in (dict(R=-1), dict(block=0), dict(qh=0), dict(kh=0), dict(kh=3), dict(most=-1), dict(n=-1), dict(pages=-1),
                dict(most=513), dict(pages=0), dict(scale=math.inf), dict(scale=math.nan), dict(scale=-math.inf)):
        assert attention(L, **bad) == 2, bad
    for bad in (dict(d=16), dict(d=96), dict(page=8), dict(page=48), dict(io=g.F32), dict(causal=2), dict(R=2 ** 24),
                dict(n=2 ** 31 - 1)):
        assert attention(L, **bad) == 4, bad
    for bad in ("q", "bt", "lens", "pt"):
        assert attention(L, **{bad: None}) == 1, bad
    assert attention(L, q=FAKE + 8) == 3
    need = g.block_attention_workspace_bytes(2, 4, 8, 2, 128, 64, 512, 5000)
    assert need > 0 and attention(L, nbytes=need - 1) == 5 and attention(L, ws=None) == 5
    assert attention(L, ws=(FAKE & ~255) + 64) == 5
    assert attention(L, R=0, q=None, lens=None, bt=None, pt=None) == 0
    # one part alone is written without a workspace, a short prefix in it
    assert g.block_attention_workspace_bytes(2, 4, 8, 2, 128, 64, 64, 0) == 0
    assert g.block_attention_workspace_bytes(2, 4, 8, 2, 128, 64, 64, 100) == 0
    assert g.block_attention_workspace_bytes(2, 4, 8, 2, 100, 64, 512, 100) == 0  # not instantiated


@pytest.mark.parametrize("R,B,Hq,Hk,d,own,prefix", [(1, 1, 1, 1, 64, 1, 0), (256, 4, 16, 4, 128, 1024, 8192), (3, 7, 16, 2, 256, 777, 2500),
                                                    (1, 1, 16, 4, 128, 1 << 20, 0), (64, 1, 8, 8, 64, 0, 1 << 22), (5, 32, 8, 1, 128, 40, 40)])
def test_attention_workspace_is_rows_times_parts(L, R, B, Hq, Hk, d, own, prefix):
    """The workspace holds d + 2 floats a row and part, plus its alignment; the
    parts of at most 4096 keys (2048 at d = 256) cover the lengths."""
    n = g.block_attention_workspace_bytes(R, B, Hq, Hk, d, 16, own, prefix)
    longest = 2048 if d == 256 else 4096
    if n == 0:
        assert own + prefix <= longest
        return
    parts, rest = divmod(n - 256, R * B * Hq * (d + 2) * 4)
    assert rest == 0 and parts >= -(-own // longest) + -(-prefix // longest) and parts >= 2


def test_rotary_frequencies():
    f, m = g.rotary_frequencies(8, device="cpu")
    assert m == 1.0 and f.dtype == torch.float64 and f.tolist() == [10000.0 ** (-i / 4) for i in range(4)]
    assert g.rotary_frequencies(8, scaling="linear", factor=4.0, device="cpu")[0].tolist() == (f / 4).tolist()
    ntk = g.rotary_frequencies(8, scaling="ntk", factor=4.0, device="cpu")[0]
    assert ntk[0] == 1.0 and math.isclose(float(ntk[3]), float(f[3]) / 4, rel_tol=1e-12)
    y, m = g.rotary_frequencies(64, scaling="yarn", factor=4.0, original_length=4096, device="cpu")
    base = g.rotary_frequencies(64, device="cpu")[0]
    turns = 4096 * base / (2 * math.pi)
    assert m == 1 + 0.1 * math.log(4.0)
    # rounding the ramp's ends outwards to whole pairs leaves the pairs beyond them as they are
    assert torch.equal(y[turns > 40], base[turns > 40]) and torch.equal(y[turns < 0.75], base[turns < 0.75] / 4)
    assert (y <= base).all() and (y >= base / 4).all()
    assert g.rotary_frequencies(0, device="cpu")[0].numel() == 0
    for bad in (dict(rotary_dim=7), dict(rotary_dim=-2), dict(rotary_dim=8, factor=0.5), dict(rotary_dim=8, base=1.0),
                dict(rotary_dim=8, scaling="yarn"), dict(rotary_dim=8, scaling="other")):
        with pytest.raises(g.FlareError):
            g.rotary_frequencies(**bad, device="cpu")


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(2, 8), torch.ones(8)
    i32 = torch.zeros(2, dtype=torch.int32)
    calls = [lambda: g.gated_norm(x, w), lambda: g.gated_norm_bwd(x, w, None, x, x), lambda: g.residual_norm(x, x, w),
             lambda: g.residual_norm_bwd(x, x, w, x, x, x),
             lambda: g.rotary(i32, torch.zeros(4, dtype=torch.float64), torch.zeros(2, 1, 8)),
             lambda: g.step_tables(i32, i32, torch.zeros(2, 2, dtype=torch.int32), i32, i32[:1], 16, 4),
             lambda: g.block_attention(torch.zeros(2, 1, 1, 64, dtype=torch.bfloat16), None, None, None, None)]
    for call in calls:
        with pytest.raises(g.FlareError, match="GPU tensor"):
            call()


def test_token_rows():
    from gated_deltanet_dual_amd.layer import _token_rows
    cpu, f = torch.device("cpu"), torch.float32
    wide = torch.zeros(5, 20)
    assert _token_rows(wide, "x", (5, 20), f, cpu) == 20
    assert _token_rows(wide[:, 4:12].unflatten(1, (2, 4)), "x", (5, 2, 4), f, cpu) == 20
    assert _token_rows(wide[:1, 4:12], "x", (1, 8), f, cpu) == 8 and _token_rows(wide[:0, 4:12], "x", (0, 8), f, cpu) == 8
    assert _token_rows(torch.zeros(5, 1, 8).transpose(0, 1), "x", (1, 5, 8), f, cpu) == 40
    for bad in (wide.t(), wide[:, ::2], torch.zeros(1, 8).expand(5, 8), torch.zeros(8).expand(5, 3, 8)):
        with pytest.raises(g.FlareError):
            _token_rows(bad, "x", tuple(bad.shape), f, cpu)
    with pytest.raises(g.FlareError):
        _token_rows(wide, "x", (5, 19), f, cpu)
    with pytest.raises(g.FlareError):
        _token_rows(wide.double(), "x", (5, 20), f, cpu)


def test_fast_division_rule():
    """The quotient by a product, as the kernels form it: exact below 2^31."""
    rng = np.random.default_rng(1)
    for d in [1, 2, 3, 5, 7, 16, 48, 100, 257, 1000, 2 ** 20 - 1, 2 ** 30 + 1, 2 ** 31 - 1]:
        s = (d - 1).bit_length()
        m = (1 << (31 + s)) // d + 1
        assert m < 2 ** 32
        for n in [0, 1, d - 1, d, 2 ** 31 - 1, *(int(x) for x in rng.integers(0, 2 ** 31, 2000)), *(k * d - 1 for k in range(1, 2000))]:
            if 0 <= n < 2 ** 31:
                assert (n * m) >> (31 + s) == n // d, (d, n)


def test_sizes_whose_products_pass_32_bits(L):
    assert rotary(L, half=2 ** 30) == 2 and rotary(L, half=2 ** 31 - 1) == 2 and rotary(L, dim=63, half=32) == 2
    # 2^20 requests x 8 heads x 2^18 parts: more workgroups than a launch holds
    assert attention(L, R=2 ** 20, block=1, qh=8, kh=8, most=2 ** 30, wide=2 ** 10, page=2 ** 20, n=0, pt=None, nbytes=2 ** 62) == 4
    assert b"workgroups" in L.flare_last_error()
    from gated_deltanet_dual_amd.layer import _i32
    assert _i32(2 ** 31 - 1, "n") == 2 ** 31 - 1
    for bad in (2 ** 31, 2 ** 32, -2 ** 31 - 1):
        with pytest.raises(g.FlareError, match="beyond 32 bits"):
            _i32(bad, "n")


def test_step_tables_outputs_are_not_their_inputs(L):
    assert tables(L, lens_out=FAKE + 64) == 2  # the added lengths, read by every workgroup
