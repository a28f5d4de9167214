"""Refusals of the softmax layers' q/k norms, caches in 4 bits and their rows, on the CPU:
the C entry points validate before anything is launched (device pointers are dummies,
never dereferenced), and the binding refuses host tensors and wrong shapes."""
import ctypes
import math

import pytest
import torch

import gated_deltanet_dual_amd as g
from gated_deltanet_dual_amd import layer

FAKE = 0x7F0000001000
CPU = torch.device("cpu")


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(g.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return g.lib()


def shape(qh=2, kh=1, dim=64, half=16, io=g.BF16, inter=0):
    return ctypes.byref(g.RotaryShape(qh, kh, dim, half, io, inter, 1.0))


def forward(L, tokens=4, s=None, pos=FAKE, freqs=FAKE, qs=128, ks=64, qw=FAKE, kw=FAKE, eps=1e-6, qo=FAKE, ko=FAKE, **sizes):
    return L.flare_qk_norm_rotary(tokens, s or shape(**sizes), pos, freqs, FAKE, qs, FAKE, ks, qw, kw, eps, qo, ko, None)


def reverse(L, tokens=4, qs=128, ks=64, qw=FAKE, kw=FAKE, eps=1e-6, do=FAKE, dqs=128, dko=FAKE, dks=64, dq=FAKE, dk=FAKE,
            dqw=FAKE, dkw=FAKE, ws=FAKE & ~255, nbytes=1 << 30, **sizes):
    return L.flare_qk_norm_rotary_bwd(tokens, shape(**sizes), FAKE, FAKE, FAKE, qs, FAKE, ks, qw, kw, eps, do, dqs, dko, dks,
                                      dq, dk, dqw, dkw, ws, nbytes, None)


def cache(L, tokens=4, v=FAKE, vs=64, slots=FAKE, kc=FAKE, vc=FAKE, pages=8, page=16, eps=1e-6, kw=FAKE, **sizes):
    return L.flare_qk_norm_rotary_cache(tokens, shape(**sizes), FAKE, FAKE, FAKE, 128, FAKE, 64, v, vs, FAKE, kw, eps, slots,
                                        FAKE, kc, vc, pages, page, None)


def cache4(L, tokens=4, v=FAKE, vs=64, slots=FAKE, kc=FAKE, ks=FAKE, vc=FAKE, vsc=FAKE, pages=8, page=16, eps=1e-6, qs=128,
           kst=64, **sizes):
    return L.flare_qk_norm_rotary_cache_fp4(tokens, shape(**sizes), FAKE, FAKE, FAKE, qs, FAKE, kst, v, vs, FAKE, FAKE, eps,
                                            slots, FAKE, kc, ks, vc, vsc, pages, page, None)


def rows(L, n=4, heads=2, dim=64, io=g.BF16, slots=FAKE, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, pages=8, page=16, ko=FAKE,
         vo=FAKE):
    return L.flare_cache_fp4_rows(n, heads, dim, io, slots, kc, ks, vc, vs, pages, page, ko, vo, None)


def test_forward(L):
    for bad in (dict(tokens=-1), dict(qh=0), dict(kh=-1), dict(dim=0), dict(half=33), dict(half=2 ** 30), dict(qs=127),
                dict(ks=63), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(kh=0)):
        assert forward(L, **bad) == 2, bad  # kh = 0: a k_weight, but no k heads
    for bad in (dict(dim=2048, qs=4096, ks=2048), dict(io=7), dict(inter=2), dict(tokens=2 ** 31), dict(tokens=2 ** 24, qh=256, qs=16384)):
        assert forward(L, **bad) == 4, bad
    for bad in ("pos", "freqs", "qo", "ko"):
        assert forward(L, **{bad: None}) == 1, bad
    assert L.flare_qk_norm_rotary(4, None, FAKE, FAKE, FAKE, 128, FAKE, 64, None, None, 1e-6, FAKE, FAKE, None) == 1
    assert forward(L, tokens=0, pos=None, freqs=None, qo=None, ko=None) == 0


def test_reverse(L):
    need = g.qk_norm_rotary_bwd_workspace_bytes(4, 64)
    assert need == 2 * 4 * 64 * 4 + 256 and g.qk_norm_rotary_bwd_workspace_bytes(1 << 20, 128) == 2 * 1024 * 128 * 4 + 256
    assert g.qk_norm_rotary_bwd_workspace_bytes(-1, 64) == 0 and g.qk_norm_rotary_bwd_workspace_bytes(4, 1025) == 0
    with pytest.raises(g.FlareError, match="beyond 32 bits"):
        g.qk_norm_rotary_bwd_workspace_bytes(4, 2 ** 32 + 64)
    for bad in (dict(dqs=127), dict(dks=63), dict(qs=127), dict(eps=-1.0)):
        assert reverse(L, **bad) == 2, bad
    for bad in ("do", "dko", "dq", "dk", "dqw", "dkw"):
        assert reverse(L, **{bad: None}) == 1, bad
    assert reverse(L, nbytes=need - 1) == 5 and reverse(L, ws=None) == 5 and reverse(L, ws=(FAKE & ~255) + 16) == 5


def test_caches(L):
    for bad in (dict(vs=63), dict(pages=-1), dict(page=0), dict(pages=2 ** 31), dict(eps=math.nan)):
        assert cache(L, **bad) == 2 and cache4(L, **bad) == 2, bad
    assert cache(L, kh=0, kw=None) == 2
    for bad in ("v", "slots", "kc", "vc"):
        assert cache(L, **{bad: None}) == 1 and cache4(L, **{bad: None}) == 1, bad
    for bad in ("ks", "vsc"):
        assert cache4(L, **{bad: None}) == 1, bad
    for dim in (48, 80, 8):  # no groups of 32
        assert cache4(L, dim=dim, half=0, qs=2 * dim, kst=dim, vs=dim) == 4
    assert cache4(L, kc=FAKE + 8) == 3 and cache4(L, vc=FAKE + 4) == 3
    assert cache(L, tokens=0, slots=None, v=None) == 0 and cache4(L, tokens=0, slots=None, v=None) == 0


def test_rows(L):
    for bad in (dict(n=-1), dict(heads=0), dict(pages=-1), dict(page=0)):
        assert rows(L, **bad) == 2, bad
    for bad in (dict(io=2), dict(dim=48), dict(dim=2048), dict(heads=70000), dict(n=2 ** 31), dict(dim=0)):
        assert rows(L, **bad) == 4, bad
    for bad in ("slots", "kc", "ks", "vc", "vs", "ko"):
        assert rows(L, **{bad: None}) == 1, bad
    assert rows(L, ko=FAKE + 2) == 3 and rows(L, kc=FAKE + 1) == 3
    assert rows(L, n=0, slots=None, ko=None) == 0


def test_binding_refuses_host_tensors():
    q, pos, f = torch.zeros(2, 1, 64), torch.zeros(2, dtype=torch.int32), torch.zeros(4, dtype=torch.float64)
    w, c4 = torch.ones(64), g.cache_fp4(1, 1, 16, 64, device="cpu")
    slots = torch.zeros(2, dtype=torch.int64)
    for call in (lambda: g.qk_norm_rotary(pos, f, q, q, w, w), lambda: g.qk_norm_rotary_bwd(pos, f, q, q, q, q, w, w),
                 lambda: g.qk_norm_rotary_cache(pos, f, q, q, q, slots, None, None),
                 lambda: g.qk_norm_rotary_cache_fp4(pos, f, q, q, q, slots, c4, c4), lambda: g.cache_fp4_rows(slots, c4)):
        with pytest.raises(g.FlareError, match="GPU tensor"):
            call()


def test_cache_shapes():
    c = g.cache_fp4(3, 2, 16, 96, device="cpu")
    assert c[0].shape == (3, 2, 16, 48) and c[1].shape == (3, 2, 3, 16) and not c[0].any() and not c[1].any()
    assert layer._chk_cache_fp4(c, "k_cache", 2, 96, CPU) == (3, 16)
    for bad in ((c[0],), None, c[0], (c[1], c[0]), (c[0], c[1].transpose(2, 3)), (c[0].int(), c[1]), (None, c[1])):
        with pytest.raises(g.FlareError):
            layer._chk_cache_fp4(bad, "k_cache", 2, 96, CPU)
    for heads, d in ((1, 96), (2, 64), (2, 100)):
        with pytest.raises(g.FlareError):
            layer._chk_cache_fp4(c, "k_cache", heads, d, CPU)
    for other in (g.cache_fp4(4, 2, 16, 96, device="cpu"), g.cache_fp4(3, 2, 32, 96, device="cpu")):
        with pytest.raises(g.FlareError):
            layer._chk_caches_fp4(c, other, 2, 96, CPU)
    for d in (0, 16, 33):
        with pytest.raises(g.FlareError):
            g.cache_fp4(1, 1, 16, d, device="cpu")
    big = (torch.empty((0, 1, 2 ** 32 + 16, 16), dtype=torch.uint8), torch.empty((0, 1, 1, 2 ** 32 + 16), dtype=torch.uint8))
    with pytest.raises(g.FlareError, match="beyond 32 bits"):
        layer._chk_cache_fp4(big, "k_cache", 1, 32, CPU)


def attention4(L, R=2, block=4, qh=8, kh=2, d=128, page=64, io=g.BF16, causal=0, scale=0.0, q=FAKE, kc=FAKE, ks=FAKE, vc=FAKE,
               vs=FAKE, pages=100, bt=FAKE, wide=8, lens=FAKE, most=512, pt=FAKE, n=5000, o=FAKE, ws=FAKE & ~255, nbytes=1 << 40):
    s = g.AttentionShape(block, qh, kh, d, page, io, causal, scale)
    return L.flare_block_attention_fp4(R, ctypes.byref(s), q, kc, ks, vc, vs, pages, bt, wide, lens, most, pt, n, o, None, ws,
                                       nbytes, None)


def test_attention(L):
    for bad in (dict(R=-1), dict(block=0), dict(qh=0), dict(kh=0), dict(kh=3), dict(most=-1), dict(n=-1), dict(pages=-1),
                dict(most=513), dict(pages=0), dict(scale=math.inf), dict(scale=math.nan), dict(pages=2 ** 31)):
        assert attention4(L, **bad) == 2, bad
    for bad in (dict(d=16), dict(d=96), dict(page=8), dict(page=48), dict(io=g.F32), dict(causal=2), dict(R=2 ** 24),
                dict(n=2 ** 31 - 1), dict(page=2 ** 25)):
        assert attention4(L, **bad) == 4, bad
    for bad in ("q", "bt", "lens", "pt", "kc", "ks", "vc", "vs", "o"):
        assert attention4(L, **{bad: None}) == 1, bad
    assert attention4(L, q=FAKE + 8) == 3 and attention4(L, kc=FAKE + 8) == 3 and attention4(L, vs=FAKE + 2) == 3
    need = g.block_attention_fp4_workspace_bytes(2, 4, 8, 2, 128, 64, 512, 5000)
    assert need > 0 and attention4(L, nbytes=need - 1) == 5 and attention4(L, ws=None) == 5
    assert attention4(L, ws=(FAKE & ~255) + 64) == 5
    assert attention4(L, R=0, q=None, lens=None, bt=None, pt=None) == 0
    assert g.block_attention_fp4_workspace_bytes(2, 4, 8, 2, 128, 64, 64, 0) == 0
    assert g.block_attention_fp4_workspace_bytes(2, 4, 8, 2, 100, 64, 512, 100) == 0  # not instantiated
    with pytest.raises(g.FlareError, match="beyond 32 bits"):
        g.block_attention_fp4_workspace_bytes(2, 4, 8, 2, 128, 64, 512, 2 ** 32 + 5)
    # more workgroups than a launch holds
    assert attention4(L, R=2 ** 20, block=1, qh=8, kh=8, most=2 ** 30, wide=2 ** 10, page=2 ** 20, n=0, pt=None, nbytes=2 ** 62) == 4


@pytest.mark.parametrize("R,B,Hq,Hk,d,own,prefix", [(1, 1, 1, 1, 64, 1, 0), (256, 4, 16, 4, 128, 1024, 8192), (3, 7, 16, 2, 256, 777, 2500),
                                                    (1, 1, 16, 4, 128, 1 << 20, 0), (64, 1, 8, 8, 64, 0, 1 << 22), (5, 32, 8, 1, 128, 40, 40)])
def test_attention_workspace_is_rows_times_parts(L, R, B, Hq, Hk, d, own, prefix):
    """d + 2 floats a row and part, plus the alignment; parts of at most 4096 keys."""
    n = g.block_attention_fp4_workspace_bytes(R, B, Hq, Hk, d, 16, own, prefix)
    if n == 0:
        assert own + prefix <= 4096
        return
    parts, rest = divmod(n - 256, R * B * Hq * (d + 2) * 4)
    assert rest == 0 and parts >= -(-own // 4096) + -(-prefix // 4096) and parts >= 2


def test_attention_refuses_host_tensors():
    c4 = g.cache_fp4(1, 1, 16, 64, device="cpu")
    with pytest.raises(g.FlareError, match="GPU tensor"):
        g.block_attention_fp4(torch.zeros(2, 1, 1, 64, dtype=torch.bfloat16), c4, c4, None, None)
