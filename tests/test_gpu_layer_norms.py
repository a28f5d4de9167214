"""The norms before and after a block (gate, residual scale), forward and
reverse mode, against their definitions in 64 bits.

Tolerances.  Inputs are of size <= 8, weights about 1, so outputs and input
gradients are of size <= ~64.  An output's last rounding is half a step of its
type.  Before it everything is fp32: a row sum of squares is a tree of at most
16 sequential adds and 10 exchanges (relative error <= 26 * 2^-24 < 2e-6), 1 /
sqrt and the products add a few 2^-24, exp and reciprocal of the gate (|g| <= 8)
at most 16 * 2^-24: 4e-6 of the terms' size covers them.  A term's size is bounded
here by the largest magnitudes of the test's own reference; of an input gradient,
whose terms cancel (fully in a row of one channel), by the terms' own sizes
(norm_reverse_size), twice for the two roundings of each term and their difference.  A weight gradient adds
T * H terms in a fixed tree of chains of at most T * H / 512 + 48 adds."""
import pytest

from layer_oracle import LINEAR, SIGMOID, SILU, act64, close, gated_norm64, norm_reverse_size, residual_norm64

pytestmark = pytest.mark.gpu
FP32 = 4e-6


@pytest.fixture(scope="module")
def g():
    import gated_deltanet_dual_amd as g
    g.lib()
    return g


def rnd(seed, *shape, io="bf16", scale=1.0):
    import torch
    gen = torch.Generator().manual_seed(seed)
    t = (torch.randn(shape, generator=gen) * scale).clamp(-8, 8)
    return t.to(torch.bfloat16 if io == "bf16" else torch.float32).cuda()


def top(t):
    return float(t.abs().max()) if t.numel() else 0.0


# a head row in one vector, a wave, several vectors a lane, a workgroup; widths
# that are no multiple of 16 bytes; one channel; one token and many
SHAPES = [(1, 1, 1), (3, 2, 16), (5, 3, 20), (33, 16, 128), (7, 5, 72), (4, 1, 2048), (2, 1, 4100), (3, 1, 16384),
          (1, 3, 257), (2, 2, 1003), (1100, 1, 64), (0, 4, 128)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,d", SHAPES)
def test_gated_norm(g, T, H, d, io):
    import torch
    for i, act in enumerate([None, LINEAR, SILU, SIGMOID]):
        x, w = rnd(1, T, H, d, io=io), 1 + 0.1 * rnd(2, d, io="f32")
        gate = None if act is None else rnd(3, T, H, d, io=io, scale=2.0)
        dy = rnd(4, T, H, d, io=io)
        a = 0 if act is None else act
        y, rstd = g.gated_norm(x, w, gate, activation=a, want_rstd=True)
        dx, dg, dw = g.gated_norm_bwd(x, w, gate, dy, rstd, activation=a)
        torch.cuda.synchronize()
        ry, rdx, rdg, rdw = gated_norm64(x, w, gate, a, 1e-6, dy)
        where = "act %s" % act
        close(y, ry, x.dtype, FP32 * top(ry), where + " y")
        cpu = lambda t: t.detach().cpu().double()  # noqa: E731
        f = 1.0 if gate is None else act64(cpu(gate), a).abs()
        size = norm_reverse_size(cpu(x), (cpu(dy) * cpu(w)).abs() * f, 1e-6)
        close(dx, rdx, x.dtype, 2 * FP32 * top(size), where + " dx")
        if gate is not None:
            close(dg, rdg, x.dtype, FP32 * top(rdg), where + " dgate")
        # chains of adds: 2^-24 each of the running sum, itself at most the sum of magnitudes
        terms = T * H * 40.0
        close(dw, rdw, torch.float32, 2.0 ** -24 * (T * H / 512 + 48) * terms ** 0.5 * 8 + FP32 * 40, where + " dweight")


@pytest.mark.parametrize("io,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("T,C", [(1, 2048), (1, 1), (3, 20), (40, 256), (5, 1003), (2, 8192), (2, 16384), (600, 72), (0, 64)])
def test_residual_norm(g, T, C, io, res):
    import torch
    for act, post, scale, with_dh in [(None, False, False, True), (SILU, True, True, True), (SIGMOID, True, False, False),
                                      (LINEAR, False, True, True)]:
        x, r = rnd(1, T, C, io=io), rnd(2, T, C, io=res, scale=2.0)
        w2, w1 = 1 + 0.1 * rnd(3, C, io="f32"), 1 + 0.1 * rnd(4, C, io="f32") if post else None
        sc = 0.5 + 0.1 * rnd(5, C, io="f32") if scale else None
        gate = None if act is None else rnd(6, T, C, io=io, scale=2.0)
        dy, dh = rnd(7, T, C, io=io), rnd(8, T, C, io=res) if with_dh else None
        a = 0 if act is None else act
        more = dict(w_post=w1, gate=gate, scale=sc, activation=a)
        h, y, rstd = g.residual_norm(x, r, w2, want_rstd=True, **more)
        got = g.residual_norm_bwd(x, r, w2, dy, dh, rstd, **more)
        torch.cuda.synchronize()
        rh, ry, want = residual_norm64(x, r, w2, w1, gate, sc, a, 1e-6, dy, dh)
        where = "act %s post %s scale %s " % (act, post, scale)
        close(h, rh, r.dtype, FP32 * top(rh), where + "h")
        close(y, ry, x.dtype, FP32 * 2 * top(ry), where + "y")
        # the sizes of the terms that each gradient is a difference of
        cpu = lambda t: t.detach().cpu().double()  # noqa: E731
        size_h = norm_reverse_size(rh, (cpu(dy) * cpu(w2)).abs(), 1e-6) + (cpu(dh).abs() if with_dh else 0.0)
        f = 1.0 if gate is None else act64(cpu(gate), a).abs()
        f = f * (1.0 if sc is None else cpu(sc).abs())
        size_x = norm_reverse_size(cpu(x), size_h * f * cpu(w1).abs(), 1e-6) if post else size_h * f
        z = (cpu(x) / (cpu(x).pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()).abs() * 1.5 if post else cpu(x).abs()
        size_g = size_h * z * (1.0 if sc is None else cpu(sc).abs()) * 1.1  # |act'| < 1.1
        for name, io_t, size in (("dx", x.dtype, size_x), ("dresidual", r.dtype, size_h), ("dgate", x.dtype, size_g)):
            if want[name] is not None:
                close(got[name], want[name], io_t, 3 * FP32 * top(size), where + name)
        for name in ("dw_pre", "dw_post", "dscale"):
            if want[name] is None:
                assert got[name] is None
            else:
                close(got[name], want[name], torch.float32, 2.0 ** -24 * (T / 512 + 48) * (T * 40.0) ** 0.5 * 8 + FP32 * 60,
                      where + name)


def test_slices_and_unaligned_rows(g):
    """x, gate and dy as slices of wider rows, at offsets that break 16-byte
    alignment: the same results as packed copies of them."""
    import torch
    for off in (0, 1, 8):
        wide = rnd(1, 19, 3 * 4 * 64 + 40)
        x = wide[:, off:off + 256].unflatten(1, (4, 64))
        gate = wide[:, 256 + off:512 + off].unflatten(1, (4, 64))
        dy = wide[:, 512 + off:768 + off].unflatten(1, (4, 64))
        w = 1 + 0.1 * rnd(2, 64, io="f32")
        y, rstd = g.gated_norm(x, w, gate, want_rstd=True)
        yp, rp = g.gated_norm(x.contiguous(), w, gate.contiguous(), want_rstd=True)
        got = g.gated_norm_bwd(x, w, gate, dy, rstd)
        want = g.gated_norm_bwd(x.contiguous(), w, gate.contiguous(), dy.contiguous(), rp)
        ry = gated_norm64(x, w, gate, SILU, 1e-6)
        close(y, ry, x.dtype, FP32 * top(ry), "sliced y")
        for a, b in zip((y, *got), (yp, *want)):
            # another split of the row sums: fp32 differences, then one rounding
            assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -7, atol=1e-5)


def test_zero_rows_and_non_finite(g):
    """A row of zeros (the prompt rows of a noisy stream) gives zeros and finite
    gradients; a row with an infinity or a NaN does not reach other rows."""
    import torch
    x, w, gate = rnd(1, 6, 2, 128), 1 + 0.1 * rnd(2, 128, io="f32"), rnd(3, 6, 2, 128)
    x[1] = 0
    x[3, 0, 5], x[4, 1, 7] = float("inf"), float("nan")
    clean = x.clone()
    clean[3, 0], clean[4, 1] = 0, 0
    y, rstd = g.gated_norm(x, w, gate, want_rstd=True)
    dx, _, _ = g.gated_norm_bwd(x, w, gate, gate, rstd)
    yc, rc = g.gated_norm(clean, w, gate, want_rstd=True)
    dxc, _, _ = g.gated_norm_bwd(clean, w, gate, gate, rc)
    assert (y[1] == 0).all() and torch.isfinite(dx[1]).all()
    keep = torch.ones(6, 2, dtype=torch.bool)
    keep[3, 0] = keep[4, 1] = False
    assert torch.equal(y[keep.cuda()], yc[keep.cuda()]) and torch.equal(dx[keep.cuda()], dxc[keep.cuda()])
    assert torch.isnan(y[4, 1]).any()


def test_reverse_modes_repeat_bit_for_bit(g):
    import torch
    x, w, gate, dy = rnd(1, 2900, 4, 128), rnd(2, 128, io="f32"), rnd(3, 2900, 4, 128), rnd(4, 2900, 4, 128)
    _, rstd = g.gated_norm(x, w, gate, want_rstd=True)
    a, b = (g.gated_norm_bwd(x, w, gate, dy, rstd) for _ in range(2))
    assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_differences(g):
    """The gradients against central differences of the forward in fp32, along
    random directions: step 2^-6, error of a difference <= (fp32 forward error 2e-5 *
    sqrt(n)) / step + third derivative * step^2."""
    import torch
    T, C = 3, 64
    x, r = rnd(1, T, C, io="f32"), rnd(2, T, C, io="f32")
    w2, w1, sc, gate = 1 + 0.1 * rnd(3, C, io="f32"), 1 + 0.1 * rnd(4, C, io="f32"), 0.5 + 0.1 * rnd(5, C, io="f32"), rnd(6, T, C, io="f32")
    dy, dh = rnd(7, T, C, io="f32"), rnd(8, T, C, io="f32")

    def loss(x, r, gate, w2, w1, sc):
        h, y = g.residual_norm(x, r, w2, w_post=w1, gate=gate, scale=sc, activation=SILU)
        return float((h.double() * dh.double()).sum() + (y.double() * dy.double()).sum())

    args = [x, r, gate, w2, w1, sc]
    _, _, rstd = g.residual_norm(x, r, w2, w_post=w1, gate=gate, scale=sc, activation=SILU, want_rstd=True)
    grads = g.residual_norm_bwd(x, r, w2, dy, dh, rstd, w_post=w1, gate=gate, scale=sc, activation=SILU)
    for i, name in enumerate(["dx", "dresidual", "dgate", "dw_pre", "dw_post", "dscale"]):
        v = rnd(20 + i, *args[i].shape, io="f32")
        v = v / v.norm()
        e = 2.0 ** -6
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + e * v, args[i] - e * v
        diff = (loss(*up) - loss(*down)) / (2 * e)
        got = float((grads[name].double() * v.double()).sum())
        assert abs(diff - got) <= 2e-2 * max(1.0, abs(got)), (name, diff, got)
