"""The weights' gradients of the norms where a training step forms them: many
workgroups that each pass several rows, whose partial sums a second launch adds.

Per column c the reference gives sum t and S = sum |t| of its terms in 64 bits (on
the GPU: up to 10^7 elements), and the kernels' result is off by at most
  (a + n 2^-24) S + 2^-24 |sum|
a  the error of a term, in its size: 4e-6 for the norm's own statistics, the gate
   (|g| <= 8) and the products, as derived in the norms' tests; three times that where the
   term holds the gradient of h, a difference of two such terms, whose size S then takes
   in place of its value;
n  the additions that a term passes: its thread's rows, the workgroup's teams, every 64th
   workgroup's partial row, 2 lane exchanges and 16 more.
A row left out, or one added to another column, moves a sum by about sqrt(rows) terms,
tens of times that bound and more."""
import pytest

pytestmark = pytest.mark.gpu
TERM = 4e-6
U = 2.0 ** -24

# rows, width, io, (passes of a workgroup's rows at most, teams of a workgroup, workgroups)
SHAPES = [
    (80000, 128, "bf16", (4, 16, 1536)),     # 16 lanes a row
    (90001, 72, "bf16", (4, 16, 1536)),      # a width that is no power of two, rows that do not fill the last pass
    (20001, 512, "bf16", (4, 4, 1536)),      # a wave a row
    (15000, 500, "f32", (3, 4, 1536)),       # a wave of two vectors a lane
    (4001, 1000, "bf16", (3, 1, 1536)),      # workgroups of 128 threads
    (2500, 2048, "bf16", (4, 1, 768)),       # of 256
    (1700, 2048, "f32", (4, 1, 512)),        # of 256, two vectors a thread
    (1300, 4095, "bf16", (3, 1, 512)),
    (700, 8192, "bf16", (3, 1, 256)),        # of 512
    (700, 4096, "f32", (3, 1, 256)),
    (600, 16384, "bf16", (3, 1, 256)),       # of 1024
    (600, 6000, "f32", (3, 1, 256)),         # of 1024, two vectors a thread
    (600, 16383, "f32", (3, 1, 256)),        # and four
]


@pytest.fixture(scope="module")
def g():
    import gated_deltanet_dual_amd as g
    g.lib()
    return g


def rnd(seed, *shape, io="bf16", scale=1.0):
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t = (torch.randn(shape, generator=gen, device="cuda") * scale).clamp(-8, 8)
    return t.to(torch.bfloat16 if io == "bf16" else torch.float32)


def check(got, terms, sizes, a, adds, where):
    want, S = terms.sum(0), sizes.sum(0)
    off = (got.double() - want).abs()
    tol = (a + adds * U) * S + U * want.abs()
    assert not (off > tol).any(), "%s: worst %.3g of its bound" % (where, float((off / tol).max()))


def additions(plan):
    passes, teams, blocks = plan
    return passes + teams + -(-blocks // 64) + 2 + 16


@pytest.mark.parametrize("rows,d,io,plan", SHAPES)
def test_gated_norm_weight(g, rows, d, io, plan):
    import torch
    H = 4 if rows % 4 == 0 else 1
    x, w, gate, dy = (rnd(i, rows // H, H, d, io=io, scale=s) for i, s in ((1, 1.0), (2, 0.1), (3, 2.0), (4, 1.0)))
    w = 1 + w.flatten(0, 1)[0].float()
    _, rstd = g.gated_norm(x, w, gate, activation=g.SILU, want_rstd=True)
    dx, dgate, dw = g.gated_norm_bwd(x, w, gate, dy, rstd, activation=g.SILU)
    X, G, D = (t.double().flatten(0, 1) for t in (x, gate, dy))
    t = D * X / torch.sqrt(X.square().mean(-1, keepdim=True) + 1e-6) * (G * torch.sigmoid(G))
    check(dw, t, t.abs(), TERM, additions(plan), "dweight")


@pytest.mark.parametrize("rows,C,io,plan", SHAPES)
def test_residual_norm_weights(g, rows, C, io, plan):
    import torch
    x, gate, dy = rnd(1, rows, C, io=io), rnd(2, rows, C, io=io, scale=2.0), rnd(3, rows, C, io=io)
    res, dh = rnd(4, rows, C, io="f32", scale=2.0), rnd(5, rows, C, io="f32")
    w2, w1, sc = (o + 0.1 * rnd(6 + i, C, io="f32") for i, o in enumerate((1.0, 1.0, 0.5)))
    more = dict(w_post=w1, gate=gate, scale=sc, activation=g.SIGMOID)
    _, _, rstd = g.residual_norm(x, res, w2, want_rstd=True, **more)
    got = g.residual_norm_bwd(x, res, w2, dy, dh, rstd, **more)
    X, G, D = x.double(), gate.double(), dy.double()
    n = X / torch.sqrt(X.square().mean(-1, keepdim=True) + 1e-6)
    del X
    f = torch.sigmoid(G)
    z = n * w1 * f * sc
    h = res.double() + z
    r2 = 1 / torch.sqrt(h.square().mean(-1, keepdim=True) + 1e-6)
    u, size_u = h * r2, (res.double().abs() + z.abs()) * r2  # h's terms can cancel
    del h, z, G
    check(got["dw_pre"], D * u, D.abs() * size_u, TERM, additions(plan), "dw_pre")
    du = D * w2
    d = dh.double() + r2 * (du - u * (du * u).mean(-1, keepdim=True))
    size = dh.double().abs() + r2 * (du.abs() + size_u * (du.abs() * size_u).mean(-1, keepdim=True))
    del u, size_u, du, D
    for name, by in (("dw_post", f * sc * n), ("dscale", f * w1 * n)):
        check(got[name], d * by, size * by.abs(), 3 * TERM, additions(plan), name)
