"""The gate's activation far from zero, fp32.  With u = 2^-24, everything relative:
  exp 4 u, 1 + exp 1 u, reciprocal 2 u: sigmoid 7 u;
  SiLU one product more, 8 u;
  1 / rms of 256 channels: squares and 4 adds of a lane, 6 lane exchanges, mean and eps
  13 u, halved by the root, root and reciprocal 1 u each: 9 u;
  three products to y: 3 u.
20 u of y in all, 24 u allowed, whatever the gate; 2^-126 where a factor or result falls
below the smallest normal number.  The gradient adds one for du u w and the derivative:
sigmoid's p (1 - p) is off by 16 u p (1 - p is a difference from 1), SiLU's p (1 + g (1 - p))
by 18 u p (1 + |g|): 40 u of |dy u w| p (1 + |g|) bounds both with the rest."""
import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TINY = 2.0 ** -126


@pytest.fixture(scope="module")
def g():
    import gated_deltanet_dual_amd as g
    g.lib()
    return g


def inputs(top):
    import torch
    gen = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(64, 256, generator=gen).cuda() for _ in range(2))
    w = (1 + 0.1 * torch.randn(256, generator=gen)).cuda()
    gate = torch.linspace(-top, top, 64 * 256).reshape(256, 64).t().contiguous().cuda()
    return x, w, gate, dy


@pytest.mark.parametrize("act", ["SILU", "SIGMOID"])
def test_far_gates(g, act):
    import torch
    x, w, gate, dy = inputs(80.0)
    a = getattr(g, act)
    y, rstd = g.gated_norm(x, w, gate, activation=a, want_rstd=True)
    _, dgate, _ = g.gated_norm_bwd(x, w, gate, dy, rstd, activation=a)
    X, G = x.cpu().double(), gate.cpu().double()
    p = 1 / (1 + torch.exp(-G))
    n = X / torch.sqrt(X.square().mean(-1, keepdim=True) + 1e-6) * w.cpu().double()
    f, d = (G * p, p * (1 + G * (1 - p))) if act == "SILU" else (p, p * (1 - p))
    want = n * f
    off = (y.cpu().double() - want).abs() / (24 * U * want.abs() + TINY)
    assert float(off.max()) <= 1, "y: %.3g of its bound at gate %.3g" % (off.max(), G.flatten()[off.argmax()])
    t = dy.cpu().double() * n
    off = (dgate.cpu().double() - t * d).abs() / (40 * U * t.abs() * p * (1 + G.abs()) + TINY)
    assert float(off.max()) <= 1, "dgate: %.3g of its bound at gate %.3g" % (off.max(), G.flatten()[off.argmax()])


def test_gates_of_any_size(g):
    """Beyond exp's range, infinite, NaN: sigmoid 0, 1 and NaN."""
    import torch
    x, w, gate, _ = inputs(1.0)
    gate[:, :8] = torch.tensor([-200.0, 200.0, -1e30, 1e30, float("-inf"), float("inf"), float("nan"), 0.0]).cuda()
    y = g.gated_norm(x, w, gate, activation=g.SIGMOID)
    plain = g.gated_norm(x, w)
    assert (y[:, [0, 2, 4]] == 0).all() and torch.equal(y[:, [1, 3, 5]], plain[:, [1, 3, 5]])
    assert torch.isnan(y[:, 6]).all() and torch.equal(y[:, 7], plain[:, 7] / 2)
    assert torch.isfinite(y[:, 7:]).all()
    y = g.gated_norm(x, w, gate, activation=g.SILU)
    assert (y[:, [0, 2]] == 0).all() and torch.isnan(y[:, 6]).all() and torch.isfinite(y[:, 7:]).all()
