"""The operators around the GDN step run together, as a hybrid model's serving
loop and training step run them: tables -> rotary and cache -> attention ->
gated norm -> residual norm for a softmax layer, block step -> gated norm ->
residual norm for a GDN layer; captured and replayed; on another stream; and
their differentiable forms.  Every stage is compared with its 64-bit definition
on the stage's own inputs, with the bounds of its own tests."""
import math

import numpy as np
import pytest

from gated_deltanet_dual_amd import workloads as wl
from gpu_util import to_dev
from layer_oracle import (SIGMOID, SILU, attention64, close, gated_norm64, residual_norm64, rotary64, step_tables_plain)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import gated_deltanet_dual_amd as g
    g.lib()
    return g


def rnd(seed, *shape, io="bf16", scale=1.0):
    import torch
    t = torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale
    return t.to(torch.bfloat16 if io == "bf16" else torch.float32).cuda()


class SoftmaxLayer:
    """One softmax layer's serving state and its step of B tokens a request."""

    def __init__(self, g, R=5, B=4, Hq=4, Hk=2, d=64, page=16, prefix=40, width=6):
        import torch
        self.g, self.R, self.B, self.Hq, self.Hk, self.d, self.page, self.prefix = g, R, B, Hq, Hk, d, page, prefix
        shared = -(-prefix // page)
        pages = R * width + shared
        ids = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
        self.prefix_table, self.free = ids[:shared].contiguous(), ids[shared:].contiguous()
        self.kc, self.vc = rnd(2, pages, Hk, page, d), rnd(3, pages, Hk, page, d)
        self.table = torch.zeros(R, width, dtype=torch.int32).cuda()
        self.lens = torch.zeros(R, dtype=torch.int32).cuda()
        self.used = torch.zeros(1, dtype=torch.int32).cuda()
        self.new = torch.full((R,), B, dtype=torch.int32).cuda()
        self.freqs, self.mscale = g.rotary_frequencies(d // 2, scaling="yarn", factor=2.0, original_length=64)
        self.w_norm, self.w_pre, self.w_post = 1 + 0.1 * rnd(4, d, io="f32"), 1 + 0.1 * rnd(5, Hq * d, io="f32"), 1 + 0.1 * rnd(6, Hq * d, io="f32")
        self.scale = 0.5 + 0.1 * rnd(7, Hq * d, io="f32")

    def step(self, qkv, gate, residual, causal):
        """qkv [R * B, (Hq + 2 Hk) * d]; returns every stage's outputs."""
        g, R, B, Hq, Hk, d = self.g, self.R, self.B, self.Hq, self.Hk, self.d
        t = g.step_tables(self.lens, self.new, self.table, self.free, self.used, self.page, R * B, position_offset=self.prefix)
        q, k, v = (qkv[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)))
        qr = g.rotary_cache(t["positions"], self.freqs, q, k, v, t["slots"], self.kc, self.vc, mscale=self.mscale)
        o = g.block_attention(qr.view(R, B, Hq, d), self.kc, self.vc, self.table, t["seq_lens"], prefix_table=self.prefix_table,
                              prefix_len=self.prefix, causal=causal)
        y = g.gated_norm(o.view(R * B, Hq, d), self.w_norm, gate, activation=SIGMOID)
        h, z = g.residual_norm(y.view(R * B, Hq * d), residual, self.w_pre, w_post=self.w_post, scale=self.scale)
        return t, qr, o, y, h, z

    def inputs(self, seed):
        n = self.R * self.B
        return (rnd(seed, n, (self.Hq + 2 * self.Hk) * self.d), rnd(seed + 1, n, self.Hq, self.d),
                rnd(seed + 2, n, self.Hq * self.d, io="f32"))

    def check(self, before, inputs, out, causal):
        """The stages of a step against their definitions; before: lens, table, used."""
        import torch
        t, qr, o, y, h, z = out
        lens, table, used = before
        R, B, Hq, Hk, d = self.R, self.B, self.Hq, self.Hk, self.d
        want = step_tables_plain(lens, [B] * R, table, self.free.cpu().tolist(), used, self.page, R * B, self.prefix)
        for name in ("cu_new", "positions", "slots", "seq_lens", "pages_used"):
            assert t[name].cpu().tolist() == want[name], name
        assert self.table.cpu().tolist() == want["block_table"] and int(t["status"]) == 0
        qkv, gate, residual = inputs
        q, k, v = (qkv[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)))
        tol = 1.2e-6 * float(qkv.abs().max()) * self.mscale
        close(qr, rotary64(q, t["positions"], self.freqs, False, self.mscale), q.dtype, tol, "q")
        slots = t["slots"]
        close(self.kc[slots // self.page, :, slots % self.page], rotary64(k, t["positions"], self.freqs, False, self.mscale),
              k.dtype, tol, "k in the cache")
        assert torch.equal(self.vc[slots // self.page, :, slots % self.page], v)
        ro, _, size = attention64(qr.view(R, B, Hq, d), self.kc, self.vc, self.table, t["seq_lens"], self.prefix_table,
                                  self.prefix, causal)
        close(o, ro, o.dtype, (2.0 ** -8 + 4e-4) * size, "attention")
        ry = gated_norm64(o.view(R * B, Hq, d), self.w_norm, gate, SIGMOID, 1e-6)
        close(y, ry, y.dtype, 4e-6 * float(ry.abs().max()), "gated norm")
        rh, rz = residual_norm64(y.view(R * B, Hq * d), residual, self.w_pre, self.w_post, None, self.scale, 0, 1e-6)
        close(h, rh, h.dtype, 4e-6 * float(rh.abs().max()), "h")
        close(z, rz, z.dtype, 8e-6 * float(rz.abs().max()), "y")


def test_softmax_layer_serving(g):
    """Three blocks a request: two denoising reads that see the block whole, then
    the causal replay that keeps it."""
    import torch
    layer = SoftmaxLayer(g)
    for block in range(3):
        before = layer.lens.cpu().tolist(), layer.table.cpu().tolist(), int(layer.used)
        for pas in range(3):
            causal = pas == 2
            inputs = layer.inputs(100 * block + 10 * pas)
            out = layer.step(*inputs, causal)
            torch.cuda.synchronize()
            # the denoising reads open the same pages again: lens and used stand still
            layer.check(before, inputs, out, causal)
        layer.lens, layer.used = out[0]["seq_lens"], out[0]["pages_used"]
    assert layer.lens.cpu().tolist() == [12] * layer.R


def test_serving_step_captured_and_replayed(g):
    """The step in a graph: every replay, on new inputs and lengths and with eager
    work between, gives the eager step's bits."""
    import torch
    layer = SoftmaxLayer(g)
    static = [t.clone() for t in layer.inputs(1)]
    kc0, vc0, lens0, table0, used0 = (t.clone() for t in (layer.kc, layer.vc, layer.lens, layer.table, layer.used))

    def reset(lens):
        layer.kc.copy_(kc0), layer.vc.copy_(vc0), layer.table.copy_(table0), layer.used.copy_(used0 + int(lens > 0) * layer.R)
        layer.lens.fill_(lens)
        if lens:
            layer.table[:, 0] = layer.free[:layer.R]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step(*static, True)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = layer.step(*static, True)
    for rep, lens in enumerate((0, 7, 3, 0)):
        new = layer.inputs(50 + 7 * rep)
        for a, b in zip(static, new):
            a.copy_(b)
        reset(lens)
        eager = [t.clone() for t in (*layer.step(*static, True)[1:], layer.kc, layer.table)]
        reset(lens)
        junk = torch.randn(1 << 18, device="cuda").sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert float(junk) == float(junk)
        for a, b in zip(eager, (*captured[1:], layer.kc, layer.table)):
            assert torch.equal(a, b), rep


def test_two_graphs_and_another_stream(g):
    """Two captured reverse modes replayed on two streams at once, each with the
    workspace its capture made, and an eager call on a third stream."""
    import torch
    x, w, gate, dy = rnd(1, 600, 4, 128), 1 + 0.1 * rnd(2, 128, io="f32"), rnd(3, 600, 4, 128), rnd(4, 600, 4, 128)
    x2 = rnd(5, 600, 4, 128)
    want = [g.gated_norm_bwd(a, w, gate, dy, g.gated_norm(a, w, gate, want_rstd=True)[1]) for a in (x, x2)]
    graphs, outs = [], []
    for a in (x, x2):
        _, rstd = g.gated_norm(a, w, gate, want_rstd=True)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(g.gated_norm_bwd(a, w, gate, dy, rstd))
        graphs.append((graph, rstd))
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(4):
        for (graph, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        with torch.cuda.stream(streams[2]):
            third = g.gated_norm_bwd(x2, w, gate, dy, graphs[1][1])
        torch.cuda.synchronize()
        for got, exp in zip((*outs, third), (*want, want[1])):
            assert all(torch.equal(a, b) for a, b in zip(got, exp))


def test_gdn_layer_serving(g):
    """The GDN block step's output through its gated norm and the next norm."""
    import torch
    s = wl.serving(seed=11, n_req=6, H=4, d=128, n_slots=8, n_evals=1)
    pool, slot = to_dev(s.pool, torch.device("cuda:0")), to_dev(s.slot_idx, torch.device("cuda:0"))
    q, k, v, a, b = s.evals[0]
    dev = torch.device("cuda:0")
    o = g.block_step(slot, pool, to_dev(q, dev, True), to_dev(k, dev, True), to_dev(v, dev, True), to_dev(a, dev), to_dev(b, dev), g.EVAL)
    rows = o.flatten(0, 1)  # [R * B, H, d]
    w, gate = 1 + 0.1 * rnd(1, 128, io="f32"), rnd(2, *rows.shape)
    y = g.gated_norm(rows, w, gate)
    res, w_pre = rnd(3, rows.shape[0], 512), 1 + 0.1 * rnd(4, 512, io="f32")
    h, z = g.residual_norm(y.flatten(1), res, w_pre)
    ry = gated_norm64(rows, w, gate, SILU, 1e-6)
    close(y, ry, y.dtype, 4e-6 * float(ry.abs().max()), "y")
    rh, rz = residual_norm64(y.flatten(1), res, w_pre, None, None, None, 0, 1e-6)
    close(h, rh, h.dtype, 4e-6 * float(rh.abs().max()), "h")
    close(z, rz, z.dtype, 8e-6 * float(rz.abs().max()), "z")


def test_differentiable_forms(g):
    """A training layer's tail and head through autograd: shared weights, a
    broadcast gate and a broadcast output gradient, against the same graph in 64
    bits.  fp32 throughout: three stages of relative error 4e-6 of the terms' size,
    sums over 48 x 4 terms of size <= 64."""
    import torch
    from gated_deltanet_dual_amd import autograd as ag
    T, H, d = 48, 4, 32
    leaf = lambda seed, *shape, io="f32": rnd(seed, *shape, io=io).requires_grad_()  # noqa: E731
    x, gate1, w, res = leaf(1, T, H, d), leaf(2, 1, H, d), leaf(3, d), leaf(4, T, H * d)
    w_pre, w_post, scale, g2 = leaf(5, H * d), leaf(6, H * d), leaf(7, H * d), leaf(8, T, H * d)
    pos, (freqs, m) = torch.arange(T, dtype=torch.int32).cuda() * 1000, g.rotary_frequencies(16, scaling="yarn", factor=4.0, original_length=100)
    leaves = [x, gate1, w, res, w_pre, w_post, scale, g2]

    def run(x, gate1, w, res, w_pre, w_post, scale, g2, ops):
        y = ops["gated"](x, w, gate1.expand(T, H, d))
        y = ops["gated"](y, w, None)  # the weight shared by two norms, and no gate
        h, z = ops["residual"](y.flatten(1), res, w_pre, w_post, g2, scale)
        q, k = ops["rotary"](z.unflatten(1, (H, d)), h.unflatten(1, (H, d))[:, :2])
        return q.sum() + (k * k).sum() + h.sum()

    def rot64(t):
        f, p, n = freqs, pos.double(), freqs.numel()
        c, s = torch.cos(p[:, None] * f)[:, None] * m, torch.sin(p[:, None] * f)[:, None] * m
        a, b = t[..., :n], t[..., n:2 * n]
        return torch.cat([a * c - b * s, a * s + b * c, t[..., 2 * n:]], -1)

    def gated64(x, w, gate):
        y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        return y if gate is None else y * gate * torch.sigmoid(gate)

    def residual64(x, res, w2, w1, gate, sc):
        h = res + sc * torch.sigmoid(gate) * (x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w1)
        return h, h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * w2

    own = dict(gated=ag.gated_norm, residual=lambda *a: ag.residual_norm(a[0], a[1], a[2], w_post=a[3], gate=a[4], scale=a[5]),
               rotary=lambda q, k: ag.rotary(pos, freqs, q, k, mscale=m))
    ref = dict(gated=gated64, residual=residual64, rotary=lambda q, k: (rot64(q), rot64(k)))
    loss = run(*leaves, own)
    loss.backward()
    copies = [t.detach().double().requires_grad_() for t in leaves]
    want = run(*copies, ref)
    want.backward()
    assert abs(float(loss.detach()) - float(want.detach())) <= 1e-4 * abs(float(want.detach())) + 1e-2
    for t, c in zip(leaves, copies):
        size = float(c.grad.abs().max())
        assert float((t.grad.double() - c.grad).abs().max()) <= 2e-4 * max(size, 1.0), t.shape


def test_rotary_gradient_differences(g):
    """Rotary's gradient along a direction against central differences (the
    rotation is linear: differences have no step error, only fp32's)."""
    import torch
    freqs, m = g.rotary_frequencies(32, factor=2.0, scaling="linear")
    pos = torch.arange(9, dtype=torch.int32).cuda() * 37
    q, v, dq = rnd(1, 9, 2, 64, io="f32"), rnd(2, 9, 2, 64, io="f32"), rnd(3, 9, 2, 64, io="f32")
    up, _ = g.rotary(pos, freqs, q + v, interleaved=True)
    down, _ = g.rotary(pos, freqs, q - v, interleaved=True)
    grad, _ = g.rotary(pos, freqs, dq, interleaved=True, inverse=True)
    a, b = float(((up - down).double() / 2 * dq.double()).sum()), float((grad.double() * v.double()).sum())
    # 1152 terms of size <= 16, each off by a few 2^-24 of it
    assert abs(a - b) <= 1152 * 16 * 8 * 2.0 ** -24


def test_calls_allocate_only_what_they_return(g):
    """With every buffer given, a call allocates nothing."""
    import torch
    x, w, gate, dy = rnd(1, 600, 4, 128), rnd(2, 128, io="f32"), rnd(3, 600, 4, 128), rnd(4, 600, 4, 128)
    y, rstd = g.gated_norm(x, w, gate, want_rstd=True)
    out = g.gated_norm_bwd(x, w, gate, dy, rstd)
    ws = torch.empty(g.gated_norm_bwd_workspace_bytes(600, 4, 128), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    g.gated_norm(x, w, gate, out=y, rstd=rstd)
    g.gated_norm_bwd(x, w, gate, dy, rstd, workspace=ws, out=out)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before


def test_binding_mistakes_on_the_gpu(g):
    import torch
    x, w = rnd(1, 6, 2, 64), rnd(2, 64, io="f32")
    with pytest.raises(g.FlareError, match="weight: dtype"):
        g.gated_norm(x, w.bfloat16())
    with pytest.raises(g.FlareError, match="gate: shape"):
        g.gated_norm(x, w, x[:5])
    with pytest.raises(g.FlareError, match="contiguous"):
        g.gated_norm(x.transpose(1, 2), rnd(2, 2, io="f32"))
    with pytest.raises(g.FlareError, match="out: shape"):
        g.gated_norm(x, w, out=x[:, :1].contiguous())
    with pytest.raises(g.FlareError, match="workspace holds"):
        g.gated_norm_bwd(x, w, None, x, torch.ones(6, 2, device="cuda"), workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(g.FlareError, match="positions: dtype"):
        g.rotary(torch.arange(6).cuda(), torch.zeros(4, dtype=torch.float64).cuda(), x)
    with pytest.raises(g.FlareError, match="freqs: dtype"):
        g.rotary(torch.arange(6, dtype=torch.int32).cuda(), torch.zeros(4).cuda(), x)
    cache = rnd(3, 4, 2, 16, 64)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    q = rnd(4, 1, 2, 4, 64)
    with pytest.raises(g.FlareError, match="prefix_table"):
        g.block_attention(q, cache, cache, i32(0).view(1, 1), i32(3), prefix_table=i32(1), prefix_len=17)
    with pytest.raises(g.FlareError, match="beyond the table"):
        g.block_attention(q, cache, cache, i32(0).view(1, 1), i32(3), max_seq_len=17)
    with pytest.raises(g.FlareError, match="bfloat16"):
        g.block_attention(q.float(), cache, cache, i32(0).view(1, 1), i32(3))
    with pytest.raises(g.FlareError, match="v_cache: shape"):
        g.block_attention(q, cache, cache[:3], i32(0).view(1, 1), i32(3))
    lens = i32(3)
    with pytest.raises(g.FlareError, match="memory of its input"):
        g.step_tables(lens, i32(1), i32(0, 0).view(1, 2), i32(5), i32(0), 16, 4, out={"seq_lens": lens})
    torch.cuda.synchronize()


def test_gradients_of_one_output_alone(g):
    """residual_norm's h or y unused: the other's gradients are those with zeros in
    its place; gradients of the gradients are refused."""
    import torch
    from gated_deltanet_dual_amd import autograd as ag
    T, C = 7, 96
    x, res, w = (rnd(i, *s, io=io).requires_grad_() for i, s, io in ((1, (T, C), "bf16"), (2, (T, C), "f32"), (3, (C,), "f32")))
    h, y = ag.residual_norm(x, res, w)
    dh, dy = rnd(4, T, C, io="f32"), rnd(5, T, C)
    zh, zy = torch.zeros_like(dh), torch.zeros_like(dy)
    for outs, grads, full in (((h,), (dh,), (dh, zy)), ((y,), (dy,), (zh, dy))):
        some = torch.autograd.grad(outs, (x, res, w), grads, retain_graph=True)
        both = torch.autograd.grad((h, y), (x, res, w), full, retain_graph=True)
        for a, b in zip(some, both):
            assert torch.equal(a, b)
    dx, = torch.autograd.grad(y, x, dy.clone().requires_grad_(), create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable|differentiat"):
        dx.float().sum().backward()
