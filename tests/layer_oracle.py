"""Plain 64-bit definitions of the operators around the GDN step, on the CPU,
that their GPU tests compare with (written from the formulas; no code shared
with the library)."""
import math

import numpy as np
import torch

LINEAR, SILU, SIGMOID = 0, 1, 2
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def act64(g, act):
    if act == LINEAR:
        return g
    p = 1.0 / (1.0 + torch.exp(-g))
    return p if act == SIGMOID else g * p


def rms64(x, w, eps):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w


def leaf(t):
    return None if t is None else t.detach().cpu().double().requires_grad_()


def gated_norm64(x, w, g, act, eps, dy=None):
    """y, or (y, dx, dgate, dweight) with dy."""
    x, w, g = leaf(x), leaf(w), leaf(g)
    y = rms64(x, w, eps)
    if g is not None:
        y = y * act64(g, act)
    if dy is None:
        return y.detach()
    y.backward(dy.detach().cpu().double())
    return y.detach(), x.grad, None if g is None else g.grad, w.grad


def residual_norm64(x, res, w_pre, w_post, g, scale, act, eps, dy=None, dh=None):
    """(h, y), or (h, y, dict of gradients) with dy."""
    x, res, w_pre, w_post, g, scale = map(leaf, (x, res, w_pre, w_post, g, scale))
    z = x if w_post is None else rms64(x, w_post, eps)
    if g is not None:
        z = z * act64(g, act)
    if scale is not None:
        z = z * scale
    h = res + z
    y = rms64(h, w_pre, eps)
    if dy is None:
        return h.detach(), y.detach()
    total = (y * dy.detach().cpu().double()).sum()
    if dh is not None:
        total = total + (h * dh.detach().cpu().double()).sum()
    total.backward()
    grad = lambda t: None if t is None else t.grad  # noqa: E731
    return h.detach(), y.detach(), {"dx": x.grad, "dresidual": res.grad, "dgate": grad(g), "dw_pre": w_pre.grad,
                                    "dw_post": grad(w_post), "dscale": grad(scale)}


def norm_reverse_size(x, du, eps):
    """The size of the terms of a norm's reverse, du >= 0 the size of its
    gradient: r (du + |u| mean(du |u|)), which r (du - u mean(du u)) may cancel
    in (a row of one channel cancels entirely), so that fp32 is off by steps of
    this and not of the result."""
    x = x.detach().double()
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    u = (x * r).abs()
    return r * (du + u * (du * u).mean(-1, keepdim=True))


def rotary64(x, positions, freqs, interleaved, mscale, sign=1.0):
    """The rotation as complex products, token by head."""
    y = x.detach().cpu().double().clone()
    f, p = freqs.cpu().double(), positions.cpu().double()
    n = f.numel()
    re = [2 * i if interleaved else i for i in range(n)]
    im = [2 * i + 1 if interleaved else n + i for i in range(n)]
    z = torch.complex(y[..., re], y[..., im]) * torch.exp(1j * sign * p[:, None] * f[None])[:, None] * mscale
    y[..., re], y[..., im] = z.real, z.imag
    return y


def step_tables_plain(seq_lens, new_lens, table, free, used, page, max_tokens, offset=0):
    """The tables, request by request."""
    table = np.array(table)
    R, width = table.shape
    cu, slots, pos, opened = [0], [], [], 0
    for r in range(R):
        held, new = int(seq_lens[r]), int(new_lens[r])
        for t in range(held, held + new):
            if t % page == 0:
                table[r, t // page] = free[used + opened]
                opened += 1
            slots.append(int(table[r, t // page]) * page + t % page)
            pos.append(t + offset)
        cu.append(cu[-1] + new)
    pad = max_tokens - len(slots)
    return {"cu_new": cu, "positions": pos + [0] * pad, "slots": slots + [-1] * pad,
            "seq_lens": [int(a) + int(b) for a, b in zip(seq_lens, new_lens)], "pages_used": [used + opened],
            "block_table": table.tolist()}


def attention64(q, k_cache, v_cache, block_table, seq_lens, prefix_table, prefix_len, causal, scale=None):
    """(o, lse, bound): the outputs in 64 bits and, for each, sum p |v| / sum p,
    what a relative error of the weights can move it by."""
    q, kc, vc = q.cpu().double(), k_cache.cpu().double(), v_cache.cpu().double()
    R, B, Hq, d = q.shape
    Hk, page = kc.shape[1], kc.shape[2]
    G = Hq // Hk
    scale = scale or 1.0 / math.sqrt(d)
    o, size = torch.zeros(R, B, Hq, d).double(), torch.zeros(R, B, Hq, d).double()
    lse = torch.full((R, B, Hq), -math.inf).double()
    bt, lens = block_table.cpu().tolist(), seq_lens.cpu().tolist()
    pt = [] if prefix_table is None else prefix_table.cpu().tolist()
    for r in range(R):
        n = max(0, lens[r])
        for b in range(B):
            own = max(0, n - (B - 1 - b)) if causal else n
            at = [(pt[j // page], j % page) for j in range(prefix_len)] + [(bt[r][j // page], j % page) for j in range(own)]
            if not at:
                continue
            pages, off = torch.tensor(at).T
            k, v = kc[pages, :, off], vc[pages, :, off]  # [n, Hk, d]
            for h in range(Hq):
                s = (k[:, h // G] @ q[r, b, h]) * scale
                p = torch.softmax(s, 0)
                o[r, b, h] = p @ v[:, h // G]
                size[r, b, h] = p @ v[:, h // G].abs()
                lse[r, b, h] = torch.logsumexp(s, 0)
    return o, lse, size


def close(got, want, io, slack=0.0, where=""):
    """|got - want| <= half a step of the value (its last rounding) + slack."""
    got = got.detach().cpu().double()
    want = want.double()
    tol = HALF_STEP[io] * want.abs() + slack
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g over its bound" % (
        where, int(bad.sum()), bad.numel(), float(((got - want).abs() - tol).max()))
