"""Plain 64-bit definitions of the softmax layers' q/k norms with rotary positions and of
caches in 4 bits, on the CPU, that their GPU tests compare with (written from the
formulas; no code shared with the library)."""
import math

import numpy as np
import torch

from layer_oracle import HALF_STEP, leaf, rms64, rotary64  # noqa: F401

STEP = 2.0 ** -24  # half a step of fp32


def rotary_leaf(x, positions, freqs, interleaved, mscale):
    """The rotation of a 64-bit tensor [T, H, d], differentiable."""
    f, p = freqs.detach().cpu().double(), positions.detach().cpu().double()
    n = f.numel()
    re = torch.arange(n) * 2 if interleaved else torch.arange(n)
    im = re + 1 if interleaved else re + n
    angle = p[:, None, None] * f
    c, s = torch.cos(angle) * mscale, torch.sin(angle) * mscale
    a, b = x[..., re], x[..., im]
    y = x.clone()
    y[..., re], y[..., im] = a * c - b * s, a * s + b * c
    return y


def norm_rotary64(x, w, positions, freqs, interleaved, mscale, eps):
    x = x if w is None else rms64(x, w, eps)
    return rotary_leaf(x, positions, freqs, interleaved, mscale)


def norm_rotary_size(x, w, freqs, interleaved, mscale, eps):
    """For each output the size of the terms it is formed of: |a| + |b| of its pair, scaled,
    where it is turned, else its own."""
    n = (x if w is None else rms64(x, w, eps)).abs()
    f = freqs.numel()
    re = torch.arange(f) * 2 if interleaved else torch.arange(f)
    im = re + 1 if interleaved else re + f
    y = n.clone()
    y[..., re] = y[..., im] = (n[..., re] + n[..., im]) * mscale
    return y


CODES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def fp4_group(x):
    """(codes, byte) of one group's 32 values in 64 bits, value by value."""
    top = max(abs(float(v)) for v in x) if all(math.isfinite(v) for v in x) else math.inf
    if not math.isfinite(top):
        return None, 255
    e = -1000 if top == 0 else math.frexp(top)[1] - 1 - 2
    if top > math.ldexp(7.0, e):
        e += 1
    e = min(max(e, -126), 125)
    codes = []
    for v in x:
        z = min(math.ldexp(abs(float(v)), -e), 8.0)
        off = np.abs(CODES - z)
        best = [c for c in range(8) if off[c] == off.min()]
        c = best[0] if len(best) == 1 else next(b for b in best if b % 2 == 0)
        codes.append(c + (8 if math.copysign(1.0, float(v)) < 0 else 0))
    return codes, e + 127


def fp4_values(x):
    """x [..., d] in 64 bits as the values that a cache in 4 bits holds."""
    g = x.detach().cpu().double().reshape(-1, 32)
    out = torch.empty_like(g)
    for i, row in enumerate(g.tolist()):
        codes, byte = fp4_group(row)
        if codes is None:
            out[i] = math.nan
        else:
            out[i] = torch.tensor([math.ldexp((-1.0 if c & 8 else 1.0) * float(CODES[c & 7]), byte - 127) for c in codes])
    return out.reshape(x.shape)


def fp4_nearest(x):
    """The same for many rows at once, in steps of the codes instead of by search."""
    g = x.detach().cpu().double().reshape(*x.shape[:-1], -1, 32)
    top = g.abs().amax(-1, keepdim=True)
    fine = torch.isfinite(top)
    e = torch.frexp(torch.where(fine & (top > 0), top, 2.0 ** -200))[1].double() - 3
    e = (e + (top > 7 * torch.exp2(e))).clamp(-126, 125)
    z = g * torch.exp2(-e)
    step = torch.where(z.abs() < 2, 0.5, torch.where(z.abs() < 4, 1.0, 2.0))
    v = (torch.round(z / step) * step).clamp(-6, 6) * torch.exp2(e)
    return torch.where(fine, v, math.nan).reshape(x.shape)


def cache_values(codes, scales):
    """The values of a cache in 4 bits, [pages, heads, page, d] in 64 bits."""
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
    d = 2 * codes.shape[-1]
    c = np.empty(codes.shape[:-1] + (d,), dtype=np.uint8)
    c[..., 0::2], c[..., 1::2] = codes & 15, codes >> 4
    v = CODES[c & 7] * np.where(c & 8, -1.0, 1.0)
    with np.errstate(invalid="ignore"):
        unit = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return torch.from_numpy(v * np.repeat(unit.swapaxes(2, 3), 32, axis=-1))


def same(got, want, where=""):
    """Equal values, NaN where NaN is wanted."""
    got, want = got.detach().cpu().double(), want.double()
    bad = ~((got == want) | (torch.isnan(got) & torch.isnan(want)))
    assert not bad.any(), "%s: %d of %d differ, the first at %s: %s for %s" % (
        where, int(bad.sum()), bad.numel(), torch.nonzero(bad)[0].tolist(), got[bad][0].item(), want[bad][0].item())
