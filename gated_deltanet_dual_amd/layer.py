"""Binding of the operators around the GDN step: the norms before and after a
block with its gate and residual scale, rotary positions, the tables of a
serving step, and the block attention of the softmax layers.

Marshalling and checks only, as in the package's other entry points: every
function names the entry point of ``include/flare_gdn.h`` it calls, checks
every tensor (dtype, shape, strides, device) before the library sees its
pointer, and enqueues on the current stream of the tensors' device.  As the
package's other calls they record no graph, whatever their inputs require:
``autograd`` has the differentiable forms, under the same names.
"""
from __future__ import annotations

import ctypes
import math

import numpy as np

from . import BF16, F32, _check, _chk as _chk_slow, _chk_buf, _fail, _gpu_device, _io_dtype_of, lib

_module = None


def _torch():
    global _module
    if _module is None:
        import torch
        _module = torch
    return _module


LINEAR, SILU, SIGMOID = 0, 1, 2
TABLES_OK, TABLES_NO_PAGES, TABLES_TOO_MANY_TOKENS, TABLES_TOO_LONG, TABLES_BAD_LENGTH = 0, 1, 2, 3, 4


class RotaryShape(ctypes.Structure):
    _fields_ = [("q_heads", ctypes.c_int32), ("k_heads", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("half", ctypes.c_int32), ("io_dtype", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("mscale", ctypes.c_float)]


class AttentionShape(ctypes.Structure):
    _fields_ = [("block", ctypes.c_int32), ("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page", ctypes.c_int32), ("io_dtype", ctypes.c_int32),
                ("causal", ctypes.c_int32), ("scale", ctypes.c_float)]


def declare(L):
    """Argument types of the entry points below (called once by lib())."""
    P, I32, I64, SZ, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    RP, AP = ctypes.POINTER(RotaryShape), ctypes.POINTER(AttentionShape)
    L.flare_gated_norm.argtypes = [I64, I32, I32, I32, P, I64, P, I64, P, I32, F, P, P, P]
    L.flare_gated_norm_bwd_workspace_size.argtypes = [I64, I32, I32]
    L.flare_gated_norm_bwd_workspace_size.restype = SZ
    L.flare_gated_norm_bwd.argtypes = [I64, I32, I32, I32, P, I64, P, I64, P, I32, P, P, I64, P, P, P, P, SZ, P]
    L.flare_residual_norm.argtypes = [I64, I32, I32, I32, P, I64, P, P, I64, P, P, P, I32, F, P, P, P, P]
    L.flare_residual_norm_bwd_workspace_size.argtypes = [I64, I32]
    L.flare_residual_norm_bwd_workspace_size.restype = SZ
    L.flare_residual_norm_bwd.argtypes = [I64, I32, I32, I32, P, I64, P, P, I64, P, P, P, I32] + [P] * 9 + [P, SZ, P]
    L.flare_rotary.argtypes = [I64, RP, P, P, P, I64, P, I64, I32, P, P, P]
    L.flare_rotary_cache.argtypes = [I64, RP, P, P, P, I64, P, I64, P, I64, P, P, P, P, I64, I32, P]
    QN = [I64, RP, P, P, P, I64, P, I64]
    L.flare_qk_norm_rotary.argtypes = QN + [P, P, F, P, P, P]
    L.flare_qk_norm_rotary_bwd_workspace_size.argtypes = [I64, I32]
    L.flare_qk_norm_rotary_bwd_workspace_size.restype = SZ
    L.flare_qk_norm_rotary_bwd.argtypes = QN + [P, P, F, P, I64, P, I64, P, P, P, P, P, SZ, P]
    L.flare_qk_norm_rotary_cache.argtypes = QN + [P, I64, P, P, F, P, P, P, P, I64, I32, P]
    L.flare_qk_norm_rotary_cache_fp4.argtypes = QN + [P, I64, P, P, F, P, P, P, P, P, P, I64, I32, P]
    L.flare_cache_fp4_rows.argtypes = [I64, I32, I32, I32, P, P, P, P, P, I64, I32, P, P, P]
    L.flare_step_tables.argtypes = [I32, P, P, P, I32, P, I64, P, I32, I32, I64, P, P, P, P, P, P, P]
    L.flare_block_attention_workspace_size.argtypes = [I32, AP, I32, I32]
    L.flare_block_attention_workspace_size.restype = SZ
    L.flare_block_attention.argtypes = [I32, AP, P, P, P, I64, P, I32, P, I32, P, I32, P, P, P, SZ, P]
    L.flare_block_attention_fp4_workspace_size.argtypes = [I32, AP, I32, I32]
    L.flare_block_attention_fp4_workspace_size.restype = SZ
    L.flare_block_attention_fp4.argtypes = [I32, AP, P, P, P, P, P, I64, P, I32, P, I32, P, I32, P, P, P, SZ, P]
    for name in ("flare_gated_norm", "flare_gated_norm_bwd", "flare_residual_norm", "flare_residual_norm_bwd",
                 "flare_rotary", "flare_rotary_cache", "flare_qk_norm_rotary", "flare_qk_norm_rotary_bwd",
                 "flare_qk_norm_rotary_cache", "flare_qk_norm_rotary_cache_fp4", "flare_cache_fp4_rows",
                 "flare_step_tables", "flare_block_attention", "flare_block_attention_fp4"):
        getattr(L, name).restype = ctypes.c_int


def _lead(t, name):
    """(device, io dtype) of the tensor that sets them for a call."""
    if t is not None and t.is_cuda:
        dtype = t.dtype
        if dtype == _torch().bfloat16 or dtype == _module.float32:
            return t.device, dtype
    return _gpu_device(t, name), _io_dtype_of(t, name)


def _run(dev, fn, *args):
    """fn(*args, stream) with the tensors' device current, on its current stream."""
    C = _module._C
    index = dev.index
    if C._cuda_getDevice() == index:
        status = fn(*args, C._cuda_getCurrentRawStream(index))
    else:
        with _module.cuda.device(dev):
            status = fn(*args, C._cuda_getCurrentRawStream(index))
    if status:
        _check(status)


def _chk(t, name, shape, dtype, dev, optional=False):
    """The package's check, its message formed only where something is wrong: a
    serving step's calls are as short as their checks."""
    if t is None or t.dtype != dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        _chk_slow(t, name, shape, dtype, dev, optional)


def _i32(value, name):
    """A size as the library's 32 bits hold it."""
    value = int(value)
    if not -0x80000000 <= value <= 0x7FFFFFFF:
        _fail("%s = %d is beyond 32 bits" % (name, value), 4)
    return value


def _ptr(t):
    return None if t is None else t.data_ptr()


def _token_rows(t, name, shape, dtype, dev):
    """t has this shape, dtype and device, and contiguous token rows; returns
    the elements between tokens (a slice of a wider row has more than its own)."""
    if t is None:
        _fail("%s is required" % name, 1)
    strides = t.stride()
    if len(strides) == 3 and t.dtype == dtype and t.shape == shape and t.device == dev:  # the usual case, in short
        token, head, channel = strides
        tokens, heads, d = shape
        if channel == 1 and head == d and (tokens <= 1 or token >= heads * d):
            return token if tokens > 1 else heads * d
    if t.dtype != dtype:
        _fail("%s: dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.shape != shape:
        _fail("%s: shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.device != dev:
        _fail("%s is on %s, expected %s" % (name, t.device, dev))
    if shape[0] > 1 and t.is_contiguous():
        return strides[0]
    row = 1
    for size, stride in zip(reversed(shape[1:]), reversed(strides[1:])):
        if size != 1 and stride != row:
            _fail("%s: a token's row must be contiguous" % name, 3)
        row *= size
    if shape[0] <= 1:
        return row
    if strides[0] < row:
        _fail("%s: token stride %d below a row of %d" % (name, strides[0], row))
    return strides[0]


def _out(t, name, shape, dtype, dev):
    """An output buffer the caller gave, or a new one."""
    if t is None:
        return _module.empty(shape, dtype=dtype, device=dev)
    _chk(t, name, shape, dtype, dev)
    return t


def _out_like(t, name, x):
    """The same, packed and like x."""
    if t is None:
        return _module.empty_like(x, memory_format=_module.contiguous_format)
    _chk(t, name, x.shape, x.dtype, x.device)
    return t


def _io(dtype):
    return BF16 if dtype == _module.bfloat16 else F32


def _workspace(t, need, dev):
    torch = _torch()
    if t is None:
        return torch.empty((need,), dtype=torch.uint8, device=dev)
    _chk_buf(t, "workspace", need, torch.uint8, dev)
    return t


# ---------------------------------------------------------------- norms

def _norm_inputs(x, weight, gate):
    """x [T, d] or [T, H, d] io, weight [d] fp32, gate like x or None; returns
    (T, H, d, io dtype, device, x stride, gate stride)."""
    dev, io = _lead(x, "x")
    shape = x.shape
    if len(shape) == 3:
        T, H, d = shape
    elif len(shape) == 2:
        (T, d), H = shape, 1
    else:
        _fail("x must be [T, d] or [T, H, d], got shape %s" % (tuple(shape),))
    if H > 0x7FFFFFFF or d > 0x7FFFFFFF:
        _fail("x: %d heads of %d channels" % (H, d), 4)
    xs = _token_rows(x, "x", shape, io, dev)
    _chk(weight, "weight", (d,), _module.float32, dev)
    gs = _token_rows(gate, "gate", shape, io, dev) if gate is not None else 0
    return T, H, d, io, dev, xs, gs


def gated_norm(x, weight, gate=None, activation=SILU, eps=1e-6, out=None, want_rstd=False, rstd=None):
    """y = x / sqrt(mean x^2 + eps) * weight * act(gate) over the last dimension
    (flare_gated_norm): the norm behind a block with its gate.  x [T, H, d] or
    [T, d] io; gate like x or None; both may be slices of wider token rows;
    weight [d] fp32.  Returns y, or (y, rstd) with want_rstd or `rstd` (fp32
    [T, H] or [T], what gated_norm_bwd reads)."""
    T, H, d, io, dev, xs, gs = _norm_inputs(x, weight, gate)
    y = _out_like(out, "out", x)
    if rstd is not None or want_rstd:
        rstd = _out(rstd, "rstd", x.shape[:-1], _module.float32, dev)
    _run(dev, lib().flare_gated_norm, T, H, d, _io(io), x.data_ptr(), xs, _ptr(gate), gs, weight.data_ptr(), activation,
         eps, y.data_ptr(), _ptr(rstd))
    return y if rstd is None else (y, rstd)


def gated_norm_bwd_workspace_bytes(T, H, d) -> int:
    """flare_gated_norm_bwd_workspace_size."""
    return int(lib().flare_gated_norm_bwd_workspace_size(int(T), _i32(H, "H"), _i32(d, "d")))


def gated_norm_bwd(x, weight, gate, dy, rstd, activation=SILU, workspace=None, out=None):
    """Reverse mode of gated_norm (flare_gated_norm_bwd).  Returns (dx, dgate,
    dweight), dgate None without a gate; `out` = such a tuple reuses buffers."""
    torch = _torch()
    T, H, d, io, dev, xs, gs = _norm_inputs(x, weight, gate)
    ds = _token_rows(dy, "dy", x.shape, io, dev)
    _chk(rstd, "rstd", x.shape[:-1], torch.float32, dev)
    dx, dgate, dweight = out if out is not None else (None, None, None)
    dx = _out_like(dx, "dx", x)
    dgate = _out_like(dgate, "dgate", gate) if gate is not None else None
    dweight = _out_like(dweight, "dweight", weight)
    need = gated_norm_bwd_workspace_bytes(T, H, d)
    workspace = _workspace(workspace, need, dev)
    _run(dev, lib().flare_gated_norm_bwd, T, H, d, _io(io), _ptr(x), xs, _ptr(gate), gs, _ptr(weight),
         int(activation), _ptr(rstd), _ptr(dy), ds, _ptr(dx), _ptr(dgate), _ptr(dweight), _ptr(workspace),
         workspace.numel())
    return dx, dgate, dweight


def _residual_inputs(x, residual, w_pre, w_post, gate, scale):
    dev, io = _lead(x, "x")
    torch = _module
    if x.dim() != 2:
        _fail("x must be [T, C], got shape %s" % (tuple(x.shape),))
    T, C = x.shape
    _i32(C, "C")
    xs = _token_rows(x, "x", (T, C), io, dev)
    res = io if residual is not None and residual.dtype == io else _io_dtype_of(residual, "residual")
    _chk(residual, "residual", (T, C), res, dev)
    _chk(w_pre, "w_pre", (C,), torch.float32, dev)
    _chk(w_post, "w_post", (C,), torch.float32, dev, optional=True)
    _chk(scale, "scale", (C,), torch.float32, dev, optional=True)
    gs = _token_rows(gate, "gate", (T, C), io, dev) if gate is not None else 0
    return T, C, io, res, dev, xs, gs


def residual_norm(x, residual, w_pre, w_post=None, gate=None, scale=None, activation=SIGMOID, eps=1e-6, out=None,
                  want_rstd=False, rstd=None):
    """What lies between two blocks, in one pass (flare_residual_norm):
        n = x / sqrt(mean x^2 + eps) * w_post   (x itself without w_post)
        h = residual + scale * act(gate) * n
        y = h / sqrt(mean h^2 + eps) * w_pre
    x, gate [T, C] io (slices of wider rows allowed); residual [T, C] fp32, or
    bf16 with bf16 io; weights and scale [C] fp32.  Returns (h, y), or
    (h, y, rstd) with want_rstd or `rstd` (fp32 [T, 2], what
    residual_norm_bwd reads); `out` = (h, y) reuses buffers."""
    T, C, io, res, dev, xs, gs = _residual_inputs(x, residual, w_pre, w_post, gate, scale)
    h, y = out if out is not None else (None, None)
    h, y = _out_like(h, "h", residual), _out_like(y, "y", x)
    if rstd is not None or want_rstd:
        rstd = _out(rstd, "rstd", (T, 2), _module.float32, dev)
    _run(dev, lib().flare_residual_norm, T, C, _io(io), _io(res), _ptr(x), xs, _ptr(residual), _ptr(gate), gs,
         _ptr(w_pre), _ptr(w_post), _ptr(scale), int(activation), float(eps), _ptr(h), _ptr(y), _ptr(rstd))
    return (h, y) if rstd is None else (h, y, rstd)


def residual_norm_bwd_workspace_bytes(T, C) -> int:
    """flare_residual_norm_bwd_workspace_size."""
    return int(lib().flare_residual_norm_bwd_workspace_size(int(T), _i32(C, "C")))


def residual_norm_bwd(x, residual, w_pre, dy, dh, rstd, w_post=None, gate=None, scale=None, activation=SIGMOID,
                      workspace=None, out=None):
    """Reverse mode of residual_norm (flare_residual_norm_bwd): dy, dh the
    gradients of y and h (dh None = 0).  Returns a dict dx, dresidual, dgate,
    dw_pre, dw_post, dscale (None for what the forward did not have); `out` =
    such a dict reuses its buffers."""
    torch = _torch()
    T, C, io, res, dev, xs, gs = _residual_inputs(x, residual, w_pre, w_post, gate, scale)
    _chk(dy, "dy", (T, C), io, dev)
    _chk(dh, "dh", (T, C), res, dev, optional=True)
    _chk(rstd, "rstd", (T, 2), torch.float32, dev)
    out = out or {}
    g = {"dx": _out_like(out.get("dx"), "dx", x),
         "dresidual": _out_like(out.get("dresidual"), "dresidual", residual),
         "dgate": _out_like(out.get("dgate"), "dgate", gate) if gate is not None else None,
         "dw_pre": _out_like(out.get("dw_pre"), "dw_pre", w_pre),
         "dw_post": _out_like(out.get("dw_post"), "dw_post", w_post) if w_post is not None else None,
         "dscale": _out_like(out.get("dscale"), "dscale", scale) if scale is not None else None}
    workspace = _workspace(workspace, residual_norm_bwd_workspace_bytes(T, C), dev)
    _run(dev, lib().flare_residual_norm_bwd, T, C, _io(io), _io(res), _ptr(x), xs, _ptr(residual), _ptr(gate), gs,
         _ptr(w_pre), _ptr(w_post), _ptr(scale), int(activation), _ptr(rstd), _ptr(dy), _ptr(dh), _ptr(g["dx"]),
         _ptr(g["dresidual"]), _ptr(g["dgate"]), _ptr(g["dw_pre"]), _ptr(g["dw_post"]), _ptr(g["dscale"]),
         _ptr(workspace), workspace.numel())
    return g


# ---------------------------------------------------------------- rotary

def rotary_frequencies(rotary_dim, base=10000.0, scaling="none", factor=1.0, original_length=0, beta_fast=32.0,
                       beta_slow=1.0, device="cuda"):
    """(freqs, mscale) for rotary(): freqs fp64 [rotary_dim / 2] on `device`, in
    radians a position, freq_i = base^(-2i / rotary_dim), stretched for contexts
    `factor` times longer than trained on:
      "none"
      "linear"  positions divided by the factor
      "ntk"     base * factor^(rotary_dim / (rotary_dim - 2)): the slowest pair
                is stretched by the factor, the fastest not at all
      "yarn"    pairs that turn more than beta_fast times within original_length
                keep their frequency, those below beta_slow are divided by the
                factor, a linear ramp between, whose ends are rounded outwards to
                whole pairs (as programs that trained with it have it);
                mscale = 1 + 0.1 ln(factor)"""
    torch = _torch()
    n = int(rotary_dim)
    if n < 0 or n % 2:
        _fail("rotary_dim must be even and not negative (got %d)" % n)
    if not (base > 1.0 and factor >= 1.0):
        _fail("rotary base must be above 1 and the factor at least 1")
    i = np.arange(n // 2, dtype=np.float64)
    mscale = 1.0
    if scaling == "ntk" and n > 2:
        base = base * factor ** (n / (n - 2))
    f = float(base) ** (-2.0 * i / max(n, 1))
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        if original_length <= 0:
            _fail("yarn scaling needs the original length")
        if not beta_fast >= beta_slow > 0:
            _fail("yarn scaling needs beta_fast of at least beta_slow, both above 0 (got %s and %s)" % (beta_fast, beta_slow))
        # the (real) index of the pair that turns `turns` times within original_length
        pair = lambda turns: n * math.log(original_length / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
        low, high = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), n - 1)
        ramp = np.clip((i - low) / max(high - low, 1e-3), 0.0, 1.0)
        ramp[i > pair(beta_slow)] = 1.0  # the first pair too, where the ramp ends before it
        f = f * (1 - ramp) + f / factor * ramp
        mscale = 1.0 + 0.1 * math.log(factor)
    elif scaling not in ("none", "ntk"):
        _fail("rotary scaling %r unknown" % (scaling,), 4)
    return torch.from_numpy(f).to(device), mscale


def _rotary_inputs(positions, freqs, q, k, interleaved, mscale):
    dev, io = _lead(q, "q")
    torch = _module
    if q.dim() != 3 or (k is not None and k.dim() != 3):
        _fail("q and k must be [T, H, d]")
    T, Hq, d = q.shape
    Hk = 0 if k is None else k.shape[1]
    if Hq > 0x7FFFFFFF or Hk > 0x7FFFFFFF or d > 0x7FFFFFFF:
        _fail("rotary: %d and %d heads of %d channels" % (Hq, Hk, d), 4)
    qs = _token_rows(q, "q", q.shape, io, dev)
    ks = 0 if k is None else _token_rows(k, "k", (T, Hk, d), io, dev)
    _chk(positions, "positions", (T,), torch.int32, dev)
    if freqs is None or freqs.dim() != 1:
        _fail("freqs must be fp64 [rotary_dim / 2]")
    _chk(freqs, "freqs", freqs.shape, torch.float64, dev)
    return T, RotaryShape(Hq, Hk, d, freqs.shape[0], _io(io), 1 if interleaved else 0, mscale), io, dev, qs, ks


def rotary(positions, freqs, q, k=None, interleaved=False, mscale=1.0, inverse=False, out=None):
    """Rotary positions on the first 2 * len(freqs) channels of every head
    (flare_rotary): pairs (i, half + i), or (2i, 2i + 1) when interleaved, turned
    by positions * freqs and scaled by mscale; the other channels pass through.
    q [T, Hq, d], k [T, Hk, d] or None, io, slices of wider rows allowed;
    positions int32 [T].  inverse=True turns back: the gradients.  Returns
    (q, k) turned, packed; `out` = (q, k) reuses buffers."""
    T, shp, io, dev, qs, ks = _rotary_inputs(positions, freqs, q, k, interleaved, mscale)
    qo, ko = out if out is not None else (None, None)
    qo = _out_like(qo, "q out", q)
    ko = _out_like(ko, "k out", k) if k is not None else None
    _run(dev, lib().flare_rotary, T, ctypes.byref(shp), _ptr(positions), _ptr(freqs), _ptr(q), qs, _ptr(k), ks,
         1 if inverse else 0, _ptr(qo), _ptr(ko))
    return qo, ko


def rotary_cache(positions, freqs, q, k, v, slots, k_cache, v_cache, interleaved=False, mscale=1.0, out=None):
    """The serving form (flare_rotary_cache): returns q turned; k turned and v
    are written to the cache's pages [num_pages, Hk, page, d], row t at slot
    slots[t] (int64, page id * page + offset; -1 writes nothing)."""
    if k is None or v is None:
        _fail("k and v are required", 1)
    T, shp, io, dev, qs, ks = _rotary_inputs(positions, freqs, q, k, interleaved, mscale)
    vs = _token_rows(v, "v", k.shape, io, dev)
    _chk(slots, "slots", (T,), _module.int64, dev)
    pages, page = _chk_cache(k_cache, v_cache, k.shape[1], k.shape[2], io, dev)
    qo = _out_like(out, "out", q)
    _run(dev, lib().flare_rotary_cache, T, ctypes.byref(shp), _ptr(positions), _ptr(freqs), _ptr(q), qs, _ptr(k), ks,
         _ptr(v), vs, _ptr(slots), _ptr(qo), _ptr(k_cache), _ptr(v_cache), pages, page)
    return qo


def _chk_cache(k_cache, v_cache, heads, d, io, dev):
    """Key and value pages [num_pages, heads, page, d]; returns (num_pages, page)."""
    if not isinstance(k_cache, _torch().Tensor) or not isinstance(v_cache, _module.Tensor) or k_cache.dim() != 4:
        _fail("k_cache and v_cache must be tensors [num_pages, heads, page, d]")
    pages, page = k_cache.shape[0], k_cache.shape[2]
    if heads > 0x7FFFFFFF or page > 0x7FFFFFFF:
        _i32(heads, "cache heads"), _i32(page, "page")
    _chk(k_cache, "k_cache", (pages, heads, page, d), io, dev)
    _chk(v_cache, "v_cache", (pages, heads, page, d), io, dev)
    return pages, page


# ---------------------------------------------------------------- q/k norms with rotary positions

def _norm_weights(q_weight, k_weight, k, dim, dev):
    if k is None and k_weight is not None:
        _fail("k_weight without k")
    if q_weight is not None:
        _chk(q_weight, "q_weight", (dim,), _module.float32, dev)
    if k_weight is not None:
        _chk(k_weight, "k_weight", (dim,), _module.float32, dev)


def qk_norm_rotary(positions, freqs, q, k=None, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, mscale=1.0,
                   out=None):
    """The norms of queries and keys for each head and their rotary positions in
    one pass (flare_qk_norm_rotary): x / sqrt(mean x^2 + eps) * weight over the
    last dimension, then rotary().  q_weight, k_weight fp32 [d], or None: that
    side is turned, not normed.  The other arguments and the result are
    rotary()'s."""
    T, shp, io, dev, qs, ks = _rotary_inputs(positions, freqs, q, k, interleaved, mscale)
    _norm_weights(q_weight, k_weight, k, shp.dim, dev)
    qo, ko = out if out is not None else (None, None)
    qo = _out_like(qo, "q out", q)
    ko = _out_like(ko, "k out", k) if k is not None else None
    _run(dev, lib().flare_qk_norm_rotary, T, ctypes.byref(shp), _ptr(positions), _ptr(freqs), _ptr(q), qs, _ptr(k), ks,
         _ptr(q_weight), _ptr(k_weight), eps, _ptr(qo), _ptr(ko))
    return qo, ko


def qk_norm_rotary_bwd_workspace_bytes(T, d) -> int:
    """flare_qk_norm_rotary_bwd_workspace_size."""
    return int(lib().flare_qk_norm_rotary_bwd_workspace_size(int(T), _i32(d, "d")))


def qk_norm_rotary_bwd(positions, freqs, q, k, dq_out, dk_out, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                       mscale=1.0, workspace=None, out=None):
    """Reverse mode of qk_norm_rotary (flare_qk_norm_rotary_bwd): dq_out, dk_out
    the gradients of its outputs (slices of wider rows allowed; k and dk_out
    None without keys).  Returns a dict dq, dk, dq_weight, dk_weight (None for
    what the forward did not have); `out` = such a dict reuses its buffers."""
    T, shp, io, dev, qs, ks = _rotary_inputs(positions, freqs, q, k, interleaved, mscale)
    _norm_weights(q_weight, k_weight, k, shp.dim, dev)
    dqs = _token_rows(dq_out, "dq_out", q.shape, io, dev)
    if k is None and dk_out is not None:
        _fail("dk_out without k")
    dks = 0 if k is None else _token_rows(dk_out, "dk_out", k.shape, io, dev)
    out = out or {}
    g = {"dq": _out_like(out.get("dq"), "dq", q),
         "dk": _out_like(out.get("dk"), "dk", k) if k is not None else None,
         "dq_weight": _out_like(out.get("dq_weight"), "dq_weight", q_weight) if q_weight is not None else None,
         "dk_weight": _out_like(out.get("dk_weight"), "dk_weight", k_weight) if k_weight is not None else None}
    if q_weight is not None or k_weight is not None:
        workspace = _workspace(workspace, lib().flare_qk_norm_rotary_bwd_workspace_size(T, shp.dim), dev)
    _run(dev, lib().flare_qk_norm_rotary_bwd, T, ctypes.byref(shp), _ptr(positions), _ptr(freqs), _ptr(q), qs, _ptr(k), ks,
         _ptr(q_weight), _ptr(k_weight), eps, _ptr(dq_out), dqs, _ptr(dk_out), dks, _ptr(g["dq"]), _ptr(g["dk"]),
         _ptr(g["dq_weight"]), _ptr(g["dk_weight"]), _ptr(workspace), 0 if workspace is None else workspace.numel())
    return g


def qk_norm_rotary_cache(positions, freqs, q, k, v, slots, k_cache, v_cache, q_weight=None, k_weight=None, eps=1e-6,
                         interleaved=False, mscale=1.0, out=None):
    """The serving form (flare_qk_norm_rotary_cache): returns q normed and
    turned; k normed and turned and v are written to the cache as by
    rotary_cache."""
    if k is None or v is None:
        _fail("k and v are required", 1)
    T, shp, io, dev, qs, ks = _rotary_inputs(positions, freqs, q, k, interleaved, mscale)
    _norm_weights(q_weight, k_weight, k, shp.dim, dev)
    vs = _token_rows(v, "v", k.shape, io, dev)
    _chk(slots, "slots", (T,), _module.int64, dev)
    pages, page = _chk_cache(k_cache, v_cache, k.shape[1], k.shape[2], io, dev)
    qo = _out_like(out, "out", q)
    _run(dev, lib().flare_qk_norm_rotary_cache, T, ctypes.byref(shp), _ptr(positions), _ptr(freqs), _ptr(q), qs, _ptr(k),
         ks, _ptr(v), vs, _ptr(q_weight), _ptr(k_weight), eps, _ptr(slots), _ptr(qo), _ptr(k_cache), _ptr(v_cache), pages,
         page)
    return qo


def cache_fp4(num_pages, heads, page, d, device="cuda"):
    """(codes, scales) of an empty cache in 4 bits, all zeros: codes uint8
    [num_pages, heads, page, d / 2], scales uint8 [num_pages, heads, d / 32,
    page].  A value is its code (0, 1/2, 1, 3/2, 2, 3, 4, 6 and a sign) times
    2^(scale - 127), the scale that of its 32 channels."""
    torch = _torch()
    if d < 32 or d % 32:
        _fail("a cache in 4 bits has groups of 32 channels, not %d" % d, 4)
    return (torch.zeros((num_pages, heads, page, d // 2), dtype=torch.uint8, device=device),
            torch.zeros((num_pages, heads, d // 32, page), dtype=torch.uint8, device=device))


def _chk_cache_fp4(cache, name, heads, d, dev):
    """(codes, scales) of a cache in 4 bits; returns (num_pages, page)."""
    if not isinstance(cache, (tuple, list)) or len(cache) != 2 or cache[0] is None or cache[0].dim() != 4:
        _fail("%s must be (codes [num_pages, heads, page, d / 2], scales [num_pages, heads, d / 32, page])" % name)
    codes, scales = cache
    pages, page = codes.shape[0], codes.shape[2]
    if d % 32:
        _fail("a cache in 4 bits has groups of 32 channels, not %d" % d, 4)
    if max(heads, page) > 0x7FFFFFFF:
        _i32(heads, "cache heads"), _i32(page, "page")
    _chk(codes, name + " codes", (pages, heads, page, d // 2), _module.uint8, dev)
    _chk(scales, name + " scales", (pages, heads, d // 32, page), _module.uint8, dev)
    return pages, page


def _chk_caches_fp4(k_cache, v_cache, heads, d, dev):
    if isinstance(k_cache, (tuple, list)) and isinstance(v_cache, (tuple, list)) and len(k_cache) == len(v_cache) == 2:
        kc, ks = k_cache
        vc, vs = v_cache
        if kc is not None and ks is not None and vc is not None and vs is not None:  # all as they should be, in short
            codes, scales, u8 = kc.shape, ks.shape, _module.uint8
            if (len(codes) == len(scales) == 4 and vc.shape == codes and vs.shape == scales and d % 32 == 0
                    and codes[1] == scales[1] == heads <= 0x7FFFFFFF and 2 * codes[3] == 32 * scales[2] == d
                    and codes[0] == scales[0] and codes[2] == scales[3] <= 0x7FFFFFFF
                    and kc.dtype == ks.dtype == vc.dtype == vs.dtype == u8 and kc.device == ks.device == vc.device == vs.device == dev
                    and kc.is_contiguous() and ks.is_contiguous() and vc.is_contiguous() and vs.is_contiguous()):
                return codes[0], codes[2]
    sizes = _chk_cache_fp4(k_cache, "k_cache", heads, d, dev)
    if _chk_cache_fp4(v_cache, "v_cache", heads, d, dev) != sizes:
        _fail("k_cache and v_cache have pages of different number or size")
    return sizes


def qk_norm_rotary_cache_fp4(positions, freqs, q, k, v, slots, k_cache, v_cache, q_weight=None, k_weight=None, eps=1e-6,
                             interleaved=False, mscale=1.0, out=None):
    """qk_norm_rotary_cache into a cache in 4 bits
    (flare_qk_norm_rotary_cache_fp4): k_cache and v_cache are (codes, scales) as
    from cache_fp4().  Without weights it is rotary_cache into such a cache."""
    if k is None or v is None:
        _fail("k and v are required", 1)
    T, shp, io, dev, qs, ks = _rotary_inputs(positions, freqs, q, k, interleaved, mscale)
    _norm_weights(q_weight, k_weight, k, shp.dim, dev)
    vs = _token_rows(v, "v", k.shape, io, dev)
    _chk(slots, "slots", (T,), _module.int64, dev)
    pages, page = _chk_caches_fp4(k_cache, v_cache, k.shape[1], k.shape[2], dev)
    qo = _out_like(out, "out", q)
    _run(dev, lib().flare_qk_norm_rotary_cache_fp4, T, ctypes.byref(shp), _ptr(positions), _ptr(freqs), _ptr(q), qs,
         _ptr(k), ks, _ptr(v), vs, _ptr(q_weight), _ptr(k_weight), eps, _ptr(slots), _ptr(qo), _ptr(k_cache[0]),
         _ptr(k_cache[1]), _ptr(v_cache[0]), _ptr(v_cache[1]), pages, page)
    return qo


def cache_fp4_rows(slots, k_cache, v_cache=None, dtype=None, out=None):
    """Rows of a cache in 4 bits as bf16 (or dtype = float32) values
    (flare_cache_fp4_rows): [T, heads, d], row t that at slots[t] (int64), zeros
    for a slot of no page.  Returns (k, v), or k without v_cache; `out` likewise
    reuses buffers."""
    torch = _torch()
    dev = _gpu_device(slots, "slots")
    io = torch.bfloat16 if dtype is None else dtype
    if io not in (torch.bfloat16, torch.float32):
        _fail("cache_fp4_rows gives bfloat16 or float32, not %s" % io, 4)
    if slots.dim() != 1:
        _fail("slots must be int64 [T]")
    T = slots.shape[0]
    _chk(slots, "slots", (T,), torch.int64, dev)
    if not isinstance(k_cache, (tuple, list)) or len(k_cache) != 2 or k_cache[0] is None or k_cache[0].dim() != 4:
        _fail("k_cache must be (codes, scales)")
    heads, d = k_cache[0].shape[1], 2 * k_cache[0].shape[3]
    pages, page = (_chk_cache_fp4(k_cache, "k_cache", heads, d, dev) if v_cache is None
                   else _chk_caches_fp4(k_cache, v_cache, heads, d, dev))
    ko, vo = (None, None) if out is None else out if v_cache is not None else (out, None)
    ko = _out(ko, "k out", (T, heads, d), io, dev)
    vo = _out(vo, "v out", (T, heads, d), io, dev) if v_cache is not None else None
    v_codes, v_scales = (None, None) if v_cache is None else v_cache
    _run(dev, lib().flare_cache_fp4_rows, T, heads, d, _io(io), _ptr(slots), _ptr(k_cache[0]), _ptr(k_cache[1]),
         _ptr(v_codes), _ptr(v_scales), pages, page, _ptr(ko), _ptr(vo))
    return ko if v_cache is None else (ko, vo)


# ---------------------------------------------------------------- serving-step tables

def step_tables(seq_lens, new_lens, block_table, free_pages, pages_used, page, max_tokens, position_offset=0,
                out=None):
    """The tables of a serving step, built on the GPU from the requests' lengths
    (flare_step_tables).  seq_lens, new_lens int32 [R]: tokens held and added;
    block_table int32 [R, max_pages]: the pages opened now are entered into it;
    free_pages int32 [F], of which the first pages_used[0] (int32 [1]) are taken.
    Returns a dict of device tensors: cu_new [R + 1], positions [max_tokens]
    (plus position_offset), slots int64 [max_tokens] (-1 behind the last token),
    seq_lens [R] and pages_used [1] after the step, status [1] (TABLES_OK, or why
    nothing was allocated).  `out` = such a dict reuses its buffers."""
    torch = _torch()
    i32 = torch.int32
    dev = _gpu_device(seq_lens, "seq_lens")
    if seq_lens.dim() != 1 or block_table is None or block_table.dim() != 2:
        _fail("seq_lens must be [R] and block_table [R, max_pages]")
    R, wide = seq_lens.shape[0], block_table.shape[1]
    page, position_offset = int(page), int(position_offset)
    if max(R, wide, page, position_offset) > 0x7FFFFFFF or min(page, position_offset) < 0:
        _i32(R, "requests"), _i32(wide, "max_pages"), _i32(page, "page"), _i32(position_offset, "position_offset")
    _chk(seq_lens, "seq_lens", (R,), i32, dev)
    _chk(new_lens, "new_lens", (R,), i32, dev)
    _chk(block_table, "block_table", (R, wide), i32, dev)
    if free_pages is None or free_pages.dim() != 1:
        _fail("free_pages must be int32 [F]")
    _chk(free_pages, "free_pages", free_pages.shape, i32, dev)
    _chk(pages_used, "pages_used", (1,), i32, dev)
    M = int(max_tokens)
    if M < 0:
        _fail("max_tokens must not be negative")
    if out is None:  # the small ones share a buffer
        cu, lens, used, status = torch.split_with_sizes(seq_lens.new_empty(2 * R + 3), (R + 1, R, 1, 1))
        t = {"cu_new": cu, "positions": seq_lens.new_empty(M), "slots": seq_lens.new_empty(M, dtype=torch.int64),
             "seq_lens": lens, "pages_used": used, "status": status}
    else:
        t = {"cu_new": _out(out.get("cu_new"), "cu_new", (R + 1,), i32, dev),
             "positions": _out(out.get("positions"), "positions", (M,), i32, dev),
             "slots": _out(out.get("slots"), "slots", (M,), torch.int64, dev),
             "seq_lens": _out(out.get("seq_lens"), "seq_lens out", (R,), i32, dev),
             "pages_used": _out(out.get("pages_used"), "pages_used out", (1,), i32, dev),
             "status": _out(out.get("status"), "status", (1,), i32, dev)}
    _run(dev, lib().flare_step_tables, R, _ptr(seq_lens), _ptr(new_lens), _ptr(block_table), wide,
         _ptr(free_pages), free_pages.shape[0], _ptr(pages_used), page, position_offset, M,
         _ptr(t["cu_new"]), _ptr(t["positions"]), _ptr(t["slots"]), _ptr(t["seq_lens"]), _ptr(t["pages_used"]),
         _ptr(t["status"]))
    return t


# ---------------------------------------------------------------- block attention

def _attention_shape(R, B, q_heads, kv_heads, d, page, max_seq_len, prefix_len):
    sizes = (("R", R), ("B", B), ("q_heads", q_heads), ("kv_heads", kv_heads), ("d", d), ("page", page),
             ("max_seq_len", max_seq_len), ("prefix_len", prefix_len))
    R, B, q_heads, kv_heads, d, page, max_seq_len, prefix_len = (_i32(n, name) for name, n in sizes)
    return R, ctypes.byref(AttentionShape(B, q_heads, kv_heads, d, page, BF16, 0, 0.0)), max_seq_len, prefix_len


def block_attention_workspace_bytes(R, B, q_heads, kv_heads, d, page, max_seq_len, prefix_len) -> int:
    """flare_block_attention_workspace_size (bf16)."""
    return int(lib().flare_block_attention_workspace_size(
        *_attention_shape(R, B, q_heads, kv_heads, d, page, max_seq_len, prefix_len)))


def block_attention_fp4_workspace_bytes(R, B, q_heads, kv_heads, d, page, max_seq_len, prefix_len) -> int:
    """flare_block_attention_fp4_workspace_size."""
    return int(lib().flare_block_attention_fp4_workspace_size(
        *_attention_shape(R, B, q_heads, kv_heads, d, page, max_seq_len, prefix_len)))


def _attention_inputs(q, what):
    """(device, R, B, Hq, d) of an attention's queries."""
    torch = _torch()
    dev = _gpu_device(q, "q")
    if q.dim() != 4:
        _fail("q must be [R, B, Hq, d], got shape %s" % (tuple(q.shape),))
    if q.dtype != torch.bfloat16:
        _fail("%s is built for bfloat16, got %s" % (what, q.dtype), 4)
    R, B, Hq, d = q.shape
    if max(R, B, Hq, d) > 0x7FFFFFFF:
        _fail("q: shape %s" % (tuple(q.shape),), 4)
    _chk(q, "q", (R, B, Hq, d), torch.bfloat16, dev)
    return dev, R, B, Hq, d


def _attend(size, attend, dev, q, caches, Hk, pages, page, block_table, seq_lens, prefix_table, prefix_len, causal, scale,
            max_seq_len, out, want_lse, lse, workspace):
    """The checks and the call that both attentions share."""
    torch = _module
    R, B, Hq, d = q.shape
    if block_table is None or block_table.dim() != 2:
        _fail("block_table must be int32 [R, max_pages]")
    wide = block_table.shape[1]
    _chk(block_table, "block_table", (R, wide), torch.int32, dev)
    _chk(seq_lens, "seq_lens", (R,), torch.int32, dev)
    n = _i32(prefix_len, "prefix_len")
    if n < 0:
        _fail("prefix_len must not be negative")
    if n > 0:
        if prefix_table is None or prefix_table.dim() != 1 or prefix_table.shape[0] * page < n:
            _fail("prefix_table must be int32 with a page for every %d of the prefix's %d keys" % (page, n))
        _chk(prefix_table, "prefix_table", prefix_table.shape, torch.int32, dev)
    most = _i32(wide * page if max_seq_len is None else max_seq_len, "max_seq_len")
    shp = AttentionShape(B, Hq, Hk, d, page, BF16, 1 if causal else 0, scale)
    o = _out_like(out, "out", q)
    if lse is not None or want_lse:
        lse = _out(lse, "lse", (R, B, Hq), torch.float32, dev)
    need = int(size(R, ctypes.byref(shp), most, n))
    if need > 0:
        workspace = _workspace(workspace, need, dev)
    _run(dev, attend, R, ctypes.byref(shp), _ptr(q), *caches, pages, _ptr(block_table), wide, _ptr(seq_lens), most,
         _ptr(prefix_table) if n > 0 else None, n, _ptr(o), _ptr(lse), _ptr(workspace),
         0 if workspace is None else workspace.numel())
    return o if lse is None else (o, lse)


def block_attention(q, k_cache, v_cache, block_table, seq_lens, prefix_table=None, prefix_len=0, causal=False,
                    scale=0.0, max_seq_len=None, out=None, want_lse=False, lse=None, workspace=None):
    """The block step of a softmax layer (flare_block_attention): q [R, B, Hq, d]
    bf16 over a prefix of prefix_len keys shared by all requests (pages
    prefix_table) and each request's own seq_lens[r] keys (pages block_table[r]),
    the block's included.  causal=False: every query sees all of them;
    causal=True: query b sees the prefix and the first seq_lens[r] - (B - 1 - b)
    own keys.  Caches [num_pages, Hk, page, d] bf16.  max_seq_len bounds seq_lens
    (default: what the table holds), and the work is cut by it: lengths beyond it
    are cut.  Returns o, or
    (o, lse) with want_lse or `lse` (fp32 [R, B, Hq])."""
    dev, R, B, Hq, d = _attention_inputs(q, "block_attention")
    if not isinstance(k_cache, _module.Tensor) or k_cache.dim() != 4:
        _fail("k_cache must be a tensor [num_pages, Hk, page, d]")
    Hk = k_cache.shape[1]
    pages, page = _chk_cache(k_cache, v_cache, Hk, d, _module.bfloat16, dev)
    L = lib()
    return _attend(L.flare_block_attention_workspace_size, L.flare_block_attention, dev, q, (_ptr(k_cache), _ptr(v_cache)),
                   Hk, pages, page, block_table, seq_lens, prefix_table, prefix_len, causal, scale, max_seq_len, out,
                   want_lse, lse, workspace)


def block_attention_fp4(q, k_cache, v_cache, block_table, seq_lens, prefix_table=None, prefix_len=0, causal=False,
                        scale=0.0, max_seq_len=None, out=None, want_lse=False, lse=None, workspace=None):
    """block_attention over a cache in 4 bits (flare_block_attention_fp4): k_cache
    and v_cache are (codes, scales) as from cache_fp4(), written by
    qk_norm_rotary_cache_fp4; the other arguments and the result are
    block_attention's."""
    dev, R, B, Hq, d = _attention_inputs(q, "block_attention_fp4")
    if not isinstance(k_cache, (tuple, list)) or len(k_cache) != 2 or k_cache[0] is None or k_cache[0].dim() != 4:
        _fail("k_cache must be (codes, scales)")
    Hk = k_cache[0].shape[1]
    pages, page = _chk_caches_fp4(k_cache, v_cache, Hk, d, dev)
    L = lib()
    caches = (_ptr(k_cache[0]), _ptr(k_cache[1]), _ptr(v_cache[0]), _ptr(v_cache[1]))
    return _attend(L.flare_block_attention_fp4_workspace_size, L.flare_block_attention_fp4, dev, q, caches, Hk, pages, page,
                   block_table, seq_lens, prefix_table, prefix_len, causal, scale, max_seq_len, out, want_lse, lse,
                   workspace)
