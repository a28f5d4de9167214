"""torch.autograd wrappers of the dual-stream Gated DeltaNet layer and of the
norms and rotary positions around it.

``gdn_dual(varlen, q, k, v, alpha, beta, qn, kn, vn, alpha_n, beta_n,
block_size, h0=None, scale=0.0, flags=0, ckpt_stride=1, window=0)`` returns
``(o, on, h_final)`` and records the reverse mode: the forward runs
flare_gdn_dual_fwd with the chunk-start states saved, the backward runs
flare_gdn_dual_bwd with the incoming output gradients.  By default every
chunk-start state is kept and so is the forward's workspace, whose chunk
matrices the backward then reads.  With ckpt_stride > 1 only every
ckpt_stride-th state is kept (the backward rebuilds the others) and nothing
else survives the forward; window > 0 runs both passes in windows of that
many chunks of every document, so their workspaces no longer grow with the
sequence.  Marshalling only, like the binding it calls: every step of the
computation runs in the library's HIP kernels.

Method: "FLARE: Diffusion for Hybrid Language Model" (papernotes.org notes),
Key designs items 2-3 (the dual-stream forward and the block-level gradient
injection into the causal chain).
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import Varlen, gdn_dual_bwd, gdn_dual_fwd, workspace_bytes, _io_of
from . import layer as _layer

_GRADS = ("dq", "dk", "dv", "dalpha", "dbeta", "dqn", "dkn", "dvn", "dalpha_n", "dbeta_n")


class GDNDualFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, varlen, block_size, scale, flags, stride, window, q, k, v, alpha, beta, qn, kn, vn, alpha_n,
                beta_n, h0):
        T, H, d = q.shape
        fws = None
        nbytes = workspace_bytes(varlen, H, d, block_size, _io_of(q), flags, window=window)
        if nbytes > 0:
            fws = torch.empty((nbytes,), dtype=torch.uint8, device=q.device)
        o, on, hf, ckpt = gdn_dual_fwd(varlen, q, k, v, alpha, beta, qn, kn, vn, alpha_n, beta_n, block_size,
                                       h0=h0, scale=scale, flags=flags, want_ckpt=True, workspace=fws,
                                       ckpt_stride=stride, window=window)
        ctx.varlen, ctx.block_size, ctx.scale, ctx.flags = varlen, block_size, scale, flags
        ctx.stride, ctx.window = stride, window
        ctx.has_h0 = h0 is not None
        # the one-pass forward's chunk matrices serve the backward; the memory
        # modes keep nothing but the strided checkpoints
        ctx.fws = fws if stride == 1 and window == 0 else None
        ctx.save_for_backward(q, k, v, alpha, beta, qn, kn, vn, alpha_n, beta_n, h0, ckpt)
        return o, on, hf

    @staticmethod
    def backward(ctx, d_o, d_on, dh_final):
        q, k, v, alpha, beta, qn, kn, vn, alpha_n, beta_n, h0, ckpt = ctx.saved_tensors
        d_o = torch.zeros_like(q) if d_o is None else d_o.contiguous()
        d_on = torch.zeros_like(q) if d_on is None else d_on.contiguous()
        if dh_final is not None:
            dh_final = dh_final.contiguous()
        g = gdn_dual_bwd(ctx.varlen, q, k, v, alpha, beta, qn, kn, vn, alpha_n, beta_n, ctx.block_size, ckpt,
                         d_o, d_on, h0=h0, dh_final=dh_final, scale=ctx.scale, flags=ctx.flags,
                         want_dh0=ctx.has_h0, fwd_workspace=ctx.fws, ckpt_stride=ctx.stride, window=ctx.window)
        ctx.fws = None
        return (None,) * 6 + tuple(g[n] for n in _GRADS) + (g["dh0"] if ctx.has_h0 else None,)


def gdn_dual(varlen: Varlen, q, k, v, alpha, beta, qn, kn, vn, alpha_n, beta_n, block_size, h0=None, scale=0.0,
             flags=0, ckpt_stride=1, window=0):
    """Differentiable dual-stream forward: (o, on, h_final).  Gradients flow
    to q, k, v, alpha, beta of both streams and to h0 (when given).
    ckpt_stride / window: the memory modes described above (window a multiple
    of ckpt_stride)."""
    return GDNDualFunction.apply(varlen, int(block_size), float(scale), int(flags), int(ckpt_stride), int(window),
                                 q, k, v, alpha, beta, qn, kn, vn, alpha_n, beta_n, h0)


# ---------------------------------------------------------------- around the GDN step
# Differentiable forms of the norms and of rotary positions.  A tensor whose
# token rows are not contiguous (a broadcast one, a transposed view) is copied
# first; a gradient that reaches the reverse mode in such a form likewise.

def _rows(t):
    """t, or a packed copy where its tokens' rows are not contiguous."""
    if t is None or t.is_contiguous():
        return t
    row = 1
    for size, stride in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if size != 1 and stride != row:
            return t.contiguous()
        row *= size
    return t if t.stride(0) >= row else t.contiguous()


class GatedNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, gate, activation, eps):
        x, gate, weight = _rows(x), _rows(gate), weight.contiguous()
        y, rstd = _layer.gated_norm(x, weight, gate, activation=activation, eps=eps, want_rstd=True)
        ctx.activation = activation
        ctx.save_for_backward(x, weight, gate, rstd)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, gate, rstd = ctx.saved_tensors
        dx, dgate, dweight = _layer.gated_norm_bwd(x, weight, gate, _rows(dy), rstd, activation=ctx.activation)
        return dx, dweight, dgate, None, None


def gated_norm(x, weight, gate=None, activation=_layer.SILU, eps=1e-6):
    """Differentiable flare_gated_norm (layer.gated_norm): gradients flow to x,
    weight and gate."""
    return GatedNormFunction.apply(x, weight, gate, int(activation), float(eps))


class ResidualNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, w_pre, w_post, gate, scale, activation, eps):
        x, gate, residual = _rows(x), _rows(gate), residual.contiguous()
        w_pre, w_post, scale = (None if w is None else w.contiguous() for w in (w_pre, w_post, scale))
        h, y, rstd = _layer.residual_norm(x, residual, w_pre, w_post=w_post, gate=gate, scale=scale,
                                          activation=activation, eps=eps, want_rstd=True)
        ctx.activation = activation
        ctx.save_for_backward(x, residual, w_pre, w_post, gate, scale, rstd)
        ctx.set_materialize_grads(False)
        return h, y

    @staticmethod
    @once_differentiable
    def backward(ctx, dh, dy):
        x, residual, w_pre, w_post, gate, scale, rstd = ctx.saved_tensors
        dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else dy.contiguous()
        dh = None if dh is None else dh.contiguous()  # h is not used further: nothing is read for it
        g = _layer.residual_norm_bwd(x, residual, w_pre, dy, dh, rstd, w_post=w_post, gate=gate, scale=scale,
                                     activation=ctx.activation)
        return g["dx"], g["dresidual"], g["dw_pre"], g["dw_post"], g["dgate"], g["dscale"], None, None


def residual_norm(x, residual, w_pre, w_post=None, gate=None, scale=None, activation=_layer.SIGMOID, eps=1e-6):
    """Differentiable flare_residual_norm (layer.residual_norm): (h, y);
    gradients flow to x, residual, gate, the weights and the scale."""
    return ResidualNormFunction.apply(x, residual, w_pre, w_post, gate, scale, int(activation), float(eps))


class RotaryFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, positions, freqs, q, k, interleaved, mscale):
        ctx.interleaved, ctx.mscale = interleaved, mscale
        ctx.save_for_backward(positions, freqs)
        q, k = _layer.rotary(positions, freqs, _rows(q), _rows(k), interleaved=interleaved, mscale=mscale)
        return (q,) if k is None else (q, k)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk=None):
        positions, freqs = ctx.saved_tensors
        # the channels that pass through are not scaled, and neither are their gradients
        dq, dk = _layer.rotary(positions, freqs, _rows(dq), _rows(dk), interleaved=ctx.interleaved,
                               mscale=ctx.mscale, inverse=True)
        return None, None, dq, dk, None, None


def rotary(positions, freqs, q, k=None, interleaved=False, mscale=1.0):
    """Differentiable flare_rotary (layer.rotary): (q, k) turned (k None without
    one); gradients flow to q and k."""
    out = RotaryFunction.apply(positions, freqs, q, k, bool(interleaved), float(mscale))
    return out if k is not None else (out[0], None)


class QkNormRotaryFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, positions, freqs, q, k, q_weight, k_weight, eps, interleaved, mscale):
        q, k = _rows(q), _rows(k)
        q_weight, k_weight = (None if w is None else w.contiguous() for w in (q_weight, k_weight))
        ctx.eps, ctx.interleaved, ctx.mscale = eps, interleaved, mscale
        ctx.save_for_backward(positions, freqs, q, k, q_weight, k_weight)
        y, z = _layer.qk_norm_rotary(positions, freqs, q, k, q_weight=q_weight, k_weight=k_weight, eps=eps,
                                     interleaved=interleaved, mscale=mscale)
        return (y,) if k is None else (y, z)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk=None):
        positions, freqs, q, k, q_weight, k_weight = ctx.saved_tensors
        g = _layer.qk_norm_rotary_bwd(positions, freqs, q, k, _rows(dq), _rows(dk), q_weight=q_weight, k_weight=k_weight,
                                      eps=ctx.eps, interleaved=ctx.interleaved, mscale=ctx.mscale)
        return None, None, g["dq"], g["dk"], g["dq_weight"], g["dk_weight"], None, None, None


def qk_norm_rotary(positions, freqs, q, k=None, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, mscale=1.0):
    """Differentiable flare_qk_norm_rotary (layer.qk_norm_rotary): (q, k) normed
    and turned (k None without one); gradients flow to q, k and the weights."""
    out = QkNormRotaryFunction.apply(positions, freqs, q, k, q_weight, k_weight, float(eps), bool(interleaved),
                                     float(mscale))
    return out if k is not None else (out[0], None)
