"""Drop-in torch layer over the C ABI: the shared parameters w[D', C', T] are the
only state, exactly as in an unrolled ("naive") EQ-Linear layer, so an existing
weight can be used as is ("Implementacao" in "Resumo Tecnico: Flash EQ-Linear":
training-free, plug-and-play replacement).

Forward packs the half spectrum of w and runs eqlinear_fwd; backward runs
eqlinear_bwd_x on the conjugate-transposed packing and eqlinear_bwd_w.  When the weight
needs a gradient, the three passes are the training entry points instead
(eqlinear_fwd_train, eqlinear_bwd_x_train, eqlinear_bwd_w_train): the forward keeps the
weight-gradient workspace, holding x's half spectrum, alive until the backward.  EQLinearP4M is the
layer over p4m's point group (rotations and reflections), run through the same kernels on
the C_4 view described in include/eqlinear.h.  With a bias,
GELU or a residual, the forward is eqlinear_fwd_fused (eqlinear_fwd_fused_train when the
weight needs a gradient) and the backward starts with eqlinear_fused_epilogue_bwd.  EQLayerNorm is the
equivariant layer norm, and EQMLPBlock the pre-norm MLP block built from both, which by default
keeps its activations for the backward in 8 bits (include/eqlinear_block.h).  EQRMSNorm is the RMS norm with
the residual's addition (include/eqlinear_rmsnorm.h).  EQLinear8bit and EQMLPBlock8bit are the inference forms of a
layer and of a block in 8-bit integers (include/eqlinear_q8.h).  Torch only allocates the buffers; every arithmetic step
runs in the HIP library.  The backward passes have no derivative of their own: asking for gradients
of gradients raises.
"""
from __future__ import annotations

import contextlib
import functools
import math

import torch
from torch.autograd.function import once_differentiable

from . import (EQL_ACT_GELU, EQL_ACT_NONE, EQL_PACK_BWDX, EQL_PACK_FWD, eqlinear_bwd_w,
               eqlinear_bwd_w_ckpt8, eqlinear_bwd_w_train, eqlinear_bwd_w_workspace_bytes, eqlinear_bwd_x,
               eqlinear_bwd_x_train, eqlinear_ckpt8_bytes, eqlinear_ckpt8_pack, eqlinear_ckpt8_spectrum,
               eqlinear_fused_epilogue_bwd, eqlinear_fused_epilogue_bwd_ckpt8, eqlinear_fwd_fused_train,
               eqlinear_fwd_train, eqlinear_fused_epilogue_bwd_workspace_bytes, eqlinear_fwd, eqlinear_fwd_fused,
               eqlinear_layernorm_bwd, eqlinear_layernorm_bwd_ckpt8, eqlinear_layernorm_bwd_workspace_bytes,
               eqlinear_layernorm_fwd,
               eqlinear_p4m_expand_weight, eqlinear_p4m_fold_weight_grad, eqlinear_pack_weight,
               eqlinear_packed_weight_bytes, eqlinear_q8_fwd, eqlinear_q8_pack_weight, eqlinear_q8_quantize,
               eqlinear_q8_rmsnorm, eqlinear_q8_rows_bytes, eqlinear_q8_weight_bytes, eqlinear_rmsnorm_bwd,
               eqlinear_rmsnorm_bwd_workspace_bytes, eqlinear_rmsnorm_fwd)


_HERE = contextlib.nullcontext()


def _on_device(t: torch.Tensor):
    """Where a launch on t's data belongs: its own device, if that is not the current one."""
    return torch.cuda.device(t.device) if t.is_cuda and t.device.index != torch.cuda.current_device() else _HERE


def _on_its_device(run):
    """A forward or backward pass whose launches go to its first tensor's device and that device's current stream."""
    @functools.wraps(run)
    def there(ctx, *args):
        t = next((v for v in args if v is not None), None)
        with _HERE if t is None else _on_device(t):
            return run(ctx, *args)
    return there


def _dense(t: torch.Tensor) -> torch.Tensor:
    """t, contiguous and on a 16-byte boundary (a slice of a larger tensor may start off one)."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _rows(t: torch.Tensor, features: int) -> torch.Tensor:
    """t as such rows."""
    return _dense(t.reshape(-1, features))


def _packed(w: torch.Tensor, mode: int) -> torch.Tensor:
    Dp, Cp, T = w.shape
    out_ch, in_ch = (Dp, Cp) if mode == EQL_PACK_FWD else (Cp, Dp)
    buf = torch.empty(eqlinear_packed_weight_bytes(out_ch, in_ch, T, w.dtype), dtype=torch.uint8, device=w.device)
    eqlinear_pack_weight(w, buf, Dp, Cp, T, w.dtype, mode)
    return buf


class EQLinearFunction(torch.autograd.Function):
    """y[..., D'*T] = x[..., C'*T] W^T with W[d*T+g, c*T+h] = w[d, c, (g-h) mod T]."""

    @staticmethod
    @_on_its_device
    def forward(ctx, x: torch.Tensor, w: torch.Tensor, keep_spectra: bool = True):
        Dp, Cp, T = w.shape
        if x.shape[-1] != Cp * T:
            raise ValueError("x has %d features, the weight expects C'*T = %d" % (x.shape[-1], Cp * T))
        if x.dtype != w.dtype:
            raise ValueError("x and w must share a dtype (fp16 or fp32)")
        w = _dense(w)
        x2 = _rows(x, Cp * T)
        N = x2.shape[0]
        y = torch.empty((N, Dp * T), dtype=x.dtype, device=x.device)
        ws_bytes = eqlinear_bwd_w_workspace_bytes(N, Cp, Dp, T, x.dtype)
        if keep_spectra and ctx.needs_input_grad[1]:
            # The weight gradient will follow: keep x's spectrum in its workspace.
            ws = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=x.device)
            eqlinear_fwd_train(x2, _packed(w, EQL_PACK_FWD), y, ws, ws_bytes, N, Cp, Dp, T, x.dtype)
        else:
            ws = None
            eqlinear_fwd(x2, _packed(w, EQL_PACK_FWD), y, N, Cp, Dp, T, x.dtype)
        ctx.save_for_backward(x2, w, ws)
        ctx.ws_bytes = ws_bytes
        ctx.lead_shape = x.shape[:-1]
        return y.reshape(*x.shape[:-1], Dp * T)

    @staticmethod
    @once_differentiable
    @_on_its_device
    def backward(ctx, dy: torch.Tensor):
        x2, w, ws = ctx.saved_tensors
        Dp, Cp, T = w.shape
        N = x2.shape[0]
        dy2 = _rows(dy.to(x2.dtype), Dp * T)
        dx = dw = None
        need_dx, need_dw = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        train = ws is not None
        if need_dx:
            dx = torch.empty((N, Cp * T), dtype=x2.dtype, device=x2.device)
            if train and need_dw:  # also leaves dy's spectrum where the weight gradient reads it
                eqlinear_bwd_x_train(dy2, _packed(w, EQL_PACK_BWDX), dx, ws, ctx.ws_bytes, N, Cp, Dp, T, x2.dtype)
            else:
                eqlinear_bwd_x(dy2, _packed(w, EQL_PACK_BWDX), dx, N, Cp, Dp, T, x2.dtype)
            dx = dx.reshape(*ctx.lead_shape, Cp * T)
        if need_dw:
            dw = torch.empty_like(w)
            if train and need_dx:
                eqlinear_bwd_w_train(dy2, dw, ws, ctx.ws_bytes, N, Cp, Dp, T, x2.dtype)
            else:
                if ws is None:
                    ws = torch.empty(max(ctx.ws_bytes, 16), dtype=torch.uint8, device=x2.device)
                eqlinear_bwd_w(x2, dy2, dw, ws, ctx.ws_bytes, N, Cp, Dp, T, x2.dtype)
        return dx, dw, None


def eqlinear(x: torch.Tensor, w: torch.Tensor, keep_spectra: bool = True) -> torch.Tensor:
    """keep_spectra: with a weight gradient, run the training entry points (the forward keeps
    the weight-gradient workspace, about the size of x and dy plus fp32 partials, until the
    backward); False runs the plain passes and keeps only x."""
    return EQLinearFunction.apply(x, w, keep_spectra)


def _act_code(act):
    if act in (None, "none"):
        return EQL_ACT_NONE
    if act == "gelu":
        return EQL_ACT_GELU
    raise ValueError("activation must be None, 'none' or 'gelu'")


class EQLinearFusedFunction(torch.autograd.Function):
    """y = act(x W^T + b) + r: b[D'] shared by the T group elements of each output
    channel, act none or GELU, r a residual of the output's shape (each optional).

    Forward: one eqlinear_fwd_fused launch, which also keeps the activation's input
    when a gradient will be needed.  Backward: eqlinear_fused_epilogue_bwd (dpre and
    the bias gradient; without an activation dpre is dy itself), then eqlinear_bwd_x
    and eqlinear_bwd_w on dpre; the residual's gradient is dy."""

    @staticmethod
    @_on_its_device
    def forward(ctx, x: torch.Tensor, w: torch.Tensor, b, r, act, grad_mode: bool, keep_spectra: bool = True):
        Dp, Cp, T = w.shape
        if x.shape[-1] != Cp * T:
            raise ValueError("x has %d features, the weight expects C'*T = %d" % (x.shape[-1], Cp * T))
        if x.dtype != w.dtype or (b is not None and b.dtype != x.dtype) or (r is not None and r.dtype != x.dtype):
            raise ValueError("x, w, bias and residual must share a dtype (fp16 or fp32)")
        code = _act_code(act)
        # The kernel reads exactly D' bias values (one per output channel, shared by its
        # T group elements): a per-feature bias of D'*T values, or a short one, is refused.
        if b is not None and (b.dim() != 1 or b.numel() != Dp):
            raise ValueError("bias must be 1-D with D' = %d values (one per output channel, shared over the "
                             "group), got shape %s" % (Dp, tuple(b.shape)))
        if b is not None and b.device != x.device:
            raise ValueError("bias must be on x's device (%s), got %s" % (x.device, b.device))
        if r is not None and r.device != x.device:
            raise ValueError("residual must be on x's device (%s), got %s" % (x.device, r.device))
        w = _dense(w)
        x2 = _rows(x, Cp * T)
        N = x2.shape[0]
        if r is not None and r.numel() != N * Dp * T:
            raise ValueError("residual must have the output's shape")
        r2 = _rows(r, Dp * T) if r is not None else None
        y = torch.empty((N, Dp * T), dtype=x.dtype, device=x.device)
        # grad_mode is the caller's grad mode (autograd runs this body with grad disabled):
        # pre is kept only when a backward can follow.
        keep = code == EQL_ACT_GELU and grad_mode and any(ctx.needs_input_grad[:3])
        pre = torch.empty_like(y) if keep else None
        bc = b.contiguous() if b is not None else None
        ws_bytes = eqlinear_bwd_w_workspace_bytes(N, Cp, Dp, T, x.dtype)
        if keep_spectra and grad_mode and ctx.needs_input_grad[1]:
            # The weight gradient will follow: keep x's spectrum in its workspace.
            wsw = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=x.device)
            eqlinear_fwd_fused_train(x2, _packed(w, EQL_PACK_FWD), bc, r2, y, pre, wsw, ws_bytes, N, Cp, Dp, T,
                                     x.dtype, code)
        else:
            wsw = None
            eqlinear_fwd_fused(x2, _packed(w, EQL_PACK_FWD), bc, r2, y, pre, N, Cp, Dp, T, x.dtype, code)
        ctx.save_for_backward(x2, w, pre, wsw)
        ctx.ws_bytes = ws_bytes
        ctx.code, ctx.has_bias, ctx.lead_shape = code, b is not None, x.shape[:-1]
        ctx.res_shape = r.shape if r is not None else None
        return y.reshape(*x.shape[:-1], Dp * T)

    @staticmethod
    @once_differentiable
    @_on_its_device
    def backward(ctx, dy: torch.Tensor):
        x2, w, pre, wsw = ctx.saved_tensors
        Dp, Cp, T = w.shape
        N = x2.shape[0]
        dy2 = _rows(dy.to(x2.dtype), Dp * T)
        dr = dy2.reshape(ctx.res_shape) if ctx.res_shape is not None and ctx.needs_input_grad[3] else None
        dx = dw = db = None
        if not any(ctx.needs_input_grad[:3]):
            return dx, dw, db, dr, None, None, None
        # Without an activation dpre = dy: the call then only sums the bias gradient.
        dpre = torch.empty_like(dy2) if ctx.code == EQL_ACT_GELU else dy2
        if ctx.has_bias and ctx.needs_input_grad[2]:
            db = torch.empty(Dp, dtype=x2.dtype, device=x2.device)
        if ctx.code == EQL_ACT_GELU or db is not None:
            ws_bytes = eqlinear_fused_epilogue_bwd_workspace_bytes(N, Dp, T, x2.dtype)
            ws = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=x2.device)
            eqlinear_fused_epilogue_bwd(dy2, pre, dpre, db, ws, ws_bytes, N, Dp, T, x2.dtype, ctx.code)
        # With a weight gradient the training entry points run on dpre: the input gradient
        # leaves dpre's spectrum beside x's (from the forward) in the workspace.
        train = wsw is not None and ctx.needs_input_grad[1]
        if ctx.needs_input_grad[0]:
            dx = torch.empty((N, Cp * T), dtype=x2.dtype, device=x2.device)
            if train:
                eqlinear_bwd_x_train(dpre, _packed(w, EQL_PACK_BWDX), dx, wsw, ctx.ws_bytes, N, Cp, Dp, T, x2.dtype)
            else:
                eqlinear_bwd_x(dpre, _packed(w, EQL_PACK_BWDX), dx, N, Cp, Dp, T, x2.dtype)
            dx = dx.reshape(*ctx.lead_shape, Cp * T)
        if ctx.needs_input_grad[1]:
            dw = torch.empty_like(w)
            if train and ctx.needs_input_grad[0]:
                eqlinear_bwd_w_train(dpre, dw, wsw, ctx.ws_bytes, N, Cp, Dp, T, x2.dtype)
            else:
                wsb = wsw if wsw is not None else torch.empty(max(ctx.ws_bytes, 16), dtype=torch.uint8,
                                                              device=x2.device)
                eqlinear_bwd_w(x2, dpre, dw, wsb, ctx.ws_bytes, N, Cp, Dp, T, x2.dtype)
        return dx, dw, db, dr, None, None, None


def eqlinear_fused(x: torch.Tensor, w: torch.Tensor, bias: torch.Tensor | None = None,
                   residual: torch.Tensor | None = None, act: str = "none", keep_spectra: bool = True) -> torch.Tensor:
    """act(x W^T + bias) + residual with the epilogue fused into the forward kernel
    (eqlinear_fwd_fused), the MLP-block epilogue of the networks the layer is built into
    ("Nivel de Rede").  bias has one value per output channel (shared by its T group
    elements); act is "none" or "gelu"; residual has the output's shape.  Differentiable
    in x, w, bias and residual.  keep_spectra as for eqlinear."""
    return EQLinearFusedFunction.apply(x, w, bias, residual, act, torch.is_grad_enabled(), keep_spectra)


class EQLinear(torch.nn.Module):
    """Equivariant linear layer over C_T: in_channels*T -> out_channels*T features."""

    def __init__(self, in_channels: int, out_channels: int, group_order: int = 4, bias: bool = False,
                 activation: str | None = None, device=None, dtype=None, keep_spectra: bool = True):
        super().__init__()
        self.in_channels, self.out_channels, self.group_order = in_channels, out_channels, group_order
        # Training through the training entry points holds the weight-gradient workspace
        # from the forward to the backward (see eqlinear); False trades that memory for the
        # weight gradient's own transforms.
        self.keep_spectra = keep_spectra
        _act_code(activation)
        self.activation = activation
        self.weight = torch.nn.Parameter(torch.empty(out_channels, in_channels, group_order, device=device,
                                                     dtype=dtype))
        # One bias per output channel, shared by its group elements (equivariant).
        self.bias = torch.nn.Parameter(torch.zeros(out_channels, device=device, dtype=dtype)) if bias else None
        with torch.no_grad():
            self.weight.normal_(0.0, 1.0 / math.sqrt(in_channels * group_order))

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None) -> torch.Tensor:
        """y = act(x W^T + bias) + residual (the parts not configured are skipped)."""
        if self.bias is None and self.activation in (None, "none") and residual is None:
            return EQLinearFunction.apply(x, self.weight, self.keep_spectra)
        return EQLinearFusedFunction.apply(x, self.weight, self.bias, residual, self.activation,
                                           torch.is_grad_enabled(), self.keep_spectra)

    def extra_repr(self) -> str:
        return "in_channels=%d, out_channels=%d, group_order=%d, bias=%s, activation=%s" % (
            self.in_channels, self.out_channels, self.group_order, self.bias is not None, self.activation)


class EQLinearP4MFunction(torch.autograd.Function):
    """The layer over p4m's point group (dihedral D4): y[..., D'*8] = x[..., C'*8] W^T with
    W[(d,g),(c,h)] = w[d, c, g h^-1], group axis r^0..r^3 then r^-m s (m = 0..3).  Run as the
    C_4 layer on 2C' x 2D' channels with the tied weight eqlinear_p4m_expand_weight builds;
    the weight gradient is the C_4 one folded back onto the shared parameters."""

    @staticmethod
    @_on_its_device
    def forward(ctx, x: torch.Tensor, w: torch.Tensor, keep_spectra: bool = True):
        Dp, Cp, G = w.shape
        if G != 8:
            raise ValueError("a p4m weight has 8 group elements per (out, in) pair, got %d" % G)
        if x.shape[-1] != Cp * 8:
            raise ValueError("x has %d features, the weight expects C'*8 = %d" % (x.shape[-1], Cp * 8))
        if x.dtype != w.dtype:
            raise ValueError("x and w must share a dtype (fp16 or fp32)")
        w4 = torch.empty((2 * Dp, 2 * Cp, 4), dtype=w.dtype, device=w.device)
        eqlinear_p4m_expand_weight(_dense(w), w4, Dp, Cp, w.dtype)
        x2 = _rows(x, Cp * 8)
        N = x2.shape[0]
        y = torch.empty((N, Dp * 8), dtype=x.dtype, device=x.device)
        ws_bytes = eqlinear_bwd_w_workspace_bytes(N, 2 * Cp, 2 * Dp, 4, x.dtype)
        if keep_spectra and ctx.needs_input_grad[1]:
            # As EQLinearFunction: keep x's spectrum for the weight gradient.
            ws = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=x.device)
            eqlinear_fwd_train(x2, _packed(w4, EQL_PACK_FWD), y, ws, ws_bytes, N, 2 * Cp, 2 * Dp, 4, x.dtype)
        else:
            ws = None
            eqlinear_fwd(x2, _packed(w4, EQL_PACK_FWD), y, N, 2 * Cp, 2 * Dp, 4, x.dtype)
        ctx.save_for_backward(x2, w4, ws)
        ctx.ws_bytes = ws_bytes
        ctx.lead_shape = x.shape[:-1]
        ctx.p4m_shape = (Dp, Cp)
        return y.reshape(*x.shape[:-1], Dp * 8)

    @staticmethod
    @once_differentiable
    @_on_its_device
    def backward(ctx, dy: torch.Tensor):
        x2, w4, ws = ctx.saved_tensors
        Dp, Cp = ctx.p4m_shape
        N = x2.shape[0]
        dy2 = _rows(dy.to(x2.dtype), Dp * 8)
        dx = dw = None
        need_dx, need_dw = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        train = ws is not None
        if need_dx:
            dx = torch.empty((N, Cp * 8), dtype=x2.dtype, device=x2.device)
            if train and need_dw:
                eqlinear_bwd_x_train(dy2, _packed(w4, EQL_PACK_BWDX), dx, ws, ctx.ws_bytes, N, 2 * Cp, 2 * Dp, 4,
                                     x2.dtype)
            else:
                eqlinear_bwd_x(dy2, _packed(w4, EQL_PACK_BWDX), dx, N, 2 * Cp, 2 * Dp, 4, x2.dtype)
            dx = dx.reshape(*ctx.lead_shape, Cp * 8)
        if need_dw:
            dw4 = torch.empty_like(w4)
            if train and need_dx:
                eqlinear_bwd_w_train(dy2, dw4, ws, ctx.ws_bytes, N, 2 * Cp, 2 * Dp, 4, x2.dtype)
            else:
                if ws is None:
                    ws = torch.empty(max(ctx.ws_bytes, 16), dtype=torch.uint8, device=x2.device)
                eqlinear_bwd_w(x2, dy2, dw4, ws, ctx.ws_bytes, N, 2 * Cp, 2 * Dp, 4, x2.dtype)
            dw = torch.empty((Dp, Cp, 8), dtype=x2.dtype, device=x2.device)
            eqlinear_p4m_fold_weight_grad(dw4, dw, Dp, Cp, x2.dtype)
        return dx, dw, None


def eqlinear_p4m(x: torch.Tensor, w: torch.Tensor, keep_spectra: bool = True) -> torch.Tensor:
    """keep_spectra as for eqlinear."""
    return EQLinearP4MFunction.apply(x, w, keep_spectra)


class EQLinearP4M(torch.nn.Module):
    """Equivariant linear layer over p4m's point group: in_channels*8 -> out_channels*8."""

    def __init__(self, in_channels: int, out_channels: int, device=None, dtype=None, keep_spectra: bool = True):
        super().__init__()
        self.in_channels, self.out_channels = in_channels, out_channels
        self.keep_spectra = keep_spectra
        self.weight = torch.nn.Parameter(torch.empty(out_channels, in_channels, 8, device=device, dtype=dtype))
        with torch.no_grad():
            self.weight.normal_(0.0, 1.0 / math.sqrt(in_channels * 8))

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return EQLinearP4MFunction.apply(x, self.weight, self.keep_spectra)

    def extra_repr(self) -> str:
        return "in_channels=%d, out_channels=%d, group=p4m" % (self.in_channels, self.out_channels)


class EQLayerNormFunction(torch.autograd.Function):
    """Layer norm of rows of C'*T features with one weight and bias per channel, shared by its
    T group elements (include/eqlinear_block.h).  Kept for the backward: x and the rows'
    statistics, or with ckpt8 the normalised rows in 8 bits and 1 / std."""

    @staticmethod
    @_on_its_device
    def forward(ctx, x: torch.Tensor, gamma, beta, T: int, eps: float, ckpt8: bool, grad_mode: bool):
        R = x.shape[-1]
        if T < 1 or R % T != 0:
            raise ValueError("x has %d features, not a multiple of the group order %d" % (R, T))
        Cp = R // T
        for name, p in (("weight", gamma), ("bias", beta)):
            if p is None:
                continue
            if p.dim() != 1 or p.numel() != Cp:
                raise ValueError("%s must be 1-D with C' = %d values (one per channel, shared over the group), got "
                                 "shape %s" % (name, Cp, tuple(p.shape)))
            if p.dtype != x.dtype or p.device != x.device:
                raise ValueError("x and %s must share a dtype (fp16 or fp32) and a device" % name)
        x2 = _rows(x, R)
        N = x2.shape[0]
        gamma, beta = (None if p is None else p.contiguous() for p in (gamma, beta))
        y = torch.empty_like(x2)
        train = grad_mode and any(ctx.needs_input_grad[:3])
        stat = lambda: torch.empty(N, dtype=torch.float32, device=x.device)  # noqa: E731
        rstd = stat() if train else None
        mean = stat() if train and not ckpt8 else None
        ckpt = (torch.empty(eqlinear_ckpt8_bytes(N, Cp, T), dtype=torch.uint8, device=x.device)
                if train and ckpt8 else None)
        eqlinear_layernorm_fwd(x2, gamma, beta, y, ckpt, mean, rstd, N, Cp, T, eps, x.dtype)
        ctx.save_for_backward(x2 if train and not ckpt8 else None, ckpt, mean, rstd, gamma)
        ctx.sizes, ctx.dtype, ctx.has_beta = (N, Cp, T), x.dtype, beta is not None
        return y.reshape(x.shape)

    @staticmethod
    @once_differentiable
    @_on_its_device
    def backward(ctx, dy: torch.Tensor):
        x2, ckpt, mean, rstd, gamma = ctx.saved_tensors
        N, Cp, T = ctx.sizes
        dy2 = _rows(dy.to(ctx.dtype), Cp * T)
        dx = torch.empty_like(dy2)
        param = lambda: torch.empty(Cp, dtype=ctx.dtype, device=dy2.device)  # noqa: E731
        dg = param() if gamma is not None and ctx.needs_input_grad[1] else None
        db = param() if ctx.has_beta and ctx.needs_input_grad[2] else None
        ws_bytes = eqlinear_layernorm_bwd_workspace_bytes(N, Cp, T, ctx.dtype)
        ws = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=dy2.device)
        if ckpt is None:
            eqlinear_layernorm_bwd(dy2, x2, mean, rstd, gamma, None, dx, dg, db, ws, ws_bytes, N, Cp, T, ctx.dtype)
        else:
            eqlinear_layernorm_bwd_ckpt8(dy2, ckpt, rstd, gamma, None, dx, dg, db, ws, ws_bytes, N, Cp, T, ctx.dtype)
        return dx.reshape(dy.shape) if ctx.needs_input_grad[0] else None, dg, db, None, None, None, None


def eq_layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                  group_order: int = 1, eps: float = 1e-5, ckpt8: bool = False) -> torch.Tensor:
    """Layer norm over the last axis (C'*T features), weight and bias [C'].  ckpt8: keep the
    normalised rows in 8 bits for the backward instead of x (a quarter or half of its memory;
    the gradients are then those of the rounded rows)."""
    return EQLayerNormFunction.apply(x, weight, bias, group_order, eps, ckpt8, torch.is_grad_enabled())


class EQLayerNorm(torch.nn.Module):
    """Equivariant layer norm over channels * T features: one weight and bias per channel."""

    def __init__(self, channels: int, group_order: int = 4, eps: float = 1e-5, device=None, dtype=None,
                 ckpt8: bool = False):
        super().__init__()
        self.channels, self.group_order, self.eps, self.ckpt8 = channels, group_order, eps, ckpt8
        self.weight = torch.nn.Parameter(torch.ones(channels, device=device, dtype=dtype))
        self.bias = torch.nn.Parameter(torch.zeros(channels, device=device, dtype=dtype))

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return eq_layer_norm(x, self.weight, self.bias, self.group_order, self.eps, self.ckpt8)

    def extra_repr(self) -> str:
        return "channels=%d, group_order=%d, eps=%g, ckpt8=%s" % (self.channels, self.group_order, self.eps, self.ckpt8)


class EQRMSNormFunction(torch.autograd.Function):
    """y = weight s / rms(s) of rows of C'*T features, one weight per channel, shared by its T group
    elements, for s = x + residual (include/eqlinear_rmsnorm.h).  Returns y, or (y, s) with a residual.
    Kept for the backward: s and the rows' 1 / rms."""

    @staticmethod
    @_on_its_device
    def forward(ctx, x: torch.Tensor, residual, gamma, T: int, eps: float, grad_mode: bool):
        N, Cp = _norm_operands(x, residual, gamma, T)
        R = Cp * T
        x2 = _rows(x, R)
        r2 = _rows(residual, R) if residual is not None else None
        gamma = gamma.contiguous() if gamma is not None else None
        y = torch.empty_like(x2)
        s = torch.empty_like(x2) if residual is not None else None
        train = grad_mode and any(ctx.needs_input_grad[:3])
        rstd = torch.empty(N, dtype=torch.float32, device=x.device) if train else None
        eqlinear_rmsnorm_fwd(x2, r2, gamma, s, y, rstd, N, Cp, T, eps, x.dtype)
        ctx.set_materialize_grads(False)
        ctx.sizes, ctx.dtype, ctx.shape = (N, Cp, T), x.dtype, x.shape
        if s is None:
            ctx.save_for_backward(x2 if train else None, rstd, gamma)
            return y.reshape(x.shape)
        s = s.reshape(x.shape)
        ctx.save_for_backward(s if train else None, rstd, gamma)
        return y.reshape(x.shape), s

    @staticmethod
    @once_differentiable
    @_on_its_device
    def backward(ctx, dy, ds=None):
        s, rstd, gamma = ctx.saved_tensors
        N, Cp, T = ctx.sizes
        R = Cp * T
        need_x, need_r, need_g = ctx.needs_input_grad[:3]
        if dy is None:  # only the sum was used
            if ds is None:
                return None, None, None, None, None, None
            dg = torch.zeros_like(gamma) if need_g else None
            return ds if need_x else None, ds if need_r else None, dg, None, None, None
        dy2 = _rows(dy.to(ctx.dtype), R)
        ds2 = _rows(ds.to(ctx.dtype), R) if ds is not None else None
        dx = torch.empty_like(dy2)
        dg = torch.empty(Cp, dtype=ctx.dtype, device=dy2.device) if need_g else None
        n = eqlinear_rmsnorm_bwd_workspace_bytes(N, Cp, T, ctx.dtype)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device=dy2.device)
        eqlinear_rmsnorm_bwd(dy2, _rows(s, R), rstd, gamma, ds2, dx, dg, ws, n, N, Cp, T, ctx.dtype)
        dx = dx.reshape(ctx.shape)
        return dx if need_x else None, dx if need_r else None, dg, None, None, None


def _norm_operands(x, residual, gamma, T):
    """(rows, channels) of a norm's input after the checks that its kernels rely on."""
    R = x.shape[-1]
    if T < 1 or R % T != 0:
        raise ValueError("x has %d features, not a multiple of the group order %d" % (R, T))
    Cp = R // T
    if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype or residual.device != x.device):
        raise ValueError("residual must have x's shape, dtype and device")
    if gamma is not None:
        if gamma.dim() != 1 or gamma.numel() != Cp:
            raise ValueError("weight must be 1-D with C' = %d values (one per channel, shared over the group), got "
                             "shape %s" % (Cp, tuple(gamma.shape)))
        if gamma.dtype != x.dtype or gamma.device != x.device:
            raise ValueError("x and weight must share a dtype (fp16 or fp32) and a device")
    return x.numel() // R if R else 0, Cp


def eq_rms_norm(x: torch.Tensor, weight: torch.Tensor | None = None, group_order: int = 1, eps: float = 1e-6,
                residual: torch.Tensor | None = None):
    """RMS norm over the last axis (C'*T features), weight [C'].  With a residual, the norm of s = x + residual
    (rounded to x's dtype): returns (y, s).  Differentiable in x, residual and weight."""
    return EQRMSNormFunction.apply(x, residual, weight, group_order, eps, torch.is_grad_enabled())


class EQRMSNorm(torch.nn.Module):
    """Equivariant RMS norm over channels * T features: one weight per channel.  Called with a residual it
    adds it first and returns (norm, sum)."""

    def __init__(self, channels: int, group_order: int = 4, eps: float = 1e-6, device=None, dtype=None):
        super().__init__()
        self.channels, self.group_order, self.eps = channels, group_order, eps
        self.weight = torch.nn.Parameter(torch.ones(channels, device=device, dtype=dtype))

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None):
        return eq_rms_norm(x, self.weight, self.group_order, self.eps, residual)

    def extra_repr(self) -> str:
        return "channels=%d, group_order=%d, eps=%g" % (self.channels, self.group_order, self.eps)


class EQMLPBlock8bitFunction(torch.autograd.Function):
    """y = x + W2 gelu(W1 norm(x) + b1) + b2 keeping, from the forward to the backward, the
    normalised rows and GELU's input as 8-bit checkpoints and nothing else of their size.

    Backward, second layer: its input is gelu of the kept values, so the checkpoint's spectrum
    takes the place of the one eqlinear_fwd_train would have kept; then GELU's own backward;
    first layer: its input is gamma h + beta; then the norm's, which adds the residual
    branch's gradient dy."""

    @staticmethod
    @_on_its_device
    def forward(ctx, x: torch.Tensor, gamma, beta, w1, b1, w2, b2, eps: float, grad_mode: bool):
        Hp, Cp, T = w1.shape
        if w2.shape != (Cp, Hp, T):
            raise ValueError("w2 must be [C', H', T] = %s for w1 [H', C', T], got %s" % ((Cp, Hp, T), tuple(w2.shape)))
        if x.shape[-1] != Cp * T:
            raise ValueError("x has %d features, the block expects C'*T = %d" % (x.shape[-1], Cp * T))
        for name, p, n in (("norm weight", gamma, Cp), ("norm bias", beta, Cp), ("b1", b1, Hp), ("b2", b2, Cp)):
            if p.dim() != 1 or p.numel() != n:
                raise ValueError("%s must be 1-D with %d values, got shape %s" % (name, n, tuple(p.shape)))
        if any(p.dtype != x.dtype or p.device != x.device for p in (gamma, beta, w1, b1, w2, b2)):
            raise ValueError("x and the block's parameters must share a dtype (fp16 or fp32) and a device")
        x2 = _rows(x, Cp * T)
        gamma, beta, b1, b2 = (p.contiguous() for p in (gamma, beta, b1, b2))
        w1, w2 = _dense(w1), _dense(w2)
        N, dt, dev = x2.shape[0], x.dtype, x.device
        train = grad_mode and any(ctx.needs_input_grad[:7])
        bytes8 = lambda c: torch.empty(eqlinear_ckpt8_bytes(N, c, T), dtype=torch.uint8, device=dev)  # noqa: E731
        h8 = bytes8(Cp) if train else None
        pre8 = bytes8(Hp) if train else None
        rstd = torch.empty(N, dtype=torch.float32, device=dev) if train else None
        u, y = torch.empty_like(x2), torch.empty_like(x2)
        a = torch.empty((N, Hp * T), dtype=dt, device=dev)
        pre = torch.empty_like(a) if train else None
        eqlinear_layernorm_fwd(x2, gamma, beta, u, h8, None, rstd, N, Cp, T, eps, dt)
        eqlinear_fwd_fused(u, _packed(w1, EQL_PACK_FWD), b1, None, a, pre, N, Cp, Hp, T, dt, EQL_ACT_GELU)
        if train:
            eqlinear_ckpt8_pack(pre, pre8, N, Hp, T, dt)
        eqlinear_fwd_fused(a, _packed(w2, EQL_PACK_FWD), b2, x2, y, None, N, Hp, Cp, T, dt, EQL_ACT_NONE)
        ctx.save_for_backward(h8, rstd, pre8, gamma, beta, w1, w2)
        ctx.rows = N
        return y.reshape(x.shape)

    @staticmethod
    @once_differentiable
    @_on_its_device
    def backward(ctx, dy: torch.Tensor):
        h8, rstd, pre8, gamma, beta, w1, w2 = ctx.saved_tensors
        Hp, Cp, T = w1.shape
        N, dt, dev = ctx.rows, w1.dtype, w1.device
        need = ctx.needs_input_grad
        empty = lambda *s: torch.empty(s, dtype=dt, device=dev)  # noqa: E731
        scratch = lambda n: torch.empty(max(n, 16), dtype=torch.uint8, device=dev)  # noqa: E731
        dy2 = _rows(dy.to(dt), Cp * T)

        def layer(g, w, ckpt, scale, shift, act, out, inp, need_w, need_x):
            """Input and weight gradient of one layer (inp -> out channels) for output gradient g.  At
            p4 fp16 the input gradient's kernel can leave g's spectrum for the weight gradient; elsewhere
            that would be a launch of its own, which eqlinear_bwd_w_ckpt8 shares with the checkpoint's (and
            with 32 MiB more, returned to the allocator after the call, it splits small layers further)."""
            dx = empty(N, inp * T) if need_x else None
            dw = torch.empty_like(w) if need_w else None
            n = eqlinear_bwd_w_workspace_bytes(N, inp, out, T, dt)
            if need_w and need_x and T == 4 and dt == torch.float16:
                ws = scratch(n)
                eqlinear_ckpt8_spectrum(ckpt, scale, shift, act, ws, n, N, inp, out, T, dt)
                eqlinear_bwd_x_train(g, _packed(w, EQL_PACK_BWDX), dx, ws, n, N, inp, out, T, dt)
                eqlinear_bwd_w_train(g, dw, ws, n, N, inp, out, T, dt)
                return dx, dw
            if need_x:
                eqlinear_bwd_x(g, _packed(w, EQL_PACK_BWDX), dx, N, inp, out, T, dt)
            if need_w:
                n += 32 << 20
                eqlinear_bwd_w_ckpt8(ckpt, scale, shift, act, g, dw, scratch(n), n, N, inp, out, T, dt)
            return dx, dw

        db2 = empty(Cp) if need[6] else None
        if db2 is not None:
            n = eqlinear_fused_epilogue_bwd_workspace_bytes(N, Cp, T, dt)
            eqlinear_fused_epilogue_bwd(dy2, None, dy2, db2, scratch(n), n, N, Cp, T, dt, EQL_ACT_NONE)
        below1, below = any(need[:4]), any(need[:3])  # gradients under the first layer's output, and under its input
        dh, dw2 = layer(dy2, w2, pre8, None, None, EQL_ACT_GELU, Cp, Hp, need[5], below1 or need[4])
        db1 = empty(Hp) if need[4] else None
        dw1 = dx = dgamma = dbeta = None
        if dh is not None:
            n = eqlinear_fused_epilogue_bwd_workspace_bytes(N, Hp, T, dt)
            eqlinear_fused_epilogue_bwd_ckpt8(dh, pre8, dh, db1, scratch(n), n, N, Hp, T, dt)
            du, dw1 = layer(dh, w1, h8, gamma, beta, EQL_ACT_NONE, Hp, Cp, need[3], below)
            if below:
                dgamma, dbeta = (empty(Cp) if k else None for k in need[1:3])
                n = eqlinear_layernorm_bwd_workspace_bytes(N, Cp, T, dt)
                eqlinear_layernorm_bwd_ckpt8(du, h8, rstd, gamma, dy2, du, dgamma, dbeta, scratch(n), n, N, Cp, T, dt)
                dx = du.reshape(dy.shape) if need[0] else None
        return dx, dgamma, dbeta, dw1, db1, dw2, db2, None, None


def _as_made(m, cls) -> bool:
    """Calling m is cls.forward and nothing else: no subclass's or instance's forward, no hooks."""
    return (isinstance(m, cls) and getattr(m.forward, "__func__", None) is cls.forward
            and not (m._forward_hooks or m._forward_pre_hooks or m._backward_hooks or m._backward_pre_hooks))


class EQMLPBlock(torch.nn.Module):
    """Pre-norm transformer MLP block, x + W2 gelu(W1 norm(x) + b1) + b2, over C_T: channels*T ->
    hidden_channels*T -> channels*T features.

    ckpt8 (the default) keeps the normalised rows and GELU's input in 8 bits for the backward:
    about C' + H' bytes per group element and row, against 2 C' + 4 H' in fp16 (4 C' + 8 H' in
    fp32) and as much again for the kept spectra when it is off; the gradients are those of the
    rounded activations (each within 1/127 of its block's largest).  The block then reads its
    submodules' parameters; where a submodule was replaced, hooked or set to compute something else,
    it calls them one after the other, as without ckpt8.  norm: "layer", or "rms" for EQRMSNorm (whose
    block keeps its activations as they are, as without ckpt8)."""

    def __init__(self, channels: int, hidden_channels: int, group_order: int = 4, eps: float = 1e-5, device=None,
                 dtype=None, ckpt8: bool = True, norm: str = "layer"):
        super().__init__()
        if norm not in ("layer", "rms"):
            raise ValueError("norm must be 'layer' or 'rms'")
        self.ckpt8 = ckpt8 and norm == "layer"
        self.norm = (EQLayerNorm if norm == "layer" else EQRMSNorm)(channels, group_order, eps, device=device, dtype=dtype)
        self.fc1 = EQLinear(channels, hidden_channels, group_order, bias=True, activation="gelu", device=device, dtype=dtype)
        self.fc2 = EQLinear(hidden_channels, channels, group_order, bias=True, device=device, dtype=dtype)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        n, a, b = self.norm, self.fc1, self.fc2
        if self.ckpt8 and self._as_made():
            return EQMLPBlock8bitFunction.apply(x, n.weight, n.bias, a.weight, a.bias, b.weight, b.bias, n.eps,
                                                torch.is_grad_enabled())
        return b(a(n(x)), residual=x)

    def _as_made(self) -> bool:
        """The submodules compute norm, gelu(W1 . + b1) and W2 . + b2, and nothing runs around them."""
        n, a, b = self.norm, self.fc1, self.fc2
        return (_as_made(n, EQLayerNorm) and _as_made(a, EQLinear) and _as_made(b, EQLinear)
                and a.activation == "gelu" and b.activation in (None, "none")
                and all(p is not None for p in (n.weight, n.bias, a.bias, b.bias)) and n.group_order == a.weight.shape[2]
                and not torch.nn.modules.module._has_any_global_hook())

    def extra_repr(self) -> str:
        return "ckpt8=%s" % self.ckpt8


class EQRows8:
    """Rows in 8 bits: what eqlinear_q8_quantize and eqlinear_q8_rmsnorm write, with the sizes to read it by."""

    __slots__ = ("data", "lead_shape", "channels", "group_order", "dtype")

    def __init__(self, data: torch.Tensor, lead_shape, channels: int, group_order: int, dtype: torch.dtype):
        self.data, self.lead_shape, self.channels, self.group_order, self.dtype = data, lead_shape, channels, group_order, dtype


def _inference(*tensors) -> None:
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        raise RuntimeError("the 8-bit layers are inference forms without a backward pass: call them under "
                           "torch.no_grad() or on tensors that need no gradient")


class _NoBackward(torch.autograd.Function):
    """y, computed from parameters that need gradients by something without a backward pass: asking for them raises."""

    @staticmethod
    def forward(ctx, y, *params):
        return y.detach()  # no view of y to autograd, which would refuse to have it changed in place

    @staticmethod
    def backward(ctx, dy):
        raise RuntimeError("the 8-bit block is an inference form without a backward pass, and its norm has parameters that "
                           "need a gradient: call it under torch.no_grad(), or freeze them with requires_grad_(False)")


def eq_quantize_8bit(x: torch.Tensor, group_order: int = 1) -> EQRows8:
    """x [..., C'*T] as 8-bit rows (a scale for each row and frequency)."""
    _inference(x)
    N, Cp = _norm_operands(x, None, None, group_order)
    data = torch.empty(max(eqlinear_q8_rows_bytes(N, Cp, group_order), 16), dtype=torch.uint8, device=x.device)
    with _on_device(x):
        eqlinear_q8_quantize(_rows(x, x.shape[-1]), data, N, Cp, group_order, x.dtype)
    return EQRows8(data, x.shape[:-1], Cp, group_order, x.dtype)


def eq_rms_norm_8bit(x: torch.Tensor, weight: torch.Tensor | None = None, group_order: int = 1, eps: float = 1e-6,
                     residual: torch.Tensor | None = None):
    """eq_rms_norm with its output as 8-bit rows: returns them, or (rows, x + residual)."""
    _inference(x, weight, residual)
    N, Cp = _norm_operands(x, residual, weight, group_order)
    R = x.shape[-1]
    data = torch.empty(max(eqlinear_q8_rows_bytes(N, Cp, group_order), 16), dtype=torch.uint8, device=x.device)
    s = torch.empty((N, R), dtype=x.dtype, device=x.device) if residual is not None else None
    with _on_device(x):
        eqlinear_q8_rmsnorm(_rows(x, R), _rows(residual, R) if residual is not None else None,
                            weight.contiguous() if weight is not None else None, s, data, N, Cp, group_order, eps, x.dtype)
    rows = EQRows8(data, x.shape[:-1], Cp, group_order, x.dtype)
    return rows if s is None else (rows, s.reshape(x.shape))


def _convertible(m, classes) -> None:
    """Refuses a module whose call is more than its class's formula: only that goes into the 8-bit form."""
    cls = next((c for c in classes if isinstance(m, c)), None)
    if cls is None:
        raise TypeError("expected an %s, got %s" % (" or an ".join(c.__name__ for c in classes), type(m).__name__))
    if not _as_made(m, cls):
        raise ValueError("the 8-bit form of this %s would leave out its hooks or its own forward" % type(m).__name__)


class EQLinear8bit(torch.nn.Module):
    """Inference form of EQLinear in 8-bit integers: the weight's half spectrum with a scale for each output
    channel and frequency, packed once; activations quantised as they come, or given as EQRows8.  Made by
    from_float, from an EQLinear or an EQLinearP4M (as the layer over C_4 on twice the channels that it runs as)
    without hooks or a forward of its own.
    Its outputs are those of the rounded layer, about 1% of their norm off the exact one."""

    def __init__(self, in_channels: int, out_channels: int, group_order: int, bias: bool = False,
                 activation: str | None = None, device=None, dtype=None):
        super().__init__()
        _act_code(activation)
        self.in_channels, self.out_channels, self.group_order = in_channels, out_channels, group_order
        self.activation = activation
        n = eqlinear_q8_weight_bytes(out_channels, in_channels, group_order)
        if n == 0:
            raise ValueError("no 8-bit weight of %d x %d channels over C_%d" % (out_channels, in_channels, group_order))
        # Zeros: a layer of zero weights until a weight is packed or loaded.
        self.register_buffer("weight8", torch.zeros(n, dtype=torch.uint8, device=device))
        self.register_buffer("bias", torch.zeros(out_channels, device=device, dtype=dtype) if bias else None)

    @classmethod
    @torch.no_grad()
    def from_float(cls, layer: torch.nn.Module) -> "EQLinear8bit":
        _convertible(layer, (EQLinear, EQLinearP4M))
        w, bias, act = layer.weight.detach(), getattr(layer, "bias", None), getattr(layer, "activation", None)
        if isinstance(layer, EQLinearP4M):
            Dp, Cp, _ = w.shape
            w4 = torch.empty((2 * Dp, 2 * Cp, 4), dtype=w.dtype, device=w.device)
            with _on_device(w):
                eqlinear_p4m_expand_weight(_dense(w), w4, Dp, Cp, w.dtype)
            w = w4
        Dp, Cp, T = w.shape
        made = cls(Cp, Dp, T, bias is not None, act, device=w.device, dtype=w.dtype)
        made.pack(w)
        if bias is not None:
            made.bias.copy_(bias)
        return made

    # The packed weight's size is no sign of its sizes (whole tiles of channels): a state holds them beside it.
    def _save_to_state_dict(self, destination, prefix, keep_vars):
        super()._save_to_state_dict(destination, prefix, keep_vars)
        destination[prefix + "sizes"] = torch.tensor([self.out_channels, self.in_channels, self.group_order])

    def _load_from_state_dict(self, state_dict, prefix, local_metadata, strict, missing_keys, unexpected_keys, error_msgs):
        key, own = prefix + "sizes", [self.out_channels, self.in_channels, self.group_order]
        sizes = state_dict[key].tolist() if key in state_dict else own
        if sizes != own:
            error_msgs.append("%sweight8 is of [output channels, input channels, group order] = %s, the layer of %s" % (
                prefix, sizes, own))
            return
        super()._load_from_state_dict(state_dict, prefix, local_metadata, strict, missing_keys, unexpected_keys, error_msgs)
        if key in unexpected_keys:
            unexpected_keys.remove(key)

    @torch.no_grad()
    def pack(self, w: torch.Tensor) -> None:
        """Packs a weight [D', C', T]."""
        if tuple(w.shape) != (self.out_channels, self.in_channels, self.group_order):
            raise ValueError("expected a weight of shape %s, got %s" % (
                (self.out_channels, self.in_channels, self.group_order), tuple(w.shape)))
        if w.device != self.weight8.device:
            raise ValueError("the weight must be on the layer's device (%s), got %s" % (self.weight8.device, w.device))
        with _on_device(w):
            eqlinear_q8_pack_weight(_dense(w), self.weight8, self.out_channels, self.in_channels, self.group_order, w.dtype)

    def forward(self, x, residual: torch.Tensor | None = None) -> torch.Tensor:
        """y = act(x W^T + bias) + residual; x: a tensor [..., C'*T] or EQRows8."""
        Dp, Cp, T = self.out_channels, self.in_channels, self.group_order
        _inference(residual)
        if not isinstance(x, EQRows8):
            if x.shape[-1] != Cp * T:
                raise ValueError("x has %d features, the weight expects C'*T = %d" % (x.shape[-1], Cp * T))
            if x.device != self.weight8.device:
                raise ValueError("x must be on the layer's device (%s), got %s" % (self.weight8.device, x.device))
            x = eq_quantize_8bit(x, T)
        if (x.channels, x.group_order) != (Cp, T) or x.data.device != self.weight8.device:
            raise ValueError("the rows have %d channels over C_%d on %s, the layer %d over C_%d on %s" % (
                x.channels, x.group_order, x.data.device, Cp, T, self.weight8.device))
        shape = (*x.lead_shape, Dp * T)
        if self.bias is not None and self.bias.dtype != x.dtype:
            raise ValueError("x and bias must share a dtype (fp16 or fp32)")
        if residual is not None and (residual.shape != shape or residual.dtype != x.dtype or residual.device != x.data.device):
            raise ValueError("residual must have the output's shape, dtype and device")
        N = math.prod(x.lead_shape)
        y = torch.empty((N, Dp * T), dtype=x.dtype, device=x.data.device)
        with _on_device(y):
            eqlinear_q8_fwd(x.data, self.weight8, self.bias, _rows(residual, Dp * T) if residual is not None else None, y,
                            N, Cp, Dp, T, x.dtype, _act_code(self.activation))
        return y.reshape(shape)

    def extra_repr(self) -> str:
        return "in_channels=%d, out_channels=%d, group_order=%d, bias=%s, activation=%s" % (
            self.in_channels, self.out_channels, self.group_order, self.bias is not None, self.activation)


class EQMLPBlock8bit(torch.nn.Module):
    """Inference form of EQMLPBlock with its two layers in 8-bit integers (of a block whose call, and its layers', is
    as it is made: no hooks, no forward of its own).  With an RMS norm, the norm writes the first layer's 8-bit rows
    itself; called with a residual (RMS norm only), the block is of x + residual, added in the norm's pass.  While
    the norm's parameters need gradients, a backward pass through the output raises."""

    def __init__(self, norm: torch.nn.Module, fc1: EQLinear8bit, fc2: EQLinear8bit):
        super().__init__()
        self.norm, self.fc1, self.fc2 = norm, fc1, fc2

    @classmethod
    def from_float(cls, block: EQMLPBlock) -> "EQMLPBlock8bit":
        """The norm is the block's own; the layers are packed anew."""
        _convertible(block, (EQMLPBlock,))
        for m in (block.fc1, block.fc2):
            _convertible(m, (EQLinear, EQLinearP4M))
        return cls(block.norm, EQLinear8bit.from_float(block.fc1), EQLinear8bit.from_float(block.fc2))

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None) -> torch.Tensor:
        _inference(x, residual)
        with torch.no_grad():
            y = self._forward(x, residual)
        trained = [p for p in self.parameters() if p.requires_grad] if torch.is_grad_enabled() else []
        return _NoBackward.apply(y, *trained) if trained else y

    def _forward(self, x: torch.Tensor, residual) -> torch.Tensor:
        n = self.norm
        if _as_made(n, EQRMSNorm) and not torch.nn.modules.module._has_any_global_hook():
            rows = eq_rms_norm_8bit(x, n.weight, n.group_order, n.eps, residual)
            if residual is not None:
                rows, x = rows
            return self.fc2(self.fc1(rows), residual=x)
        if residual is not None:
            if not isinstance(n, EQRMSNorm):
                raise ValueError("only a block with an RMS norm takes a residual")
            u, x = n(x, residual)
        else:
            u = n(x)
        return self.fc2(self.fc1(u), residual=x)
