"""torch.autograd wrapper of the hybrid training path ("Sparser, Faster,
Lighter Transformer Language Models", section 2.B.3; the L1 coefficient from
the news article "Sakana AI and NVIDIA TwELL boosts LLM training speed by
21.9%", recipe list).

``SparseGatedFFNFunction`` runs one activation-sparse gated FFN layer
through the C-ABI: the gate GEMM with the TwELL epilogue, the TwELL -> hybrid
conversion and the hybrid forward; its backward is the hybrid backward with
the L1 term on h.  ``SparseFFNStack`` chains layers with residual additions.
Argument marshalling only: every step runs in libtwell's kernels, on torch's
current stream, with nothing read back.

Weights may be bf16 or fp32 master copies (cast to bf16 for the kernels on
every call); their gradients come back from the library in fp32 and are
returned in the weights' own dtype, as autograd requires, so fp32 masters keep
fp32 gradients.  The activation stream x is bf16 (its gradient too).

``AddRMSNormFunction`` is the residual addition and norm in front of an FFN
(fused forward and backward), and ``Fp8LinearFunction`` a linear layer whose
three products (y, dx, dW) run on e4m3 operands with block scales.  Both refuse
to be differentiated twice.
"""
from __future__ import annotations

import torch

from . import (Hybrid, TwELL, hybrid_ffn_bwd, hybrid_ffn_bwd_tc, hybrid_ffn_fwd,
               hybrid_ffn_fwd_tc, twell_gate_pack, twell_gemm_fp8, twell_quant_fp8,
               twell_rms_norm, twell_rms_norm_bwd, twell_to_hybrid)


def _rows(g):
    """A gradient as the kernels read it: autograd may hand over an expanded or
    a transposed one."""
    return g if g.stride(-1) == 1 and (g.shape[0] < 2 or g.stride(0) >= g.shape[1]) \
        else g.contiguous()


class _Once(torch.autograd.Function):
    """Gradients as they are, to be differentiated no further."""

    @staticmethod
    def forward(ctx, anchor, *grads):
        return tuple(None if g is None else g.view_as(g) for g in grads)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("this function's gradient cannot be differentiated")


def _once(*grads):
    """What a backward returns.  Where it is itself being recorded (create_graph),
    a derivative of it is refused, not left out."""
    if not torch.is_grad_enabled():
        return grads
    g = next(g for g in grads if g is not None)
    return _Once.apply(torch.empty(0, device=g.device, requires_grad=True), *grads)


class AddRMSNormFunction(torch.autograd.Function):
    """(y, total): total = x + residual, y = bf16 of the norm of total times
    weight.  x and residual [T][D] and weight [D] are bf16 or fp32 each, total has
    residual's type.  Without a residual total is x and only y is returned."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        o = twell_rms_norm(x, weight, residual=residual, eps=eps, rstd=True)
        total = x if residual is None else o.total
        ctx.save_for_backward(total, weight, o.rstd)
        ctx.types = (x.dtype, weight.dtype)
        ctx.added = residual is not None
        return (o.y, total) if ctx.added else o.y

    @staticmethod
    def backward(ctx, dy, dtotal=None):
        total, weight, rstd = ctx.saved_tensors
        if dtotal is not None:
            dtotal = _rows(dtotal)
        dx, dw = twell_rms_norm_bwd(total, weight, rstd, _rows(dy), dtotal=dtotal)
        return _once(dx.to(ctx.types[0]), dw.to(ctx.types[1]), dx if ctx.added else None, None)


class Fp8LinearFunction(torch.autograd.Function):
    """y [T][N] = x W^T on e4m3 operands: x [T][K] and the gradient dy in blocks of
    1 x 128 along the dimension each product sums over (so both are also quantised
    transposed, for dW), W [N][K] in blocks of 128 x 128.  x and W are bf16 or
    fp32; y has x's type, dx too, and dW is computed in fp32.  ``status``: the
    device int32 that the products OR their flags into (default:
    ``status_word()``)."""

    @staticmethod
    def forward(ctx, x, weight, status=None):
        need_x, need_w = ctx.needs_input_grad[:2]
        ctx.status = status
        qx = twell_quant_fp8(x, transposed=need_w)
        qw = twell_quant_fp8(weight, block_rows=128, transposed=need_x)
        ctx.save_for_backward(qx.qt, qx.scale_t, qw.qt, qw.scale_t)
        ctx.sizes = (x.shape, weight.shape)
        ctx.types = (x.dtype, weight.dtype)
        return twell_gemm_fp8(qx.q, qx.scale, qw.q, qw.scale, dtype=x.dtype, status=status)

    @staticmethod
    def backward(ctx, dy):
        xt, xt_scale, wt, wt_scale = ctx.saved_tensors
        need_x, need_w = ctx.needs_input_grad[:2]
        (T, K), (N, _) = ctx.sizes
        dx = dw = None
        q = twell_quant_fp8(_rows(dy), rows=need_x, transposed=need_w)
        if need_x:
            dx = twell_gemm_fp8(q.q, q.scale, wt, wt_scale, dtype=ctx.types[0],
                                status=ctx.status)
        if need_w:
            # (a sum over no rows is not a product the kernel takes)
            dw = (twell_gemm_fp8(q.qt, q.scale_t, xt, xt_scale, dtype=torch.float32,
                                 status=ctx.status) if T
                  else torch.zeros((N, K), dtype=torch.float32, device=dy.device))
            dw = dw.to(ctx.types[1])
        return _once(dx, dw, None)


class Fp8Linear(torch.nn.Module):
    """Linear layer without a bias whose products run on e4m3 operands
    (``Fp8LinearFunction``); the parameter is an fp32 master copy."""

    def __init__(self, weight):
        super().__init__()
        self.weight = torch.nn.Parameter(weight.detach().float())
        self.register_buffer("status", torch.zeros((1,), dtype=torch.int32, device=weight.device),
                             persistent=False)

    def forward(self, x):
        return Fp8LinearFunction.apply(x, self.weight, self.status)

    def status_flags(self) -> int:
        """OR of the flags of the layer's products, forward and backward, since
        ``status`` was last zeroed (synchronises)."""
        return int(self.status.item())


class SparseGatedFFNFunction(torch.autograd.Function):
    """y = (ReLU(x W_g) * (x W_u)) W_d through TwELL and the hybrid format.

    Inputs: x [T][D] bf16, Wg_t / Wu_t / Wd [F][D] bf16 or fp32; ``l1_coeff`` adds
    l1_coeff * sum(h) to the loss; ``cap`` is the ELL capacity per 128-column
    tile (rows above it in some tile go to the dense backup, at most
    ``max_dense`` of them); ``tensor_cores`` selects hybrid_ffn_*_tc.
    Returns y [T][D] fp32.  The device status words of the call (TwELL and
    hybrid) are appended to ``status_sink`` when it is a list."""

    @staticmethod
    def forward(ctx, x, Wg_t, Wu_t, Wd, l1_coeff, cap, max_dense, tensor_cores, status_sink):
        T, _ = x.shape
        F = Wg_t.shape[0]
        w16 = [w if w.dtype == torch.bfloat16 else w.to(torch.bfloat16).contiguous()
               for w in (Wg_t, Wu_t, Wd)]
        # with the TwELL width equal to the ELL capacity, a (row, tile) spills
        # only in rows that overflow to the dense backup: max_dense * n_t
        # spill slices suffice (more rows than that set TWELL_FLAG_DENSE_FULL)
        h = TwELL(T, F, cap, spill_cap=max(1, max_dense) * (F // 128), device=x.device)
        twell_gate_pack(x, w16[0], h)
        hyb = Hybrid(T, F, cap, max_dense, device=x.device)
        twell_to_hybrid(h, hyb)
        fwd = hybrid_ffn_fwd_tc if tensor_cores else hybrid_ffn_fwd
        y, u_ell, U_dense = fwd(x, hyb, w16[1], w16[2])
        ctx.save_for_backward(x, *w16, u_ell, U_dense)
        ctx.w_dtypes = (Wg_t.dtype, Wu_t.dtype, Wd.dtype)
        ctx.hyb = hyb
        ctx.l1 = float(l1_coeff)
        ctx.tc = bool(tensor_cores)
        if status_sink is not None:
            status_sink.extend([h.status, hyb.status])
        return y

    @staticmethod
    def backward(ctx, dy):
        x, Wg_t, Wu_t, Wd, u_ell, U_dense = ctx.saved_tensors
        bwd = hybrid_ffn_bwd_tc if ctx.tc else hybrid_ffn_bwd
        dx, dWg, dWu, dWd = bwd(x, ctx.hyb, u_ell, U_dense, Wg_t, Wu_t, Wd,
                                dy.float().contiguous(), ctx.l1)
        dt = ctx.w_dtypes
        return (dx.to(x.dtype), dWg.to(dt[0]), dWu.to(dt[1]), dWd.to(dt[2]),
                None, None, None, None, None)


class SparseFFNStack(torch.nn.Module):
    """L residual blocks x <- x + FFN_l(bf16(x)): the residual stream and its
    gradient stay fp32; each layer's input is the stream rounded to bf16.

    Parameters are fp32 master copies of the given weights (gradients in
    fp32); the kernels see them rounded to bf16 on every call.

    ``bias_feature``: when set, feature D - 1 of x is a constant bias input
    (the gate's threshold feature, as in the synthetic workloads) and the
    residual update leaves it unchanged, so every layer sees the same
    activation-density control.

    ``norms``: norm weights [D], one per layer, make the blocks pre-norm: each
    layer's input is the bf16 RMS norm of the stream, computed together with
    the addition of the layer before it (``AddRMSNormFunction``)."""

    def __init__(self, weights, l1_coeff=2e-5, cap=32, max_dense=1024, tensor_cores=True,
                 bias_feature=True, norms=None, eps=1e-6):
        super().__init__()
        if norms is not None and len(norms) != len(weights):
            raise ValueError("one norm weight per layer")
        self.norms = None if norms is None else torch.nn.ParameterList(
            torch.nn.Parameter(n.detach().float()) for n in norms)
        self.eps = eps
        self.Wg = torch.nn.ParameterList(torch.nn.Parameter(w[0].float()) for w in weights)
        self.Wu = torch.nn.ParameterList(torch.nn.Parameter(w[1].float()) for w in weights)
        self.Wd = torch.nn.ParameterList(torch.nn.Parameter(w[2].float()) for w in weights)
        self.l1 = l1_coeff
        self.cap = cap
        self.max_dense = max_dense
        self.tc = tensor_cores
        self.bias_feature = bias_feature
        self.last_status = []

    def forward(self, x):
        """x [T][D] (any float dtype) -> the fp32 stream after the last layer."""
        self.last_status = []
        s = x.float()
        y = None  # the last layer's output, not yet added where the next norm adds it
        for i, (Wg, Wu, Wd) in enumerate(zip(self.Wg, self.Wu, self.Wd)):
            if self.norms is None:
                a = s.to(torch.bfloat16)
            elif y is None:
                a = AddRMSNormFunction.apply(s, self.norms[i], None, self.eps)
            else:
                a, s = AddRMSNormFunction.apply(y, self.norms[i], s, self.eps)
            y = SparseGatedFFNFunction.apply(a, Wg, Wu, Wd, self.l1, self.cap, self.max_dense,
                                             self.tc, self.last_status)
            if self.bias_feature:
                y = torch.cat([y[:, :-1], torch.zeros_like(y[:, -1:])], dim=1)
            if self.norms is None:
                s, y = s + y, None
        return s if y is None else s + y

    def status_flags(self) -> int:
        """OR of the device status words of the last forward (synchronises)."""
        flags = 0
        for s in self.last_status:
            flags |= int(s.item())
        return flags
