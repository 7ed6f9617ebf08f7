"""Pre-norm sparse FFN block for serving, its gate in 8 bits.

One block of a ReLU Transformer's FFN as a decode loop or a prompt runs it:

    total = x + residual;  a = norm(total) * w        twell_rms_norm
    h = ReLU(a W_g), packed into TwELL                twell_gate_pack_fp8
    y = sum of the active h_j (a . W_u[:, j]) W_d[j]  twell_ffn_fwd

The norm leaves a in bf16 (for the up projection) and in e4m3 with a scale for
each 128 features (for the gate) in one pass.  At the densities this format is
for, the dense gate is nearly all of what the FFN reads for a few tokens and
nearly all of its products for many; its weights are kept in e4m3 with a scale
for each 128 x 128 block, quantised once here.  Argument marshalling only:
every step runs in libtwell's kernels.
"""
from __future__ import annotations

import torch

from . import (TwELL, twell_ffn_fwd, twell_gate_pack_fp8, twell_quant_fp8, twell_rms_norm)


class Fp8GateFFN:
    """Weights of one block: norm [D] (bf16 or fp32), Wg_t [F][D] (bf16 or fp32,
    quantised here), Wu_t and Wd [F][D] bf16; ``width`` slots per row and tile of
    the TwELL."""

    def __init__(self, norm, Wg_t, Wu_t, Wd, width=8, eps=1e-6):
        if Wu_t.shape != Wg_t.shape or Wd.shape != Wg_t.shape or norm.shape != Wg_t.shape[1:]:
            raise ValueError("shape mismatch: norm [D], Wg_t, Wu_t and Wd [F][D]")
        if any(w.device != Wg_t.device for w in (norm, Wu_t, Wd)):
            raise ValueError("the weights are on different devices")
        self.norm, self.Wu_t, self.Wd = norm, Wu_t, Wd
        self.width, self.eps = width, eps
        gate = twell_quant_fp8(Wg_t, block_rows=128)
        self.Wg_q, self.Wg_scale = gate.q, gate.scale
        # of the calls that bring no TwELL of their own
        self.status = torch.zeros((1,), dtype=torch.int32, device=Wg_t.device)

    def buffers(self, T):
        """The TwELL of a call of T rows; a decode loop keeps one per batch size."""
        return TwELL(T, self.Wg_q.shape[0], self.width, device=self.Wg_q.device)

    def __call__(self, x, residual=None, h=None):
        """x [T][D] bf16 or fp32 (and the residual stream, added to it); returns
        (y [T][D] fp32, total).  ``h``: the TwELL to use (``buffers``); its status
        word holds the call's flags.  Without one the call allocates its own, and
        its flags go to the block's word (``status_flags``)."""
        own = h is None
        h = self.buffers(x.shape[0]) if own else h
        status = self.status if own else h.status
        a = twell_rms_norm(x, self.norm, residual=residual, eps=self.eps, fp8=True)
        twell_gate_pack_fp8(a.q, a.scale, self.Wg_q, self.Wg_scale, h, status=status)
        y = twell_ffn_fwd(a.y, h, self.Wu_t, self.Wd, status=status)
        return y, (x if residual is None else a.total)

    def status_flags(self) -> int:
        """OR of the flags of every call without an ``h`` since ``status`` was last
        zeroed (synchronises).  Zero: every y returned so far is complete."""
        return int(self.status.item())
