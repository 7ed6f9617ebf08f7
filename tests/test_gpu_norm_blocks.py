"""The norm and the 8-bit products where they are used: torch.autograd (the fused
add + norm, the e4m3 linear layer, the pre-norm stack) and the serving block,
against plain 64-bit implementations of the same steps.

Tolerances: as in the kernels' own tests for what one kernel computes; for
chains of several, the bar of the stack without norms (2e-2 RMS, 5e-3 RMS in
the mean) on the kernels' own gate decisions."""
import numpy as np
import pytest
import torch

import activation_sparse_gated_gate_gb300 as tw
from _gpu import ensure_built
from activation_sparse_gated_gate_gb300.autograd import (AddRMSNormFunction, Fp8Linear,
                                                         Fp8LinearFunction, SparseFFNStack)
from activation_sparse_gated_gate_gb300.block import Fp8GateFFN

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def plain_norm(t, w, eps):
    return t / torch.sqrt((t * t).mean(1, keepdim=True) + eps) * w


@pytest.mark.parametrize("xt,rt", [(F32, F32), (BF16, F32), (F32, None), (BF16, BF16)])
@pytest.mark.parametrize("expanded", [False, True])
def test_norm_function_gradients(xt, rt, expanded):
    g = _gen(1)
    T, D, eps = 37, 200, 1e-5
    x = _randn(g, T, D).to(xt).requires_grad_(True)
    w = (1 + 0.1 * _randn(g, D)).requires_grad_(True)
    r = None if rt is None else (2 * _randn(g, T, D)).to(rt).requires_grad_(True)
    cy = torch.full((), 0.5, device="cuda") if expanded else _randn(g, T, D)
    ct = torch.full((), -0.25, device="cuda") if expanded else _randn(g, T, D)
    out = AddRMSNormFunction.apply(x, w, r, eps)
    y, total = out if r is not None else (out, None)
    loss = (y.float() * cy).sum()
    if total is not None:
        loss = loss + (total.float() * ct).sum()
    loss.backward()
    # the same in 64 bits, on the stream and the incoming gradients as they are kept
    x64, w64 = x.detach().to(F64).requires_grad_(True), w.detach().to(F64).requires_grad_(True)
    r64 = None if r is None else r.detach().to(F64).requires_grad_(True)
    t64 = x64 if r is None else x64 + r64
    ref = (plain_norm(t64, w64, eps) * cy.to(BF16).to(F64)).sum()
    if r is not None:
        ref = ref + (t64 * ct.to(rt).to(F64)).sum()
    ref.backward()
    # a bf16 stream is rounded (2^-8) before the backward reads it: n and dx follow;
    # bf16 gradients round once more, and dx of a bf16 stream once before x's type
    loose = BF16 in (xt, rt)
    for a, b in ((x, x64), (w, w64)) + (() if r is None else ((r, r64),)):
        scale = float(b.grad.abs().max())
        tol = 4 * 2.0 ** -8 if loose else 64 * E
        assert float((a.grad.to(F64) - b.grad).abs().max()) <= tol * scale
        assert a.grad.dtype == a.dtype


def dequant(q, s, block):
    R, C = q.shape
    s = s.to(F64).repeat_interleave(block, 0)[:R].repeat_interleave(128, 1)[:, :C]
    return q.float().to(F64) * s


@pytest.mark.parametrize("T,N,K", [(1, 16, 8), (5, 300, 130), (257, 128, 640), (1000, 384, 257)])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_linear(T, N, K, dt):
    g = _gen(T + N + K)
    x = _randn(g, T, K).to(dt).requires_grad_(True)
    lin = Fp8Linear(_randn(g, N, K) / K ** 0.5)
    dy = _randn(g, T, N).to(dt)
    y = lin(x)
    assert y.dtype == dt
    y.backward(dy)
    w = lin.weight.detach()
    # the products of the quantised operands, each in 64 bits
    qx, qw = tw.twell_quant_fp8(x.detach(), transposed=True), \
        tw.twell_quant_fp8(w, block_rows=128, transposed=True)
    qd = tw.twell_quant_fp8(dy, transposed=True)
    cases = ((y.detach(), dequant(qx.q, qx.scale, 1), dequant(qw.q, qw.scale, 128), K),
             (x.grad, dequant(qd.q, qd.scale, 1), dequant(qw.qt, qw.scale_t, 128), N),
             (lin.weight.grad, dequant(qd.qt, qd.scale_t, 1), dequant(qx.qt, qx.scale_t, 1), T))
    for got, a, b, k in cases:
        ref = a @ b.t()
        tol = (k + 8) * 2 * E * (a.abs() @ b.abs().t()) + 1e-40
        if got.dtype == BF16:
            tol = tol + 2.0 ** -8 * (ref.abs() + tol)
        assert ((got.to(F64) - ref).abs() <= tol).all()
    # and near the layer in full precision: each operand is off by at most half a unit
    # of e4m3 (2^-4 relative, 2^-10 of its scale below the normal range)
    def off(v, scale, block):
        s = dequant(torch.ones_like(v), scale, block)
        return torch.maximum(v.abs() * 2.0 ** -4, s * 2.0 ** -10) * (1 + 1e-6)

    x64, w64 = x.detach().to(F64), w.to(F64)
    ex, ew = off(x64, qx.scale, 1), off(w64, qw.scale, 128)
    tol = ex @ w64.abs().t() + x64.abs() @ ew.t() + ex @ ew.t()
    full = x64 @ w64.t()
    assert ((y.detach().to(F64) - full).abs() <= tol * 1.001 + 2.0 ** -8 * full.abs() + 1e-6).all()


def test_linear_partial_and_empty():
    g = _gen(9)
    x, w = _randn(g, 32, 64), _randn(g, 48, 64)
    wr = w.clone().requires_grad_(True)
    Fp8LinearFunction.apply(x, wr).sum().backward()          # expanded gradient, no dx
    assert wr.grad.shape == w.shape
    xr = x.clone().requires_grad_(True)
    Fp8LinearFunction.apply(xr, w).sum().backward()
    assert xr.grad.shape == x.shape
    wr.grad = None
    Fp8LinearFunction.apply(x[:0], wr).sum().backward()
    assert (wr.grad == 0).all()


def test_prenorm_stack():
    # two pre-norm layers with gates at about 8 %: the loss's gradients against 64-bit
    # autograd over the same steps, on the gate decisions the kernels took
    g = _gen(3)
    T, D, F, C, L, lam = 320, 128, 512, 32, 2, 2e-5
    layers = [(_randn(g, F, D) / D ** 0.5, _randn(g, F, D) / D ** 0.5, 0.2 * _randn(g, F, D) / F ** 0.5)
              for _ in range(L)]
    for wg, _, _ in layers:
        wg[:, -1] = -1.5
    norms = [1 + 0.05 * _randn(g, D) for _ in range(L)]
    for n in norms:
        n[-1] = 1.0
    x = _randn(g, T, D)
    x[:, -1] = 1.0
    stack = SparseFFNStack([tuple(t.to(BF16) for t in l) for l in layers], l1_coeff=lam, cap=C,
                           max_dense=T, tensor_cores=False, norms=norms)
    xr = x.clone().requires_grad_(True)
    dout = _randn(g, T, D)
    out = stack(xr)
    (out * dout).sum().backward()
    assert stack.status_flags() == 0

    x64 = x.to(F64).requires_grad_(True)
    p64 = [[p.detach().to(BF16).to(F64).requires_grad_(True) for p in l]
           for l in zip(stack.Wg, stack.Wu, stack.Wd)]
    n64 = [n.detach().to(F64).requires_grad_(True) for n in stack.norms]
    s, loss = x64, 0.0
    keep = torch.ones(D, dtype=F64, device="cuda")
    keep[-1] = 0.0
    for (wg, wu, wd), n in zip(p64, n64):
        a = plain_norm(s, n, 1e-6)
        a = a + (a.detach().to(BF16).to(F64) - a.detach())    # bf16 input, gradient through
        z32 = torch.empty((T, F), device="cuda")
        h = tw.TwELL(T, F, 128)
        tw.twell_gate_pack(a.detach().to(BF16), wg.detach().to(BF16), h, z_debug=z32)
        z = (a @ wg.t()) * (z32 > 0)
        loss = loss + lam * z.sum()
        s = s + ((z * (a @ wu.t())) @ wd) * keep
    (loss + (s * dout.to(F64)).sum()).backward()
    got, ref = out.detach().to(F64) - x.to(F64), s.detach() - x64.detach()
    assert float((got - ref).abs().max()) <= 2e-2 * float(ref.pow(2).mean().sqrt())
    pairs = [(xr.grad, x64.grad)] + [(a.grad, b.grad) for a, b in zip(stack.norms, n64)]
    for i, ps in enumerate(zip(stack.Wg, stack.Wu, stack.Wd)):
        pairs += [(a.grad, b.grad) for a, b in zip(ps, p64[i])]
    for a, b in pairs:
        r = float(b.pow(2).mean().sqrt())
        assert float((a.to(F64) - b).abs().max()) <= 2e-2 * max(r, 0.05 * float(b.abs().max()))
        assert float((a.to(F64) - b).pow(2).mean().sqrt()) <= 5e-3 * r


def test_stack_refuses_a_wrong_number_of_norms():
    w = tuple(torch.zeros((128, 64), dtype=BF16, device="cuda") for _ in range(3))
    with pytest.raises(ValueError):
        SparseFFNStack([w], norms=[])


@pytest.mark.parametrize("T", [1, 16, 300])
@pytest.mark.parametrize("residual", [True, False])
def test_serving_block(T, residual):
    g = _gen(T)
    D, F = 256, 1024
    norm = 1 + 0.1 * _randn(g, D)
    wg = _randn(g, F, D) / D ** 0.5
    wg[:, -1] = -1.0
    wu, wd = (_randn(g, F, D) / D ** 0.5).to(BF16), (_randn(g, F, D) / F ** 0.5).to(BF16)
    block = Fp8GateFFN(norm, wg, wu, wd, width=16)
    x = _randn(g, T, D)
    r = _randn(g, T, D) if residual else None
    h = block.buffers(T)
    y, total = block(x, r, h=h)
    assert int(h.status.item()) == 0
    t = x if r is None else x + r
    assert (total == t).all()
    a = tw.twell_rms_norm(t, norm, fp8=True)
    z = dequant(a.q, a.scale, 1) @ dequant(block.Wg_q, block.Wg_scale, 128).t()
    u = a.y.to(F64) @ wu.to(F64).t()
    ref = (z.clamp_min(0) * u) @ wd.to(F64)
    # fp32 sums throughout; a gate within rounding of zero contributes as little
    assert float((y.to(F64) - ref).abs().max()) <= 1e-5 * float(ref.abs().max()) + 1e-30
    # and in full precision: 8 bits on the gate's two operands
    full = ((plain_norm(t.to(F64), norm.to(F64), 1e-6) @ wg.to(F64).t()).clamp_min(0) * u) @ wd.to(F64)
    assert float((y.to(F64) - full).norm()) <= 0.2 * float(full.norm())
    # a second call on the same buffers, captured and replayed
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, _ = block(x, r, h=h)
    graph.replay()
    torch.cuda.synchronize()
    assert float((y2 - y).abs().max()) <= 1e-5 * float(y.abs().max())


def test_serving_block_refuses_shapes():
    w = torch.zeros((128, 64), dtype=BF16, device="cuda")
    with pytest.raises(ValueError):
        Fp8GateFFN(torch.ones(32, device="cuda"), w, w, w)
    with pytest.raises(ValueError):
        Fp8GateFFN(torch.ones(64, device="cuda"), w, w[:64], w)
