"""The norm, the choice of experts and their FFNs from 4-bit weights run together, as a decode
loop does, against 64-bit arithmetic from the formulas."""
import numpy as np
import pytest
import torch

import activation_sparse_gated_gate_gb300 as tw
from activation_sparse_gated_gate_gb300.block import Int4Experts
from tests._gpu import ensure_built
from tests.test_gpu_moe import check_choice, check_y, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def make(E, F, D, seed=0, act="relu", top_k=2, **kw):
    g = torch.Generator().manual_seed(seed)
    w = [torch.randn((E, F, D), generator=g) / D ** 0.5 for _ in range(3)]
    router = (2 * torch.randn((E, D), generator=g) / D ** 0.5).cuda() if E > 1 else None
    norm = (1 + 0.1 * torch.randn((D,), generator=g)).cuda()
    return Int4Experts(norm, router, *(v.cuda() for v in w), top_k=top_k if E > 1 else 1, act=act,
                       **kw)


def check_block(block, x, residual, y, total, o):
    """total and the norm by their formulas; the experts on the norm as it was rounded
    (half a bf16 step, 2^-8 of it, beside the fp32 norm's own few ulps)."""
    xd = f64(x) + (0 if residual is None else f64(residual))
    if residual is not None:
        step = 2.0 ** -8 if residual.dtype is torch.bfloat16 else 2.0 ** -23
        assert (np.abs(f64(total) - xd) <= step * np.abs(xd)).all()
    a = xd / np.sqrt((xd ** 2).mean(1, keepdims=True) + block.eps) * f64(block.norm)
    n = tw.twell_rms_norm(x, block.norm, residual=residual, eps=block.eps).y
    assert (np.abs(f64(n) - a) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(a) + 1e-30).all()
    w = [block.Wg, block.Wu, block.Wd]
    if block.router is None:
        one = np.ones((len(xd), 1))
        check_y(o, n, w, block.act, one, 0 * one)
    else:
        wt, dw = check_choice(o, n, block.router, block.top_k, block.renormalise)
        check_y(o, n, w, block.act, wt, dw)
    assert y is o.y


@pytest.mark.parametrize("act,renormalise", [("relu", True), ("silu", False)])
@pytest.mark.parametrize("T,x_type,r_type", [(1, torch.float32, torch.float32),
                                             (5, torch.bfloat16, torch.bfloat16),
                                             (20, torch.float32, None)])
def test_block(T, x_type, r_type, act, renormalise):
    D = 512
    block = make(8, 96, D, act=act, renormalise=renormalise, group=64, zero_points=True)
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, D), generator=g).to(x_type).cuda()
    r = None if r_type is None else torch.randn((T, D), generator=g).to(r_type).cuda()
    y, total, o = block(x, r)
    check_block(block, x, r, y, total, o)


def test_one_expert():
    block = make(1, 200, 256, seed=3, group=32)
    x = torch.randn((4, 256)).cuda()
    y, total, o = block(x)
    assert total is x
    check_block(block, x, None, y, total, o)


def test_given_choice():
    block = make(4, 64, 256, seed=4)
    x = torch.randn((6, 256)).cuda()
    _, _, o = block(x)
    ids, weights = o.ids.clone(), o.weights.clone()
    ids[4:] = -1                                   # two rows of padding
    y, _, _ = block(x, ids=ids, weights=weights)
    n = tw.twell_rms_norm(x, block.norm, eps=block.eps).y
    w64 = f64(weights)
    check_y(tw.Moe(y, ids, weights), n, [block.Wg, block.Wu, block.Wd], "relu", w64, 0 * w64)
    assert not y[4:].any()


def test_decode_loop_and_graph():
    """Layers one after the other, a projection from 4-bit weights between them; the loop
    captured and replayed on other inputs."""
    D = 256
    blocks = [make(8, 64, D, seed=s) for s in (1, 2)]
    g = torch.Generator().manual_seed(9)
    proj = tw.twell_quant_int4((torch.randn((D, D), generator=g) / D ** 0.5).cuda(), group=64)

    def step(x, stream):
        for b in blocks:
            y, stream, _ = b(x, stream)
            x = tw.twell_gemv_int4(y.to(torch.bfloat16), proj, dtype=torch.float32)
        return x, stream

    x = torch.randn((3, D), generator=g).cuda()
    s = torch.randn((3, D), generator=g).cuda()
    step(x, s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, s)
    for seed in (1, 2):
        h = torch.Generator().manual_seed(seed)
        x.copy_(torch.randn((3, D), generator=h))
        s.copy_(torch.randn((3, D), generator=h))
        graph.replay()
        ref = step(x, s)
        assert all(torch.equal(a, b) for a, b in zip(out, ref))


def test_refusals():
    w = torch.zeros((2, 8, 64), device="cuda")
    norm, r = torch.ones((64,), device="cuda"), torch.zeros((2, 64), device="cuda")
    for bad in (lambda: Int4Experts(norm, None, w, w, w), lambda: Int4Experts(norm, r, w, w, w[:1]),
                lambda: Int4Experts(norm[:32], r, w, w, w), lambda: Int4Experts(norm, r[:1], w, w, w),
                lambda: Int4Experts(norm, None, w[:1], w[:1], w[:1], top_k=2),
                lambda: Int4Experts(norm, r, w[0], w[0], w[0])):
        with pytest.raises(ValueError):
            bad()
