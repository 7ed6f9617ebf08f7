"""What the norm and 8-bit calls do around their kernels: which tensors they refuse,
whose status word they use, and the outputs that a caller hands in."""
import numpy as np
import pytest
import torch

import activation_sparse_gated_gate_gb300 as tw
import oracle
from _gpu import assert_twell_equal, ensure_built, fetch_twell
from activation_sparse_gated_gate_gb300 import autograd
from activation_sparse_gated_gate_gb300.autograd import (AddRMSNormFunction, Fp8Linear,
                                                         Fp8LinearFunction, SparseFFNStack,
                                                         SparseGatedFFNFunction)
from activation_sparse_gated_gate_gb300.block import Fp8GateFFN

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _operands(g, M, N, K):
    return tw.twell_quant_fp8(_randn(g, M, K)), tw.twell_quant_fp8(_randn(g, N, K), block_rows=128)


# ---------------------------------------- refusals of tensors a kernel would write to


BAD_STATUS = [
    (lambda: torch.zeros(1, dtype=torch.int32), TypeError),                    # on the host
    (lambda: torch.zeros(1, dtype=torch.int64, device="cuda"), TypeError),
    (lambda: torch.zeros(1, device="cuda"), TypeError),
    (lambda: torch.zeros(0, dtype=torch.int32, device="cuda"), ValueError),
    (lambda: 7, TypeError)]


@pytest.mark.parametrize("make,error", BAD_STATUS)
def test_refuses_a_status_that_is_no_int32_word_of_the_device(make, error):
    qa, qb = _operands(_gen(1), 16, 256, 256)
    h = tw.TwELL(16, 256, 8)
    with pytest.raises(error):
        tw.twell_gemm_fp8(qa.q, qa.scale, qb.q, qb.scale, status=make())
    with pytest.raises(error):
        tw.twell_gate_pack_fp8(qa.q, qa.scale, qb.q, qb.scale, h, status=make())


def test_refuses_a_twell_of_another_device():
    qa, qb = _operands(_gen(2), 16, 256, 256)
    with pytest.raises(ValueError):
        tw.twell_gate_pack_fp8(qa.q, qa.scale, qb.q, qb.scale, tw.TwELL(16, 256, 8, device="cpu"))


def test_refuses_a_workspace_it_cannot_write():
    x, w, rstd = torch.ones((4, 64), device="cuda"), torch.ones(64, device="cuda"), \
        torch.ones(4, device="cuda")
    n = tw.twell_rms_norm_bwd_workspace(4, 64)
    with pytest.raises(TypeError):
        tw.twell_rms_norm_bwd(x, w, rstd, x, ws=torch.empty(n, dtype=torch.uint8))
    with pytest.raises(ValueError):
        tw.twell_rms_norm_bwd(x, w, rstd, x,
                              ws=torch.empty((n, 2), dtype=torch.uint8, device="cuda")[:, 0])
    wide = torch.empty(n + 16, dtype=torch.uint8, device="cuda")
    for off in (4, 8):
        with pytest.raises(tw.TwellError):
            tw.twell_rms_norm_bwd(x, w, rstd, x, ws=wide[off:off + n])
    a = tw.twell_rms_norm_bwd(x, w, rstd, x, ws=wide[16:])
    b = tw.twell_rms_norm_bwd(x, w, rstd, x)
    assert all((s == t).all() for s, t in zip(a, b))


def test_block_refuses_weights_of_several_devices():
    w, n = torch.zeros((128, 64), dtype=BF16, device="cuda"), torch.ones(64, device="cuda")
    for bad in ((n.cpu(), w, w, w), (n, w, w.cpu(), w), (n, w, w, w.cpu())):
        with pytest.raises(ValueError):
            Fp8GateFFN(*bad)


# --------------------------------------------------------------- status of a call


def _block(g, D=256, F=1024, p=0.02):
    norm, wg = torch.ones(D, device="cuda"), _randn(g, F, D) / D ** 0.5
    wu, wd = (_randn(g, F, D) / 16).to(BF16), (_randn(g, F, D) / 32).to(BF16)
    return Fp8GateFFN(norm, wg - 1.0 / D ** 0.5, wu, wd)


@pytest.mark.parametrize("T", [3, 300])
def test_block_without_buffers_keeps_the_flags(T):
    g = _gen(T)
    block, x = _block(g), _randn(g, T, 256)
    y, _ = block(x)
    assert block.status_flags() == 0
    prev = tw.twell_gate_pack_wait_limit(5)
    try:
        block(x)
        torch.cuda.synchronize()
    finally:
        tw.twell_gate_pack_wait_limit(prev)
    assert block.status_flags() & tw.FLAG_TIMEOUT
    block.status.zero_()
    again, _ = block(x)
    assert block.status_flags() == 0
    assert float((again - y).abs().max()) <= 1e-5 * float(y.abs().max())
    # with buffers of the caller's, in their own word
    h = block.buffers(T)
    prev = tw.twell_gate_pack_wait_limit(5)
    try:
        block(x, h=h)
        torch.cuda.synchronize()
    finally:
        tw.twell_gate_pack_wait_limit(prev)
    assert int(h.status.item()) & tw.FLAG_TIMEOUT and block.status_flags() == 0


def test_linear_keeps_the_flags_of_its_products():
    g = _gen(31)
    lin = Fp8Linear(_randn(g, 384, 256))
    x = _randn(g, 40, 256).requires_grad_(True)
    shared = int(tw.status_word().item())
    lin(x).sum().backward()
    assert lin.status_flags() == 0 and "status" not in lin.state_dict()
    for backward in (False, True):
        y = lin(x)
        prev = tw.twell_gate_pack_wait_limit(5)
        try:
            y.sum().backward() if backward else lin(x)
            torch.cuda.synchronize()
        finally:
            tw.twell_gate_pack_wait_limit(prev)
        assert lin.status_flags() & tw.FLAG_TIMEOUT
        lin.status.zero_()
    # none of it in the word that calls without a status share
    assert int(tw.status_word().item()) == shared
    assert Fp8LinearFunction.apply(x, lin.weight).shape == (40, 384)


def test_the_shared_status_word_is_zero_before_it_is_used(monkeypatch):
    # first asked for on a stream with work in front of it, then written from another:
    # the zeroing must not come after the flag
    monkeypatch.setattr(tw, "_STATUS", {})
    side = torch.cuda.Stream()
    torch.zeros(1, dtype=torch.int32, device="cuda").bitwise_or_(1)  # (its kernels are loaded)
    with torch.cuda.stream(side):
        torch.cuda._sleep(1000)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
        word = tw.status_word()
    word.bitwise_or_(tw.FLAG_TIMEOUT)
    torch.cuda.synchronize()
    assert int(word.item()) == tw.FLAG_TIMEOUT
    assert tw.status_word() is word


# ------------------------------------------------------------------ empty batches


@pytest.mark.parametrize("dt", [BF16, F32])
def test_linear_of_an_empty_batch_with_odd_widths(dt):
    # K = 130 and N = 300: neither a multiple of 16
    g = _gen(41)
    lin = Fp8Linear(_randn(g, 300, 130))
    x = torch.empty((0, 130), dtype=dt, device="cuda", requires_grad=True)
    y = lin(x)
    assert y.shape == (0, 300) and y.dtype == dt
    y.sum().backward()
    assert x.grad.shape == (0, 130) and (lin.weight.grad == 0).all()


def test_products_without_rows_or_columns():
    qa, qb = _operands(_gen(42), 24, 200, 130)
    for rows, cols in ((0, 200), (24, 0), (0, 0)):
        c = tw.twell_gemm_fp8(qa.q[:rows], qa.scale[:rows], qb.q[:cols], qb.scale[:-(-cols // 128)])
        assert c.shape == (rows, cols)
    h = tw.TwELL(0, 256, 8)
    wide = tw.twell_quant_fp8(torch.ones((256, 130), device="cuda"), block_rows=128)
    assert tw.twell_gate_pack_fp8(qa.q[:0], qa.scale[:0], wide.q, wide.scale, h) is h


# --------------------------------------------------------- sizes near 32 bits' end


@pytest.mark.parametrize("axis", [0, 1])
def test_quant_of_2_31_rows_or_columns(axis):
    # 2^31 - 8 of them: rounded up to whole blocks they pass 31 bits.  Every stretch as by
    # itself
    n, step = 2**31 - 8, 2**28
    v = torch.empty(n, dtype=BF16, device="cuda")
    for a in range(0, n, step):
        v[a:a + step] = _randn(_gen(a // step), min(step, n - a)).to(BF16)
    if axis == 0:
        o = tw.twell_quant_fp8(v.view(n, 1), rows=False, transposed=True)
        q, scale = o.qt, o.scale_t
    else:
        o = tw.twell_quant_fp8(v.view(1, n))
        q, scale = o.q, o.scale
    assert q.shape == (1, n) and scale.shape == (1, 2**24)
    for a in range(0, n, step):
        b = min(a + step, n)
        part = tw.twell_quant_fp8(v[a:b].view(1, b - a))
        assert (part.q.view(torch.uint8) == q[:, a:b].view(torch.uint8)).all()
        assert (part.scale == scale[:, a // 128:-(-b // 128)]).all()
    del v, o, q, scale
    torch.cuda.empty_cache()


# ------------------------------------------------------------- waits that run out


FORMS = [(512, 1024, 2048, 1), (4, 1024, 2048, 128),   # a cluster per tile
         (4, 8192, 512, 128),                          # the decode kernel
         (300, 8192, 512, 128), (1000, 3200, 384, 1),  # a CTA per tile
         (4096, 4096, 2048, 128), (4096, 4096, 2048, 1),  # pairs of CTAs
         (2500, 2000, 1100, 128)]                      # and a last round of quarters


@pytest.mark.parametrize("M,N,K,block", FORMS)
def test_a_call_that_gives_up_drains_what_it_issued(M, N, K, block):
    # bounds that run out at different places of the pipeline.  What is in flight then
    # arrives, so that the call ends long before the second that each wait for it may
    # take; the next call is right
    g = _gen(M + N + K)
    qa = tw.twell_quant_fp8(_randn(g, M, K))
    qb = tw.twell_quant_fp8(_randn(g, N, K), block_rows=block)
    want = tw.twell_gemm_fp8(qa.q, qa.scale, qb.q, qb.scale)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    gave_up = 0
    for ns in (1, 5, 50, 200, 400, 700, 1000, 1500, 2000, 3000, 5000, 8000) * 3:
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        prev = tw.twell_gate_pack_wait_limit(ns)
        try:
            a.record()
            tw.twell_gemm_fp8(qa.q, qa.scale, qb.q, qb.scale, status=st)
            b.record()
        finally:
            tw.twell_gate_pack_wait_limit(prev)
        again = tw.twell_gemm_fp8(qa.q, qa.scale, qb.q, qb.scale)
        torch.cuda.synchronize()
        assert a.elapsed_time(b) < 500
        assert (again == want).all()
        gave_up += int(st.item()) == tw.FLAG_TIMEOUT
        st.zero_()
    assert gave_up > 0


# --------------------------------------------------- outputs that the caller hands in


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("fp8", [True, False])
def test_norm_allocates_y_when_asked_for_bf16(bf16, fp8):
    # whether or not q and scale were given
    x, w = _randn(_gen(51), 6, 256), torch.ones(256, device="cuda")
    want = tw.twell_rms_norm(x, w, fp8=True)
    q, scale = torch.empty((6, 256), dtype=E4M3, device="cuda"), torch.empty((6, 2), device="cuda")
    o = tw.twell_rms_norm(x, w, q=q, scale=scale, bf16=bf16, fp8=fp8)
    assert o.q is q and (q.float() == want.q.float()).all() and (scale == want.scale).all()
    if bf16:
        assert (o.y == want.y).all()
    else:
        assert o.y is None


MARK = 0xA5


def _inside(rows, cols, off, pitch):
    """A [rows][cols] e4m3 view that starts `off` bytes into a marked buffer of that pitch,
    and a function that tells whether a byte around it changed."""
    buf = torch.full((rows * pitch + off + 64,), MARK, dtype=torch.uint8, device="cuda")
    assert buf.data_ptr() % 128 == 0
    view = buf[off:off + rows * pitch].view(rows, pitch)[:, :cols]

    def changed():
        inside = torch.zeros_like(buf, dtype=torch.bool)
        inside[off:off + rows * pitch].view(rows, pitch)[:, :cols] = True
        return bool((buf[~inside] != MARK).any())

    return view.view(E4M3), changed


def _same(a, b):
    return bool((a.view(torch.uint8) == b.view(torch.uint8)).all())


# start and pitch (beyond the columns) of the rows: on 1, 2, 4, 8 and 16 bytes
PLACES = [(0, 0), (1, 3), (2, 2), (4, 4), (8, 0), (8, 8), (16, 5), (3, 16), (16, 16)]


@pytest.mark.parametrize("off,more", PLACES)
@pytest.mark.parametrize("R,C", [(5, 7), (37, 200), (130, 256), (300, 1001), (128, 392)])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_quant_into_rows_anywhere(off, more, R, C, block, dt):
    x = _randn(_gen(R + C), R, C).to(dt)
    want = tw.twell_quant_fp8(x, block_rows=block, transposed=True)
    for rows, transposed in ((True, False), (False, True), (True, True)):
        q, q_changed = _inside(R, C, off, C + more)
        qt, qt_changed = _inside(C, R, off, R + more)
        s, st = torch.empty_like(want.scale), torch.empty_like(want.scale_t)
        o = tw.twell_quant_fp8(x, block_rows=block, rows=rows, transposed=transposed,
                               out=tw.QuantFp8(q, s, qt, st))
        if rows:
            assert o.q.data_ptr() == q.data_ptr() and _same(q, want.q) and (s == want.scale).all()
        if transposed:
            assert _same(qt, want.qt) and (st == want.scale_t).all()
        assert not q_changed() and not qt_changed()


@pytest.mark.parametrize("off,more", PLACES)
@pytest.mark.parametrize("T,D", [(1, 9), (5, 136), (37, 200), (64, 256), (9, 1001), (3, 8200)])
@pytest.mark.parametrize("xt", [BF16, F32])
def test_norm_into_e4m3_rows_anywhere(off, more, T, D, xt):
    g = _gen(T + D)
    x, r, w = _randn(g, T, D).to(xt), _randn(g, T, D), 1 + 0.1 * _randn(g, D)
    want = tw.twell_rms_norm(x, w, residual=r, fp8=True)
    q, changed = _inside(T, D, off, D + more)
    scale = torch.empty_like(want.scale)
    o = tw.twell_rms_norm(x, w, residual=r, q=q, scale=scale)
    # (the row's sum is taken in another order where the rows are read element by element:
    # y is off by (D / 2 + 8) 2^-24 either way, so e4m3 by a step where that crosses a tie)
    tol = 2 * (D / 2 + 8) * 2.0 ** -24
    assert ((o.scale - want.scale).abs() <= (tol + 2.0 ** -23) * want.scale).all()
    a, b = q.float() * 1.0, want.q.float()
    step = torch.maximum(b.abs(), a.abs()) * 2.0 ** -3
    assert ((a - b).abs() <= torch.clamp(step, min=2.0 ** -9)).all()
    assert ((a != b).float().mean() <= 0.01) or D < 100
    assert (o.total == want.total).all()
    assert not changed()


# --------------------------------------------------------------- second derivatives


@pytest.mark.parametrize("which", ["norm", "add", "linear"])
def test_a_second_derivative_is_refused(which):
    # not left out: a penalty on a gradient would otherwise have no gradient itself
    g = _gen(61)
    x = _randn(g, 16, 128).requires_grad_(True)
    w = torch.ones(128, device="cuda", requires_grad=True)
    if which == "linear":
        y = Fp8Linear(_randn(g, 256, 128))(x)
    elif which == "add":
        y = AddRMSNormFunction.apply(x, w, _randn(g, 16, 128), 1e-6)[0]
    else:
        y = AddRMSNormFunction.apply(x, w, None, 1e-6)
    dx, = torch.autograd.grad(y.float().sum(), x, create_graph=True)
    assert (dx == torch.autograd.grad(y.float().sum(), x, retain_graph=True)[0]).all()
    with pytest.raises(RuntimeError, match="cannot be differentiated"):
        (x.square().sum() + dx.square().sum()).backward()


# -------------------------------------------- two launches, and the forms between


@pytest.mark.parametrize("block", [1, 128])
def test_a_product_of_two_launches_in_a_graph(block):
    # the last round's quarters start as the launch before them leaves, in a graph too
    g = _gen(71)
    qa, qa2 = (tw.twell_quant_fp8(_randn(g, 2500, 1100)) for _ in range(2))
    qb = tw.twell_quant_fp8(_randn(g, 2000, 1100), block_rows=block)
    wants = [tw.twell_gemm_fp8(a.q, a.scale, qb.q, qb.scale) for a in (qa, qa2)]
    a, s = tw.twell_quant_fp8(torch.zeros((2500, 1100), device="cuda"))[:2]
    c, out = torch.empty_like(wants[0]), torch.empty_like(wants[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            c.zero_()
            tw.twell_gemm_fp8(a, s, qb.q, qb.scale, out=c)
            out.copy_(c)
    for i in (0, 1, 0, 1):
        a.view(torch.uint8).copy_((qa, qa2)[i].q.view(torch.uint8))
        s.copy_((qa, qa2)[i].scale)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert (out == wants[i]).all()


@pytest.mark.parametrize("tensor_cores", [True, False])
def test_prenorm_stack_steps(tensor_cores, monkeypatch):
    # what goes into and comes out of each layer's FFN, forward and backward, held against
    # direct calls of the norm on the same values: bit for bit (the FFN functions have
    # their own tests)
    g = _gen(81)
    T, D, F, C = 320, 128, 1024, 32
    layers = [tuple((_randn(g, *s) * f).to(BF16) for s, f in (((F, D), D ** -0.5),) * 2
                    + (((F, D), 0.2 * F ** -0.5),)) for _ in range(2)]
    for wg, _, _ in layers:
        wg[:, -1] = -1.5
    norms = [1 + 0.05 * _randn(g, D) for _ in range(2)]
    x = _randn(g, T, D)
    x[:, -1] = 1.0
    seen = []

    class Seen:
        @staticmethod
        def apply(a, *rest):
            at = {"a": a.detach()}
            y = SparseGatedFFNFunction.apply(a, *rest)
            at["y"] = y.detach()
            a.register_hook(lambda d: at.__setitem__("da", d))
            y.register_hook(lambda d: at.__setitem__("dy", d))
            seen.append(at)
            return y

    monkeypatch.setattr(autograd, "SparseGatedFFNFunction", Seen)
    args = {} if tensor_cores else {"tensor_cores": False}
    stack = SparseFFNStack(layers, cap=C, max_dense=T, norms=norms, eps=1e-5, **args)
    xr = x.clone().requires_grad_(True)
    dout = _randn(g, T, D)
    out = stack(xr)
    out.backward(dout)
    assert stack.status_flags() == 0 and len(seen) == 2 and stack.tc == tensor_cores

    def no_bias(t):
        t = t.clone()
        t[:, -1] = 0.0
        return t

    w0, w1 = (n.detach() for n in stack.norms)
    o0 = tw.twell_rms_norm(x, w0, eps=1e-5, rstd=True)
    o1 = tw.twell_rms_norm(no_bias(seen[0]["y"]), w1, residual=x, eps=1e-5, rstd=True)
    assert (seen[0]["a"] == o0.y).all() and (seen[1]["a"] == o1.y).all()
    assert (out == o1.total + no_bias(seen[1]["y"])).all()
    assert float(seen[0]["y"].abs().max()) > 0 and float(seen[1]["da"].abs().max()) > 0
    assert (seen[1]["dy"] == no_bias(dout)).all()
    dx1, dw1 = tw.twell_rms_norm_bwd(o1.total, w1, o1.rstd, seen[1]["da"], dtotal=dout)
    assert (stack.norms[1].grad == dw1).all() and (seen[0]["dy"] == no_bias(dx1)).all()
    dx0, dw0 = tw.twell_rms_norm_bwd(x, w0, o0.rstd, seen[0]["da"])
    assert (stack.norms[0].grad == dw0).all() and (xr.grad == dx0 + dx1).all()
    for p in (*stack.Wg, *stack.Wu, *stack.Wd):
        assert float(p.grad.abs().max()) > 0


# batches between a decode step and a prompt: either side of where the decode form's
# columns for every K block end (64 tokens at 2048, 32 at 4096, 16 at 8192)
@pytest.mark.parametrize("T,D,F", [
    (17, 8192, 512), (16, 8192, 384), (32, 4096, 768), (33, 4096, 768), (64, 2048, 1024),
    (65, 2048, 1024), (100, 4096, 512), (128, 2048, 2048), (129, 2304, 1152), (192, 2048, 1024),
    (255, 2048, 1024), (512, 2304, 1152)])
def test_gate_of_middle_batches(T, D, F):
    # element by element: fp32 sums of exact products, off by (D + 8) 2 e sum |x w|
    g = _gen(T + D)
    x, w = _randn(g, T, D), _randn(g, F, D) / D ** 0.5
    x[:, -1] = 1.0
    w[:, -1] = -2.0                      # about 2 % active
    qx, qw = tw.twell_quant_fp8(x), tw.twell_quant_fp8(w, block_rows=128)
    h, z = tw.TwELL(T, F, 8), torch.empty((T, F), device="cuda")
    tw.twell_gate_pack_fp8(qx.q, qx.scale, qw.q, qw.scale, h, z_debug=z)
    a = qx.q.double() * qx.scale.double().repeat_interleave(128, 1)[:, :D]
    b = qw.q.double() * qw.scale.double().repeat_interleave(128, 0)[:F].repeat_interleave(
        128, 1)[:, :D]
    tol = (D + 8) * 2 * 2.0 ** -24 * (a.abs() @ b.abs().t())
    assert ((z.double() - a @ b.t()).abs() <= tol).all()
    assert int(h.status.item()) == 0
    assert_twell_equal(fetch_twell(h), oracle.twell_pack(z.cpu().numpy(), 128, 8))
    act = (z > 0).cpu().numpy()
    bits = h.block_bits.cpu().numpy().view(np.uint32)
    for k in range((T + 127) // 128):
        any_ = act[k * 128:(k + 1) * 128].any(0).reshape(-1, 32)
        want = (any_.astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(1)
        np.testing.assert_array_equal(bits[k].astype(np.uint64), want)
    # and the general product of the same operands
    c = tw.twell_gemm_fp8(qx.q, qx.scale, qw.q, qw.scale, dtype=F32)
    assert ((c.double() - a @ b.t()).abs() <= tol).all()


# products and gates of few rows: either side of the decode form's rows (32, the gate's 128)
# and of its 76 column tiles
@pytest.mark.parametrize("M", [1, 16, 32, 33, 64])
@pytest.mark.parametrize("N", [9728, 9729, 10240])
@pytest.mark.parametrize("K", [300, 1024])
def test_few_row_products_beside_the_decode_form(M, N, K):
    qa, qb = _operands(_gen(M + N + K), M, N, K)
    a = qa.q.double() * qa.scale.double().repeat_interleave(128, 1)[:, :K]
    b = qb.q.double() * qb.scale.double().repeat_interleave(128, 0)[:N].repeat_interleave(
        128, 1)[:, :K]
    tol = (K + 8) * 2 * 2.0 ** -24 * (a.abs() @ b.abs().t())
    c = tw.twell_gemm_fp8(qa.q, qa.scale, qb.q, qb.scale, dtype=F32)
    assert ((c.double() - a @ b.t()).abs() <= tol).all()


@pytest.mark.parametrize("T", [1, 128, 129])
@pytest.mark.parametrize("F", [9728, 9856])
def test_gates_beside_the_decode_form(T, F):
    test_gate_of_middle_batches(T, 512, F)


@pytest.mark.parametrize("T,D,F", [(2500, 1100, 2048), (2500, 1024, 2048), (2049, 1000, 2304)])
def test_gates_with_a_ragged_last_round(T, D, F):
    # 80 and 81 tiles of 256 x 256, from eight K blocks on with a last round of quarters
    test_gate_of_middle_batches(T, D, F)


# ------------------------------------------------- a gate that gave up leaves no garbage


def _gate_call(T, D, F, fp8):
    g = _gen(T + D + F)
    x, w = _randn(g, T, D), _randn(g, F, D) / D ** 0.5
    x[:, -1] = 1.0
    w[:, -1] = -1.0
    if fp8:
        qx, qw = tw.twell_quant_fp8(x), tw.twell_quant_fp8(w, block_rows=128)
        return lambda h: tw.twell_gate_pack_fp8(qx.q, qx.scale, qw.q, qw.scale, h)
    x, w = x.to(BF16), w.to(BF16)
    return lambda h: tw.twell_gate_pack(x, w, h)


def _counts_hold(call, T, F):
    h = tw.TwELL(T, F, 8)
    call(h)
    good = h.cnt.clone()
    assert int(h.status.item()) == 0
    gave_up = 0
    for ns in (1, 5, 100, 500, 1000, 2000, 4000, 8000):
        h.cnt.fill_(255)        # what memory that was never written may hold
        h.spill_slot.fill_(1 << 30)
        h.status.zero_()
        prev = tw.twell_gate_pack_wait_limit(ns)
        try:
            call(h)
            torch.cuda.synchronize()
        finally:
            tw.twell_gate_pack_wait_limit(prev)
        flags, n = int(h.status.item()), int(h.spill_n.item())
        gave_up += flags == tw.FLAG_TIMEOUT
        assert flags in (0, tw.FLAG_TIMEOUT)
        assert ((h.cnt == good) | (h.cnt == 0)).all()
        spilled = h.spill_slot[h.cnt.int() > 8]
        assert ((spilled >= 0) & (spilled < n)).all()
    assert gave_up > 0


@pytest.mark.parametrize("T,D,F", [(16, 2048, 1024), (300, 2048, 1024), (4096, 512, 4096),
                                   (2500, 2048, 2048)])
def test_a_gate_that_gives_up_counts_only_what_it_packed(T, D, F):
    # whoever reads the TwELL next finds the slices that were not packed empty
    _counts_hold(_gate_call(T, D, F, True), T, F)


@pytest.mark.parametrize("T,D,F", [(16, 2048, 1024), (300, 2048, 1024), (200, 64, 1024),
                                   (4096, 512, 4096)])
def test_a_bf16_gate_that_gives_up_counts_only_what_it_packed(T, D, F):
    _counts_hold(_gate_call(T, D, F, False), T, F)


# ------------------------------------------------------- more than 2^31 elements


def test_norm_of_more_than_2_31_elements():
    # the last rows as by themselves
    T, D = 270_000, 8192
    x = torch.empty((T, D), dtype=BF16, device="cuda")
    for a in range(0, T, 90_000):
        x[a:a + 90_000] = torch.randn((90_000, D), generator=_gen(a), device="cuda", dtype=F32).to(BF16)
    w = 1 + 0.1 * _randn(_gen(1), D)
    o = tw.twell_rms_norm(x, w, residual=x, fp8=True, rstd=True)
    dx, _ = tw.twell_rms_norm_bwd(o.total, w, o.rstd, o.y, dtotal=x)
    for rows in (slice(0, 3), slice(262_140, 262_150), slice(T - 3, T)):
        p = tw.twell_rms_norm(x[rows], w, residual=x[rows], fp8=True, rstd=True)
        assert (o.y[rows] == p.y).all() and (o.total[rows] == p.total).all()
        assert _same(o.q[rows], p.q) and (o.scale[rows] == p.scale).all()
        d, _ = tw.twell_rms_norm_bwd(p.total, w, p.rstd, p.y, dtotal=x[rows])
        assert (dx[rows] == d).all()
    q = tw.twell_quant_fp8(x, transposed=True)
    part = tw.twell_quant_fp8(x[T - 1000:])
    assert _same(q.q[T - 1000:], part.q) and (q.scale[T - 1000:] == part.scale).all()
    first = (T - 1000 + 127) // 128 * 128                       # whole blocks of 128 rows
    part = tw.twell_quant_fp8(x[first:], rows=False, transposed=True)
    assert _same(q.qt[:, first:], part.qt) and (q.scale_t[:, first // 128:] == part.scale_t).all()
    del x, o, dx, q
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dt", [BF16, F32])
def test_product_of_more_than_2_31_elements(dt):
    # one block of K: the sums are the same in every form
    M, N, K = 68_000, 32_768, 128
    qa, qb = _operands(_gen(91), M, N, K)
    c = tw.twell_gemm_fp8(qa.q, qa.scale, qb.q, qb.scale, dtype=dt)
    for rows in (slice(0, 300), slice(65_530, 65_560), slice(M - 200, M)):
        p = tw.twell_gemm_fp8(qa.q[rows], qa.scale[rows], qb.q, qb.scale, dtype=dt)
        assert (c[rows] == p).all()
    del c
    torch.cuda.empty_cache()
