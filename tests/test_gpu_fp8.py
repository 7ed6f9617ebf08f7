"""e4m3 quantisation by blocks of 128, the product of such operands and the gate
built on it, against plain 64-bit implementations.

Tolerances, with e = 2^-24: amax is exact and the scale one rounding (2 e);
v (448 / amax) has two roundings before e4m3's own (half a unit: 2^-4 relative,
2^-10 below 2^-6).  A product of two e4m3 values is exact in fp32; K of them
summed in any order, then scaled and summed over the blocks, are off by at most
(K + 8) 2 e sum |a b| (twice e per addition: the tensor core may truncate);
bf16 output (eight significant bits) adds 2^-8 |c|."""
import numpy as np
import pytest
import torch

import activation_sparse_gated_gate_gb300 as tw
import oracle
from _gpu import assert_twell_equal, ensure_built, fetch_twell

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
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


def block_amax(v, block):
    R, C = v.shape
    nr, nc = -(-R // block), -(-C // 128)
    p = torch.zeros((nr * block, nc * 128), dtype=torch.float64, device=v.device)
    p[:R, :C] = v.double().abs()
    return p.view(nr, block, nc, 128).amax(dim=(1, 3)).clamp_min(2.0 ** -64)


def spread(s, block, R, C):
    return s.double().repeat_interleave(block, 0)[:R].repeat_interleave(128, 1)[:, :C]


def check_quant(q, scale, v, block):
    R, C = v.shape
    amax = block_amax(v, block)
    assert q.shape == (R, C) and q.dtype == E4M3 and scale.shape == amax.shape
    assert ((scale.double() - amax / 448).abs() <= 2 * E * amax / 448).all()
    t = v.double() * (448 / spread(amax, block, R, C))
    half = torch.maximum(t.abs() * 2.0 ** -4, torch.full_like(t, 2.0 ** -10))
    assert ((q.float().double() - t).abs() <= half * (1 + 1e-9) + 4 * E * t.abs()).all()
    # the largest of each block sits on 448
    top = q.float().abs().double()
    assert (block_amax(top, block)[amax > 2.0 ** -64] == 448).all()


QSHAPES = [(1, 1), (1, 128), (3, 7), (16, 16), (130, 200), (128, 128), (257, 384), (64, 1001),
           (1000, 136), (4, 2304)]


@pytest.mark.parametrize("R,C", QSHAPES)
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("block", [1, 128])
def test_quant(R, C, dt, block):
    g = _gen(R * 1009 + C)
    x = (_randn(g, R, C) * torch.exp(_randn(g, R, 1))).to(dt)
    o = tw.twell_quant_fp8(x, block_rows=block, transposed=True)
    check_quant(o.q, o.scale, x, block)
    check_quant(o.qt, o.scale_t, x.t(), block)
    if block == 128:  # the transpose holds the same values
        assert (o.qt.float() == o.q.float().t()).all()
        assert (o.scale_t == o.scale.t()).all()
    only = tw.twell_quant_fp8(x, block_rows=block)
    assert only.qt is None and (only.q.float() == o.q.float()).all()
    only_t = tw.twell_quant_fp8(x, block_rows=block, rows=False, transposed=True)
    assert only_t.q is None and (only_t.qt.float() == o.qt.float()).all()


def test_quant_strides_and_reuse():
    g = _gen(3)
    wide = _randn(g, 150, 700)
    for off in (0, 4, 3):
        x = wide[:, off:off + 320]
        o = tw.twell_quant_fp8(x, transposed=True)
        want = tw.twell_quant_fp8(x.contiguous(), transposed=True)
        for a, b in zip(o, want):
            assert (a.float() == b.float()).all()
        again = tw.twell_quant_fp8(-x, transposed=True, out=o)
        assert again.q.data_ptr() == o.q.data_ptr()
        assert (o.q.float() == -want.q.float()).all()


def test_quant_special_values():
    x = torch.zeros((4, 256), device="cuda")
    x[1, :128] = 1e-30
    x[2, 3] = float("nan")
    x[2, 4] = 2.0
    x[3, 130] = float("inf")
    x[3, 5] = -1.0
    o = tw.twell_quant_fp8(x)
    assert (o.q[0].float() == 0).all() and (o.scale[0] > 0).all()
    assert (o.q[1].float() == 0).all()
    q2 = o.q[2].float()
    assert torch.isnan(q2[3]) and q2[4] == 448 and torch.isfinite(o.scale[2]).all()
    assert o.q[3, 5].float() == -448 and torch.isinf(o.scale[3, 1])
    assert torch.isnan(o.q[3, 130].float())


def operands(g, M, N, K, block):
    a = (_randn(g, M, K) * torch.exp(0.5 * _randn(g, M, 1))).to(BF16)
    b = _randn(g, N, K) * torch.exp(0.5 * _randn(g, N, 1))
    return tw.twell_quant_fp8(a), tw.twell_quant_fp8(b, block_rows=block)


def check_product(c, qa, qb, block):
    M, K = qa.q.shape
    N = qb.q.shape[0]
    a = qa.q.float().double() * spread(qa.scale, 1, M, K)
    b = qb.q.float().double() * spread(qb.scale, block, N, K)
    ref = a @ b.t()
    tol = (K + 8) * 2 * E * (a.abs() @ b.abs().t()) + 1e-40
    if c.dtype == BF16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    assert ((c.double() - ref).abs() <= tol).all()
    return ref


PSHAPES = [(1, 1, 1), (1, 128, 128), (1, 2048, 2048), (3, 40, 130), (4, 256, 1001),
           (16, 384, 256), (100, 130, 96), (128, 128, 128), (130, 257, 300), (257, 1000, 513),
           (64, 4096, 640), (300, 640, 2304), (1000, 1536, 272), (2049, 2304, 136),
           (4096, 2049, 400), (1, 2048, 8192), (16, 300, 4100), (130, 1500, 3000), (7, 9, 2050)]


@pytest.mark.parametrize("M,N,K", PSHAPES)
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_product(M, N, K, block, dt):
    qa, qb = operands(_gen(M * 7 + N * 3 + K), M, N, K, block)
    c = tw.twell_gemm_fp8(qa.q, qa.scale, qb.q, qb.scale, dtype=dt)
    check_product(c, qa, qb, block)
    again = tw.twell_gemm_fp8(qa.q, qa.scale, qb.q, qb.scale, dtype=dt)
    assert (again == c).all()
    assert int(tw.status_word().item()) == 0


# 80 and 81 tiles of 256 x 256: the last round's few run as quarters, in a second launch
@pytest.mark.parametrize("M,N,K", [(2500, 2000, 1100), (2049, 2304, 1024)])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_product_with_a_ragged_last_round(M, N, K, block, dt):
    test_product(M, N, K, block, dt)


def test_second_launches_in_order():
    # what follows a call on its stream sees both of its launches, what precedes it
    # is done before either: outputs overwritten just before and read just after
    qa, qb = operands(_gen(23), 2500, 2000, 1100, 128)
    want = tw.twell_gemm_fp8(qa.q, qa.scale, qb.q, qb.scale)
    gates = [gate_inputs(24 + i, 16, 512, 1024, 0.03 * (i + 1)) for i in range(2)]
    h = tw.TwELL(16, 1024, 8)
    wants = []
    for x, w in gates:
        tw.twell_gate_pack_fp8(x.q, x.scale, w.q, w.scale, h)
        wants.append((h.cnt.clone(), int(h.spill_n.item())))
    assert wants[0][1] != wants[1][1] > 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c, seen, counts = torch.empty_like(want), [], []
        for i in range(40):
            c.zero_()
            tw.twell_gemm_fp8(qa.q, qa.scale, qb.q, qb.scale, out=c)
            seen.append((c != want).sum())
            x, w = gates[i % 2]
            h.spill_n.fill_(7)
            tw.twell_gate_pack_fp8(x.q, x.scale, w.q, w.scale, h)
            counts.append((h.cnt.clone(), h.spill_n.clone()))
    side.synchronize()
    assert sum(int(n) for n in seen) == 0
    for i, (cnt, n) in enumerate(counts):
        assert (cnt == wants[i % 2][0]).all() and int(n) == wants[i % 2][1]


def test_product_into_wider_rows():
    qa, qb = operands(_gen(5), 70, 200, 256, 128)
    want = tw.twell_gemm_fp8(qa.q, qa.scale, qb.q, qb.scale)
    for off in (0, 8, 3):
        buf = torch.full((70, 264), 9.0, dtype=BF16, device="cuda")
        tw.twell_gemm_fp8(qa.q, qa.scale, qb.q, qb.scale, out=buf[:, off:off + 200])
        assert (buf[:, off:off + 200] == want).all()
        assert (buf[:, :off] == 9).all() and (buf[:, off + 200:] == 9).all()


def test_product_ignores_bytes_past_k():
    qa, qb = operands(_gen(6), 33, 140, 200, 128)
    want = tw.twell_gemm_fp8(qa.q, qa.scale, qb.q, qb.scale, dtype=F32)
    a = torch.full((33, 256), float("nan"), device="cuda").to(E4M3)
    b = torch.full((140, 256), float("nan"), device="cuda").to(E4M3)
    a[:, :200], b[:, :200] = qa.q, qb.q
    got = tw.twell_gemm_fp8(a[:, :200], qa.scale, b[:, :200], qb.scale, dtype=F32)
    assert (got == want).all()


def test_nan_stays_in_its_row_and_column():
    qa, qb = operands(_gen(7), 40, 300, 384, 128)
    want = tw.twell_gemm_fp8(qa.q, qa.scale, qb.q, qb.scale)
    qa.q[7, 130] = torch.tensor(float("nan"), device="cuda").to(E4M3)
    qb.q[250, 5] = torch.tensor(float("nan"), device="cuda").to(E4M3)
    got = tw.twell_gemm_fp8(qa.q, qa.scale, qb.q, qb.scale)
    bad = torch.isnan(got)
    assert bad[7].all() and bad[:, 250].all()
    bad[7] = True
    bad[:, 250] = True
    assert (got[~bad] == want[~bad]).all()


def test_product_nothing_to_do():
    qa, qb = operands(_gen(8), 8, 128, 128, 128)
    c = tw.twell_gemm_fp8(qa.q[:0], qa.scale[:0], qb.q, qb.scale)
    assert c.shape == (0, 128)


def test_product_on_another_stream_and_in_a_graph():
    qa, qb = operands(_gen(9), 64, 512, 640, 128)
    want = tw.twell_gemm_fp8(qa.q, qa.scale, qb.q, qb.scale)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = tw.twell_gemm_fp8(qa.q, qa.scale, qb.q, qb.scale, stream=side)
    side.synchronize()
    assert (got == want).all()
    qa2, _ = operands(_gen(10), 64, 512, 640, 128)
    out = torch.empty((64, 512), dtype=BF16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tw.twell_gemm_fp8(qa.q, qa.scale, qb.q, qb.scale, out=out)
    qa.q.view(torch.uint8).copy_(qa2.q.view(torch.uint8))
    qa.scale.copy_(qa2.scale)
    graph.replay()
    torch.cuda.synchronize()
    assert (out == tw.twell_gemm_fp8(qa2.q, qa2.scale, qb.q, qb.scale)).all()


@pytest.mark.parametrize("M,N,K,block", [
    (512, 1024, 2048, 1), (4, 1024, 2048, 128),   # a cluster per tile
    (4, 8192, 512, 128),                          # the decode kernel
    (300, 8192, 512, 128), (1000, 3200, 384, 1),  # a CTA per tile
    (4096, 4096, 512, 128), (4096, 4096, 512, 1),   # pairs of CTAs
    (2500, 2000, 1100, 128)])                       # and a last round of quarters
def test_a_wait_that_runs_out(M, N, K, block):
    # a bound of a few nanoseconds on every pipeline wait: the call returns, sets
    # the flag, and the next one is right again
    qa, qb = operands(_gen(12), M, N, K, block)
    want = tw.twell_gemm_fp8(qa.q, qa.scale, qb.q, qb.scale)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    prev = tw.twell_gate_pack_wait_limit(5)
    try:
        tw.twell_gemm_fp8(qa.q, qa.scale, qb.q, qb.scale, status=st)
        torch.cuda.synchronize()
    finally:
        tw.twell_gate_pack_wait_limit(prev)
    assert int(st.item()) & tw.FLAG_TIMEOUT
    assert (tw.twell_gemm_fp8(qa.q, qa.scale, qb.q, qb.scale) == want).all()


def gate_inputs(seed, T, D, F, p):
    g = _gen(seed)
    x = _randn(g, T, D)
    x[:, -1] = 1.0
    w = _randn(g, F, D) / D ** 0.5
    w[:, -1] = -(2.0 ** 0.5) * float(torch.erfinv(torch.tensor(1.0 - 2.0 * p)))
    return tw.twell_quant_fp8(x), tw.twell_quant_fp8(w, block_rows=128)


@pytest.mark.parametrize("T,D,F,p,W,cap", [
    (1, 64, 128, 0.3, 8, None), (5, 1, 256, 0.5, 8, None), (64, 256, 1024, 0.05, 16, None),
    (1, 2048, 2048, 0.01, 8, None), (16, 2048, 1024, 0.005, 8, None),
    (77, 72, 384, 0.10, 8, None), (130, 200, 640, 0.02, 8, None),
    (300, 512, 2048, 0.02, 8, None), (200, 128, 1024, 0.50, 8, None),
    (64, 128, 1024, 0.50, 8, 4), (257, 333, 3200, 0.05, 128, None),
    (2300, 256, 2432, 0.02, 8, None)])
def test_gate(T, D, F, p, W, cap):
    qx, qw = gate_inputs(T + D + F, T, D, F, p)
    h = tw.TwELL(T, F, W, spill_cap=cap)
    z = torch.empty((T, F), dtype=F32, device="cuda")
    tw.twell_gate_pack_fp8(qx.q, qx.scale, qw.q, qw.scale, h, z_debug=z)
    torch.cuda.synchronize()
    check_product(z, qx, qw, 128)
    full = tw.FLAG_SPILL_FULL if cap is not None else 0
    assert int(h.status.item()) == full
    ref = oracle.twell_pack(z.cpu().numpy(), 128, W)
    if cap is None:
        assert_twell_equal(fetch_twell(h), ref)
    else:
        np.testing.assert_array_equal(h.cnt.cpu().numpy().astype(np.int64), ref.cnt)
    # the union bitmap of each block of 128 rows
    act = (z > 0).cpu().numpy()
    bits = h.block_bits.cpu().numpy().view(np.uint32)
    for b in range((T + 127) // 128):
        any_ = act[b * 128:(b + 1) * 128].any(0).reshape(-1, 32)
        want = (any_.astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(1)
        np.testing.assert_array_equal(bits[b].astype(np.uint64), want)


def test_gate_with_a_ragged_last_round():
    test_gate(2500, 4100, 2048, 0.02, 8, None)


def test_gate_feeds_the_ffn():
    # norm -> 8-bit gate -> up/down, against the dense definition on the operands'
    # values in 64 bits
    g = _gen(21)
    T, D, F = 200, 256, 1024
    x = _randn(g, T, D)
    wn = torch.ones(D, device="cuda")
    o = tw.twell_rms_norm(x, wn, fp8=True)
    qw = tw.twell_quant_fp8(_randn(g, F, D) / 16 - 0.01, block_rows=128)
    wu, wd = (_randn(g, F, D) / 16).to(BF16), (_randn(g, F, D) / 32).to(BF16)
    h = tw.TwELL(T, F, 64)
    tw.twell_gate_pack_fp8(o.q, o.scale, qw.q, qw.scale, h)
    y = tw.twell_ffn_fwd(o.y, h, wu, wd)
    a = o.q.float().double() * spread(o.scale, 1, T, D)
    b = qw.q.float().double() * spread(qw.scale, 128, F, D)
    ref = ((a @ b.t()).clamp_min(0) * (o.y.double() @ wu.double().t())) @ wd.double()
    assert float((y.double() - ref).abs().max()) <= 1e-5 * float(ref.abs().max())
    assert int(h.status.item()) == 0


@pytest.mark.parametrize("T,D,F", [(16, 2048, 1024), (300, 2048, 1024), (4096, 512, 4096)])
def test_gate_wait_that_runs_out(T, D, F):
    qx, qw = gate_inputs(30, T, D, F, 0.02)
    h = tw.TwELL(T, F, 8)
    prev = tw.twell_gate_pack_wait_limit(5)
    try:
        tw.twell_gate_pack_fp8(qx.q, qx.scale, qw.q, qw.scale, h)
        torch.cuda.synchronize()
    finally:
        tw.twell_gate_pack_wait_limit(prev)
    assert int(h.status.item()) & tw.FLAG_TIMEOUT
    h.status.zero_()
    z = torch.empty((T, F), dtype=F32, device="cuda")
    tw.twell_gate_pack_fp8(qx.q, qx.scale, qw.q, qw.scale, h, z_debug=z)
    assert_twell_equal(fetch_twell(h), oracle.twell_pack(z.cpu().numpy(), 128, 8))
    assert int(h.status.item()) == 0


def test_refusals():
    qa, qb = operands(_gen(40), 16, 256, 256, 128)
    a, sa, b, sb = qa.q, qa.scale, qb.q, qb.scale
    with pytest.raises(TypeError):
        tw.twell_gemm_fp8(a.float(), sa, b, sb)
    with pytest.raises(TypeError):
        tw.twell_gemm_fp8(a, sa.double(), b, sb)
    with pytest.raises(ValueError):
        tw.twell_gemm_fp8(a[:, :240], sa, b, sb)
    with pytest.raises(ValueError):
        tw.twell_gemm_fp8(a, sa[:, :1], b, sb)
    with pytest.raises(ValueError):
        tw.twell_gemm_fp8(a, sa, b, sb[:1])
    with pytest.raises(ValueError):
        tw.twell_gemm_fp8(a[:, 8:136], sa[:, :1].contiguous(), b[:, 8:136],
                          sb[:, :1].contiguous())      # rows off 16-byte boundaries
    with pytest.raises(ValueError):
        tw.twell_gemm_fp8(a, sa, b, sb, out=torch.empty((16, 255), dtype=BF16, device="cuda"))
    with pytest.raises(TypeError):
        tw.twell_gemm_fp8(a, sa, b, sb, out=torch.empty((16, 256), dtype=torch.half,
                                                        device="cuda"))
    with pytest.raises(ValueError):
        tw.twell_quant_fp8(torch.zeros((4, 64), device="cuda"), block_rows=64)
    with pytest.raises(TypeError):
        tw.twell_quant_fp8(torch.zeros((4, 64), dtype=torch.half, device="cuda"))
    with pytest.raises(ValueError):
        tw.twell_quant_fp8(torch.zeros((4, 64), device="cuda"), rows=False)
    h = tw.TwELL(16, 256, 8)
    with pytest.raises(ValueError):
        tw.twell_gate_pack_fp8(a, sa, b, sb, tw.TwELL(15, 256, 8))
    with pytest.raises(ValueError):
        tw.twell_gate_pack_fp8(a, sa, b, sb[:1], h)
    h.struct.width = 0
    with pytest.raises(tw.TwellError):
        tw.twell_gate_pack_fp8(a, sa, b, sb, h)
