"""Weights in 4 bits: quantisation, values and few-row products against 64-bit arithmetic
from the definition.

Tolerances.  Codes, scales, zero points and fp32 values are exact.  A product's sums are
fp32: the products of a bf16 and a 4-bit integer are exact in them, so with S = sum_k |w x|
over K terms an fp32 result is within (K + 8) 2^-23 S of the exact one (a term of at
most one ulp for each addition, and the scale's product), and a bf16 result within half a bf16
step, 2^-8 of it, more.
"""
import numpy as np
import pytest
import torch

import activation_sparse_gated_gate_gb300 as tw
from tests._gpu import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def weights(rows, K, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn((rows, K), generator=g) * torch.exp(0.5 * torch.randn((rows, 1), generator=g))
    w = torch.where(torch.rand(w.shape, generator=g) < 0.01, 8 * w, w)
    return w.to(dtype)


def bf16(v):
    return torch.from_numpy(np.asarray(v, np.float32)).to(torch.bfloat16).double().numpy()


def quantised(w, group, zero_points):
    """(codes, scale, zero) of w (fp64 array) by the definition."""
    rows, K = w.shape
    n = -(-K // group)
    codes = np.empty((rows, K))
    scale, zero = np.empty((rows, n)), np.full((rows, n), 8.0)
    for j in range(n):
        v = w[:, j * group:(j + 1) * group]
        if zero_points:
            lo, hi = np.minimum(v.min(1), 0), np.maximum(v.max(1), 0)
            s = bf16(np.float32(hi - lo).astype(np.float64) / 15)
        else:
            s = bf16(np.abs(v).max(1) / 7)
        live = s > 0
        d = np.where(live, s, 1.0)
        if zero_points:
            z = np.where(live, np.clip(np.rint(-lo / d), 0, 15), 8)
            q = np.clip(np.rint(v / d[:, None]) + z[:, None], 0, 15)
            zero[:, j] = z
        else:
            q = np.clip(np.rint(v / d[:, None]), -8, 7) + 8
        codes[:, j * group:(j + 1) * group] = np.where(live[:, None], q, 8)
        scale[:, j] = s
    return codes, scale, zero


def wide(codes, scale, zero, group):
    j = np.arange(codes.shape[1]) // group
    return (codes - zero[:, j]) * scale[:, j]


def check_quant(w, group, zero_points, src=None):
    src = w if src is None else src
    q = tw.twell_quant_int4(src.cuda() if not src.is_cuda else src, group=group,
                            zero_points=zero_points)
    codes, scale, zero = quantised(w.double().cpu().numpy(), group, zero_points)
    n = scale.shape[1]
    np.testing.assert_array_equal(q.scale[:, :n].double().cpu().numpy(), scale)
    assert not q.scale[:, n:].float().any()
    if zero_points:
        np.testing.assert_array_equal(q.zero[:, :n].cpu().numpy(), zero)
        assert (q.zero[:, n:] == 8).all()
    else:
        assert q.zero is None
    np.testing.assert_array_equal(q.codes().cpu().numpy(), codes)
    v = wide(codes, scale, zero, group)
    np.testing.assert_array_equal(
        tw.twell_dequant_int4(q, dtype=torch.float32).double().cpu().numpy(), v)
    assert torch.equal(tw.twell_dequant_int4(q).cpu(), torch.from_numpy(v).to(torch.bfloat16))
    return q


@pytest.mark.parametrize("zero_points", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 7), (5, 8), (17, 40), (33, 128), (2, 129),
                                    (64, 200), (9, 1000), (130, 2048), (7, 1999)])
def test_quant(rows, K, dtype, group, zero_points):
    check_quant(weights(rows, K, rows + K, dtype), group, zero_points)


@pytest.mark.parametrize("zero_points", [False, True])
@pytest.mark.parametrize("off,pitch", [(0, 264), (1, 264), (8, 264), (0, 257)])
def test_quant_strided(off, pitch, zero_points):
    full = weights(20, pitch + off, 3)
    w = full[:, off:off + 248]
    check_quant(w, 64, zero_points, full.cuda()[:, off:off + 248])


@pytest.mark.parametrize("K", [128, 250])
@pytest.mark.parametrize("zero_points", [False, True])
def test_quant_ties_and_small(zero_points, K):
    """Quotients that are ties or one ulp beside them, scales that are subnormal, groups of
    zeros, values of one sign."""
    w = torch.zeros((12, K))
    step = torch.arange(K) % 15 - 7
    w[0] = 0.5 * step                       # scale 0.5: halves of codes are ties
    w[0, 1::2] += 0.25
    w[1] = w[0] * (1 + 2.0 ** -23)
    w[2] = w[0] * (1 - 2.0 ** -24)
    w[3] = w[0] * 3
    w[4] = step * 2.0 ** -126               # scales near bf16's smallest
    w[5] = step * 1.4 * 2.0 ** -133
    w[6] = step * 2.0 ** -149
    w[7] = step.abs() + 1                   # one sign
    w[8] = -w[7]
    w[9, 5] = 1e-3
    w[10] = step * 2.0 ** 120
    check_quant(w, 32, zero_points)
    check_quant(w, 128, zero_points)


@pytest.mark.parametrize("K", [256, 255])
@pytest.mark.parametrize("zero_points", [False, True])
def test_quant_not_finite(zero_points, K):
    w = weights(6, K, 5)
    w[0, 3], w[1, 40], w[2, 100] = float("nan"), float("inf"), float("-inf")
    q = tw.twell_quant_int4(w.cuda(), group=32, zero_points=zero_points)
    v = tw.twell_dequant_int4(q, dtype=torch.float32).cpu()
    bad = torch.zeros(6, K, dtype=torch.bool)
    bad[0, :32] = bad[1, 32:64] = bad[2, 96:128] = True
    assert torch.equal(v.isnan(), bad)
    w[bad] = 0.0
    ref = tw.twell_dequant_int4(tw.twell_quant_int4(w.cuda(), group=32, zero_points=zero_points),
                                dtype=torch.float32).cpu()
    assert torch.equal(v[~bad], ref[~bad])


def test_quant_experts_out_and_codes():
    w = weights(6 * 10, 300, 9).view(6, 10, 300).cuda()
    q = tw.twell_quant_int4(w, group=64, zero_points=True)
    assert q.shape == (6, 10, 300) and q.code.shape == (6, 10, 192)
    flat = tw.twell_quant_int4(w.view(60, 300), group=64, zero_points=True)
    assert torch.equal(q.code.view(60, 192), flat.code)
    again = tw.twell_quant_int4(2 * w, group=64, zero_points=True, out=q)
    assert again is q and torch.equal(q.scale.float().view(60, -1), 2 * flat.scale.float())
    back = tw.Int4.of_codes(flat.codes(), flat.scale[:, :5], flat.zero[:, :5], group=64)
    for a, b in zip(back, flat):
        assert a == b if isinstance(a, int) else torch.equal(a, b)
    v = tw.twell_dequant_int4(q)
    out = torch.empty((60, 320), dtype=torch.bfloat16, device="cuda")[:, :300]
    tw.twell_dequant_int4(tw.Int4(flat.code, q.scale.view(60, -1), flat.zero, 300, 64), out=out)
    assert torch.equal(out, v.view(60, 300))


def check_gemv(x, q, dtype, out=None):
    y = tw.twell_gemv_int4(x, q, out=out, dtype=dtype)
    j = np.arange(q.K) // q.group
    z = 8.0 if q.zero is None else q.zero.double().cpu().numpy()[:, j]
    w = (q.codes().double().cpu().numpy() - z) * q.scale.double().cpu().numpy()[:, j]
    xd = x.double().cpu().numpy()
    ref, size = xd @ w.T, np.abs(xd) @ np.abs(w).T
    tol = (q.K + 8) * 2.0 ** -23 * size
    if dtype is torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    got = y.double().cpu().numpy()
    assert got.shape == ref.shape and (np.abs(got - ref) <= tol).all()
    return y


@pytest.mark.parametrize("group,zero_points", [(32, False), (32, True), (64, True), (128, False),
                                               (128, True)])
@pytest.mark.parametrize("T,N,K", [(1, 1, 1), (1, 16, 128), (2, 40, 100), (3, 17, 1000),
                                   (7, 64, 2048), (8, 129, 264), (9, 33, 513), (16, 100, 640),
                                   (17, 65, 1999), (31, 200, 256), (33, 70, 1024), (64, 130, 384),
                                   (65, 20, 128), (200, 48, 320)])
def test_gemv(T, N, K, group, zero_points):
    q = tw.twell_quant_int4(weights(N, K, T + N).cuda(), group=group, zero_points=zero_points)
    x = weights(T, K, 7, torch.bfloat16).cuda()
    check_gemv(x, q, torch.float32)
    check_gemv(x, q, torch.bfloat16)


@pytest.mark.parametrize("T,N", [(1, 8001), (2, 30007), (9, 30007), (16, 20000), (20, 8001),
                                 (33, 20000)])
def test_gemv_many_rows(T, N):
    """Few warps share K, blocks run one after the other."""
    K = 1100
    q = tw.twell_quant_int4(weights(N, K, N).cuda(), group=128)
    check_gemv(weights(T, K, 3, torch.bfloat16).cuda(), q, torch.float32)


@pytest.mark.parametrize("K,off,pitch", [(256, 0, 264), (256, 8, 264), (256, 1, 260), (250, 2, 252)])
@pytest.mark.parametrize("T", [1, 12, 40])
def test_gemv_strided(T, K, off, pitch):
    q = tw.twell_quant_int4(weights(50, K, 1).cuda(), group=32, zero_points=True)
    full = weights(T, pitch + off, 2, torch.bfloat16).cuda()
    out = torch.full((T, 60), 7.0, device="cuda")
    check_gemv(full[:, off:off + K], q, torch.float32, out=out[:, 3:53])
    assert (out[:, :3] == 7).all() and (out[:, 53:] == 7).all()


def test_gemv_empty_and_repeat():
    q = tw.twell_quant_int4(weights(300, 1030, 1).cuda(), group=64)
    assert tw.twell_gemv_int4(torch.empty((0, 1030), dtype=torch.bfloat16, device="cuda"),
                              q).shape == (0, 300)
    none = tw.twell_quant_int4(torch.empty((0, 64), device="cuda"))
    x = weights(20, 1030, 4, torch.bfloat16).cuda()
    assert tw.twell_gemv_int4(x[:, :64].contiguous(), none).shape == (20, 0)
    y = tw.twell_gemv_int4(x, q, dtype=torch.float32)
    for _ in range(3):
        assert torch.equal(tw.twell_gemv_int4(x, q, dtype=torch.float32), y)


def test_gemv_not_finite():
    """Infinities and NaN of a row of x stay in its row, those of a group in its columns."""
    w = weights(64, 256, 8)
    q = tw.twell_quant_int4(w.cuda(), group=32)
    x = weights(4, 256, 9, torch.bfloat16).cuda()
    y = tw.twell_gemv_int4(x, q, dtype=torch.float32)
    x[1, 200] = float("nan")
    w[5, 17] = float("inf")
    bad = tw.twell_gemv_int4(x, tw.twell_quant_int4(w.cuda(), group=32), dtype=torch.float32)
    nan = torch.zeros((4, 64), dtype=torch.bool, device="cuda")
    nan[1], nan[:, 5] = True, True
    assert torch.equal(bad.isnan(), nan) and torch.equal(bad[~nan], y[~nan])


def test_gemv_streams_and_graph():
    q = tw.twell_quant_int4(weights(256, 512, 1).cuda())
    x = weights(4, 512, 2, torch.bfloat16).cuda()
    ref = tw.twell_gemv_int4(x, q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = tw.twell_gemv_int4(x, q, stream=s)
    s.synchronize()
    assert torch.equal(y, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tw.twell_gemv_int4(x, q)
    x.copy_(weights(4, 512, 3, torch.bfloat16))
    graph.replay()
    assert torch.equal(out, tw.twell_gemv_int4(x, q))


def test_refusals():
    w = torch.randn((6, 64), device="cuda")
    q = tw.twell_quant_int4(w, group=32, zero_points=True)
    x = torch.randn((2, 64), device="cuda").to(torch.bfloat16)

    def bad(error, f, *a, **k):
        with pytest.raises(error):
            f(*a, **k)

    bad(TypeError, tw.twell_quant_int4, w.half())
    bad(TypeError, tw.twell_quant_int4, w.cpu())
    bad(ValueError, tw.twell_quant_int4, w[0])
    bad(ValueError, tw.twell_quant_int4, w.t())
    bad(ValueError, tw.twell_quant_int4, w[:, :0])
    bad(ValueError, tw.twell_quant_int4, w, group=16)
    bad(ValueError, tw.twell_quant_int4, w, group=64, out=q)
    bad(ValueError, tw.twell_quant_int4, w, group=32, out=q)
    bad(ValueError, tw.twell_quant_int4, w[:5], group=32, zero_points=True, out=q)
    bad(ValueError, tw.twell_quant_int4, w.view(2, 3, 64)[:, :2], group=32)
    bad(TypeError, tw.twell_dequant_int4, w)
    bad(TypeError, tw.twell_dequant_int4, q, dtype=torch.float16)
    bad(ValueError, tw.twell_dequant_int4, q, out=torch.empty((6, 63), device="cuda"))
    bad(TypeError, tw.twell_gemv_int4, x.float(), q)
    bad(TypeError, tw.twell_gemv_int4, x, w)
    bad(ValueError, tw.twell_gemv_int4, x[:, :32], q)
    bad(ValueError, tw.twell_gemv_int4, x[0], q)
    bad(ValueError, tw.twell_gemv_int4, x, tw.twell_quant_int4(w.view(2, 3, 64), group=32))
    bad(TypeError, tw.twell_gemv_int4, x, q, dtype=torch.float16)
    bad(ValueError, tw.twell_gemv_int4, x, q, out=torch.empty((2, 5), device="cuda"))
    bad(ValueError, tw.twell_gemv_int4, x, q._replace(scale=q.scale[:, :1]))
    bad(TypeError, tw.twell_gemv_int4, x, q._replace(scale=q.scale.float()))
    bad(TypeError, tw.twell_gemv_int4, x, q._replace(zero=q.zero.int()))
    bad(ValueError, tw.twell_gemv_int4, x, q._replace(code=q.code[:, :32]))
    bad(ValueError, tw.twell_gemv_int4, x, q._replace(group=20))
    bad(TypeError, tw.twell_gemv_int4, x, q._replace(code=q.code.cpu()))
    bad(TypeError, tw.twell_gemv_int4, x, tuple(q))
    bad(TypeError, tw.twell_dequant_int4, tuple(q))
    bad(TypeError, tw.twell_quant_int4, w, group=32, zero_points=True, out=tuple(q))
    bad(ValueError, tw.twell_gemv_int4, x, q._replace(K=64.0))
    held = torch.empty((6 * 64 + 8,), dtype=torch.uint8, device="cuda")
    bad(tw.TwellError, tw.twell_gemv_int4, x, q._replace(code=held[8:].view(6, 64)))
    assert tw.twell_gemv_int4(x, q).isfinite().all()


def test_more_than_2_31_bytes():
    """Rows behind 2^31 bytes of codes and 2^31 elements of values."""
    N, K = 70000, 65536
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("needs 24 GB")
    w = torch.zeros((N, K), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    w[-40:] = torch.randn((40, K), generator=g, device="cuda").to(torch.bfloat16)
    q = tw.twell_quant_int4(w, group=64)
    last = tw.twell_quant_int4(w[-40:].contiguous(), group=64)
    assert torch.equal(q.code[-40:], last.code) and torch.equal(q.scale[-40:], last.scale)
    x = torch.randn((3, K), generator=g, device="cuda").to(torch.bfloat16)
    y = tw.twell_gemv_int4(x, q, dtype=torch.float32)
    del w
    check_gemv(x, last, torch.float32)
    ref = tw.twell_gemv_int4(x, last, dtype=torch.float32)
    assert torch.allclose(y[:, -40:], ref, rtol=1e-5, atol=1e-5 * float(ref.abs().max()))
    assert not y[:, :-40].any()
    v = tw.twell_dequant_int4(q)
    assert torch.equal(v[-40:], tw.twell_dequant_int4(last)) and not v[:1000].any()
