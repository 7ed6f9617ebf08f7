"""Residual addition with root-mean-square norm, forward and backward, against
plain 64-bit implementations.

Tolerances, with e = 2^-24 (an fp32 rounding), b = 2^-8 (a bf16 rounding: eight
significant bits):
the sum of D squares is off by at most (D + 2) e relative (any order), rstd by
half of that and a few roundings, so n = s rstd and y by (D/2 + 8) e |y|, and a
bf16 result by b |result| more.  dx sums D terms g n: (D + 16) e times the
terms' magnitudes.  dw sums T terms: (T + 16) e sum |dy n|.  e4m3 keeps three
bits below the leading one (half a unit is 2^-4 relative, 2^-10 absolute below
2^-6), plus the fp32 roundings of y and of the scale."""
import numpy as np
import pytest
import torch

import activation_sparse_gated_gate_gb300 as tw
from _gpu import ensure_built

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
B = 2.0 ** -8
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def plain_norm(x, w, r, eps):
    s = x.double() if r is None else x.double() + r.double()
    rstd = 1.0 / torch.sqrt((s * s).sum(1) / s.shape[1] + eps)
    return s, rstd, s * rstd[:, None] * w.double()


def check_e4m3(q, scale, v):
    """q [R][C] e4m3 and scale per 1 x 128 of v (64 bits, off by at most its
    fp32 rounding)."""
    R, C = v.shape
    nb = -(-C // 128)
    p = torch.zeros((R, nb * 128), dtype=torch.float64, device=v.device)
    p[:, :C] = v.abs()
    amax = p.view(R, nb, 128).amax(2).clamp_min(2.0 ** -64)
    rel = (C + 16) * E
    assert ((scale.double() - amax / 448).abs() <= rel * amax / 448).all()
    t = v / scale.double().repeat_interleave(128, 1)[:, :C]
    got = q.float().double()
    half = torch.maximum(t.abs() * 2.0 ** -4, torch.full_like(t, 2.0 ** -10))
    assert ((got - t).abs() <= half * (1 + 1e-6) + t.abs() * 2 * rel).all()


SHAPES = [(1, 1), (1, 2048), (3, 7), (5, 64), (2, 130), (4, 256), (64, 257), (33, 1001),
          (300, 1536), (17, 2304), (7, 4096), (3, 8200), (2, 9216), (2, 16383), (2, 16384)]


@pytest.mark.parametrize("T,D", SHAPES)
@pytest.mark.parametrize("xt,rt,wt", [(BF16, BF16, BF16), (F32, F32, F32), (F32, BF16, BF16),
                                      (BF16, F32, F32), (BF16, None, F32), (F32, None, BF16)])
def test_forward(T, D, xt, rt, wt):
    g = _gen(T * 100003 + D)
    x = _randn(g, T, D).to(xt)
    r = None if rt is None else (3 * _randn(g, T, D)).to(rt)
    w = (1 + 0.1 * _randn(g, D)).to(wt)
    o = tw.twell_rms_norm(x, w, residual=r, eps=1e-5, fp8=True, rstd=True)
    s, rstd, y = plain_norm(x, w, r, 1e-5)
    if r is None:
        assert o.total is None
    else:
        assert o.total.dtype == rt
        torch.testing.assert_close(o.total, (x.float() + r.float()).to(rt), rtol=0, atol=0)
    rel = (D / 2 + 8) * E
    assert ((o.rstd.double() - rstd).abs() <= rel * rstd).all()
    assert ((o.y.double() - y).abs() <= (B * (1 + rel) + rel) * y.abs() + 1e-40).all()
    assert o.q.shape == (T, D) and (T == 1 or o.q.stride(0) % 16 == 0)
    check_e4m3(o.q, o.scale, y)


def test_only_what_is_asked_for():
    g = _gen(1)
    x, w = _randn(g, 6, 256), torch.ones(256, device="cuda")
    o = tw.twell_rms_norm(x, w)
    assert o.total is o.q is o.scale is o.rstd is None and o.y.dtype == BF16
    o8 = tw.twell_rms_norm(x, w, bf16=False, fp8=True)
    assert o8.y is None
    check_e4m3(o8.q, o8.scale, plain_norm(x, w, None, 1e-6)[2])


def test_rows_apart_and_in_place():
    # x a slice of wider rows (an odd offset, so element by element), the
    # residual updated in place inside a wider buffer, y into a slice
    g = _gen(2)
    T, D = 37, 192
    for off in (0, 1, 8):
        wide = _randn(g, T, 3 * D + 16).to(BF16)
        x = wide[:, off:off + D]
        buf = _randn(g, T, D + 64)
        before = buf.clone()
        r = buf[:, 32:32 + D]
        w = 1 + 0.1 * _randn(g, D)
        s, _, y = plain_norm(x, w, r, 1e-6)
        ybuf = torch.full((T, 2 * D), 7.0, dtype=BF16, device="cuda")
        want = (x.float() + r).clone()
        tw.twell_rms_norm(x, w, residual=r, total=r, y=ybuf[:, D:])
        torch.testing.assert_close(buf[:, 32:32 + D], want, rtol=0, atol=0)
        assert (buf[:, :32] == before[:, :32]).all() and (buf[:, -32:] == before[:, -32:]).all()
        assert (ybuf[:, :D] == 7.0).all()
        rel = (D / 2 + 8) * E
        assert ((ybuf[:, D:].double() - y).abs() <= (B + 2 * rel) * y.abs()).all()


def test_zero_rows_tiny_and_huge_values():
    D = 384
    x = torch.zeros((6, D), device="cuda")
    x[1] = 1e-25                      # squares underflow: eps alone is left
    x[2, 5] = 1e18                    # squares near fp32's top
    x[3, ::2] = -3e-3
    x[4] = 2.0 ** -70
    x[5, 300:] = 1.0
    w = torch.ones(D, device="cuda")
    o = tw.twell_rms_norm(x, w, fp8=True, rstd=True)
    s, rstd, y = plain_norm(x, w, None, 1e-6)
    assert ((o.rstd.double() - rstd).abs() <= (D + 8) * E * rstd).all()
    assert ((o.y.double() - y).abs() <= 1.01 * B * y.abs() + 1e-38).all()
    assert (o.q[0].float() == 0).all() and torch.isfinite(o.scale).all()
    check_e4m3(o.q, o.scale, y)


def test_a_bad_row_stays_in_its_row():
    g = _gen(3)
    x, w = _randn(g, 5, 256), torch.ones(256, device="cuda")
    good = tw.twell_rms_norm(x, w, fp8=True, rstd=True)
    x[1, 17] = float("nan")
    x[3, 200] = float("inf")
    o = tw.twell_rms_norm(x, w, fp8=True, rstd=True)
    for t in (0, 2, 4):
        assert (o.y[t] == good.y[t]).all() and (o.scale[t] == good.scale[t]).all()
        assert (o.q[t].float() == good.q[t].float()).all()
    assert torch.isnan(o.y[1]).all() and torch.isnan(o.q[1].float()).all()
    assert torch.isnan(o.y[3, 200]) and (o.y[3, :200] == 0).all()


def plain_bwd(s, w, rstd, dy, dt):
    s, w, rstd, dy = s.double(), w.double(), rstd.double()[:, None], dy.double()
    n, g = s * rstd, dy * w
    dx = rstd * (g - n * (g * n).sum(1, keepdim=True) / s.shape[1])
    scale = rstd * (g.abs() + n.abs() * (g * n).abs().sum(1, keepdim=True) / s.shape[1])
    if dt is not None:
        dx, scale = dx + dt.double(), scale + dt.double().abs()
    return dx, scale, (dy * n).sum(0), (dy * n).abs().sum(0)


@pytest.mark.parametrize("T,D", [(1, 1), (1, 2048), (3, 7), (5, 64), (700, 130), (4, 256),
                                 (1000, 257), (777, 1001), (3001, 1536), (517, 2304), (7, 4096),
                                 (165, 8192), (3, 8200), (2, 9216), (200, 16383), (2, 16384)])
@pytest.mark.parametrize("st,gt,wt,stream", [(BF16, BF16, BF16, True), (F32, BF16, F32, True),
                                             (F32, F32, F32, False), (BF16, F32, BF16, False)])
def test_backward(T, D, st, gt, wt, stream):
    g = _gen(T * 100003 + D + 1)
    s = (2 * _randn(g, T, D)).to(st)
    w = (1 + 0.1 * _randn(g, D)).to(wt)
    dy = _randn(g, T, D).to(gt)
    dt = _randn(g, T, D).to(st) if stream else None
    rstd = (1.0 / torch.sqrt((s.double() ** 2).mean(1) + 1e-6)).float()
    dx, dw = tw.twell_rms_norm_bwd(s, w, rstd, dy, dtotal=dt)
    rx, sx, rw, sw = plain_bwd(s, w, rstd, dy, dt)
    assert dx.dtype == st and dw.dtype == F32
    tol = (D + 16) * E * sx + (B * rx.abs() if st == BF16 else 0)
    assert ((dx.double() - rx).abs() <= tol + 1e-40).all()
    assert ((dw.double() - rw).abs() <= (T + 16) * E * sw + 1e-40).all()
    # the same bits again, and with dtotal's buffer as the output
    dx2, dw2 = tw.twell_rms_norm_bwd(s, w, rstd, dy, dtotal=dt, dx=None if dt is None else dt)
    assert (dx2 == dx).all() and (dw2 == dw).all()


# rows of many threads: either side of where a thread's share of a row and the
# rows in flight change, more rows than blocks and fewer
@pytest.mark.parametrize("T,D", [(1, 5120), (311, 5128), (460, 8192), (2, 8200), (333, 9216),
                                 (170, 10240), (170, 10248), (1001, 5632), (950, 8192),
                                 (800, 12288), (3, 12296)])
@pytest.mark.parametrize("st,gt,wt,stream", [(BF16, BF16, BF16, True), (F32, BF16, F32, True),
                                             (F32, F32, BF16, True), (BF16, F32, BF16, False)])
def test_backward_wide(T, D, st, gt, wt, stream):
    test_backward(T, D, st, gt, wt, stream)


@pytest.mark.parametrize("D", [2048, 6144, 9216, 12296])
def test_backward_over_dtotal(D):
    # dx may be dtotal's own memory: the same values as into another
    g = _gen(D)
    s, dy = 2 * _randn(g, 700, D), _randn(g, 700, D).to(BF16)
    w, dt = 1 + 0.1 * _randn(g, D), _randn(g, 700, D)
    rstd = (s.square().mean(1) + 1e-6).rsqrt()
    dx, dw = tw.twell_rms_norm_bwd(s, w, rstd, dy, dtotal=dt)
    again, dw2 = tw.twell_rms_norm_bwd(s, w, rstd, dy, dtotal=dt, dx=dt)
    assert again is dt and (dt == dx).all() and (dw == dw2).all()


def test_backward_against_differences():
    # central differences of L = sum(c y) + sum(d total) in 64 bits, through the
    # forward's definition; a step of 1e-5 leaves about 1e-9 relative
    g = _gen(11)
    T, D, eps = 3, 24, 1e-3
    x = _randn(g, T, D)
    w = 1 + 0.1 * _randn(g, D)
    c, d = _randn(g, T, D), _randn(g, T, D)
    rstd = plain_norm(x, w, None, eps)[1].float()
    dx, dw = tw.twell_rms_norm_bwd(x, w, rstd, c, dtotal=d)

    def loss(xx, ww):
        y = xx / torch.sqrt((xx * xx).mean(1, keepdim=True) + eps) * ww
        return float((c.double() * y).sum() + (d.double() * xx).sum())

    h = 1e-5
    for t in range(T):
        for j in range(D):
            e = torch.zeros((T, D), dtype=torch.float64, device="cuda")
            e[t, j] = h
            num = (loss(x.double() + e, w.double()) - loss(x.double() - e, w.double())) / (2 * h)
            assert abs(num - float(dx[t, j])) <= 2e-5 * (1 + abs(num))
    for j in range(D):
        e = torch.zeros(D, dtype=torch.float64, device="cuda")
        e[j] = h
        num = (loss(x.double(), w.double() + e) - loss(x.double(), w.double() - e)) / (2 * h)
        assert abs(num - float(dw[j])) <= 2e-5 * (1 + abs(num))


def test_no_rows():
    x = torch.empty((0, 96), device="cuda")
    w = torch.ones(96, device="cuda")
    o = tw.twell_rms_norm(x, w, residual=x.to(BF16), fp8=True, rstd=True)
    assert o.y.shape == (0, 96) and o.total.dtype == BF16 and o.scale.shape == (0, 1)
    dw = torch.full((96,), 5.0, device="cuda")
    dx, dw = tw.twell_rms_norm_bwd(x, w, o.rstd, o.y, dw=dw)
    assert dx.shape == (0, 96) and (dw == 0).all()


def test_another_stream():
    g = _gen(5)
    x, w = _randn(g, 512, 1536), torch.ones(1536, device="cuda")
    want = tw.twell_rms_norm(x, w, fp8=True, rstd=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = tw.twell_rms_norm(x, w, fp8=True, rstd=True, stream=side)
    dx, dw = tw.twell_rms_norm_bwd(x, w, got.rstd, got.y, stream=side)
    side.synchronize()
    assert (got.y == want.y).all() and (got.q.float() == want.q.float()).all()
    dx0, dw0 = tw.twell_rms_norm_bwd(x, w, want.rstd, want.y)
    assert (dx == dx0).all() and (dw == dw0).all()


def test_refusals():
    x, w = torch.zeros((4, 64), device="cuda"), torch.ones(64, device="cuda")
    with pytest.raises(TypeError):
        tw.twell_rms_norm(x.cpu(), w)
    with pytest.raises(TypeError):
        tw.twell_rms_norm(x.half(), w)
    with pytest.raises(TypeError):
        tw.twell_rms_norm(x, w.half())
    with pytest.raises(ValueError):
        tw.twell_rms_norm(x, w[:63])
    with pytest.raises(ValueError):
        tw.twell_rms_norm(x, w, residual=x[:3])
    with pytest.raises(ValueError):
        tw.twell_rms_norm(x, w, total=torch.empty_like(x))
    with pytest.raises(ValueError):
        tw.twell_rms_norm(x.t(), torch.ones(4, device="cuda"))
    with pytest.raises(ValueError):
        tw.twell_rms_norm(x, w, q=torch.empty((4, 64), dtype=torch.float8_e4m3fn, device="cuda"))
    with pytest.raises(ValueError):
        tw.twell_rms_norm(x, w, residual=x, total=torch.empty((4, 65), device="cuda"))
    with pytest.raises(tw.TwellError):
        tw.twell_rms_norm(x, w, eps=-1.0)
    with pytest.raises(tw.TwellError):
        tw.twell_rms_norm(x[:1].expand(4, 64), w)          # rows on top of each other
    with pytest.raises(tw.TwellError):
        tw.twell_rms_norm(torch.zeros((1, 16392), device="cuda"),
                          torch.ones(16392, device="cuda"))
    rstd = torch.ones(4, device="cuda")
    with pytest.raises(ValueError):
        tw.twell_rms_norm_bwd(x, w, rstd[:3], x)
    with pytest.raises(TypeError):
        tw.twell_rms_norm_bwd(x, w, rstd, x, dtotal=x.to(BF16))
    with pytest.raises(tw.TwellError):
        tw.twell_rms_norm_bwd(x, w, rstd, x, ws=torch.empty(4, dtype=torch.uint8, device="cuda"))
    # nothing above left the context in error
    assert np.isfinite(float(tw.twell_rms_norm(x, w).y.sum()))
