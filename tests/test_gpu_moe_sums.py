"""What the mixture-of-experts layer keeps of its last product: h in all of its 24 bits, sums in
fp32 however many neurons there are, infinities of W_d."""
import numpy as np
import pytest
import torch

import activation_sparse_gated_gate_gb300 as tw
from tests._gpu import ensure_built
from tests.test_gpu_moe import f64, layer, tokens, values

pytestmark = pytest.mark.gpu
U = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def held(w, bits, group=32, scale=1.0):
    """Integers -8 .. 7 [E][F][D] times a power of two, exact in either form."""
    if bits == 16:
        return (w * scale).to(torch.bfloat16).cuda()
    *lead, D = w.shape
    s = torch.full((*lead, -(-D // group)), scale, device="cuda")
    return tw.Int4.of_codes((w + 8).to(torch.uint8).cuda(), s, group=group)


def routed(T, D, w, x, dtype):
    ids = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    return tw.twell_moe_decode(x, None, *w, ids=ids, weights=torch.ones((T, 1), device="cuda"),
                               dtype=dtype).y


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("T,D", [(1, 8), (8, 136), (20, 64)])
def test_all_bits_of_h(T, D, bits, dtype):
    """Two neurons whose h differ in the last of 22 bits, one added and one taken off: every
    product and sum is exact, and so is y = 2^-21, which is one bf16 too."""
    x = torch.zeros((T, D))
    x[:, 0], x[:, 1], x[:, 2] = 1.0, 2.0 ** -10, 2.0 ** -11
    wg, wu, wd = (torch.zeros((1, 2, D)) for _ in range(3))
    wg[0, 0, :2] = 1                       # z = 1 + 2^-10, v = 1 + 2^-11
    wu[0, 0, 0] = wu[0, 0, 2] = 1
    wg[0, 1, 0] = 1                        # z = 1, v = 1 + 2^-10 + 2^-11
    wu[0, 1, :3] = 1
    wd[0, 0], wd[0, 1] = 1, -1
    y = routed(T, D, [held(v, bits) for v in (wg, wu, wd)], x.to(torch.bfloat16).cuda(), dtype)
    assert (y.double() == 2.0 ** -21).all()


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("act", ["relu", "silu"])
@pytest.mark.parametrize("T,E,k,F,D", [(1, 16, 8, 1024, 2048), (8, 16, 4, 300, 1000),
                                       (64, 16, 8, 512, 2048)])
def test_bf16_is_the_rounded_fp32(T, E, k, F, D, act, bits):
    """y's type decides how y is rounded and nothing else."""
    r, w = layer(E, F, D, bits, seed=T, group=128)
    x = tokens(T, D)
    a = tw.twell_moe_decode(x, r, *w, top_k=k, act=act, dtype=torch.float32)
    b = tw.twell_moe_decode(x, r, *w, top_k=k, act=act, dtype=torch.bfloat16)
    assert torch.equal(a.y.to(torch.bfloat16), b.y)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("sign", ["same", "any"])
@pytest.mark.parametrize("T,k", [(256, 8), (256, 2), (16, 1)])
@pytest.mark.parametrize("F", [1024, 2048, 14336])
def test_sums_over_many_neurons(F, T, k, sign, bits):
    """z, v and h are exact but for h's own rounding, so that y's error is the last product's.
    In units of 2^-23 of the sums: h's rounding 1/2; a step of 16 neurons is three products of
    the tensor core, whose sums truncate, 6 at the most.  Then n = F / 16 steps are added in fp32.
    Of one sign: the i-th sum is about i / n of the whole, each addition rounds by at most 1/2 of
    its own, (n + 1) / 4 together, and no less can be promised, because these h stand on a grid
    (the first row's are multiples of 2^-6 and a little more) and may all be rounded the same
    way: 8 + n / 4.  (One chain of truncating additions is off by about 1/3 an addition and three
    a step, always downwards: n / 2 and more.)  Of either sign, sums meet the grid anywhere:
    0.29 sqrt(n / 2) in the mean square, held against twice that, 8 + 0.6 sqrt(n).  T and k decide
    how many warps stand side by side on columns, and so how long a warp's sums are: all of F
    with the largest."""
    D, g = 4096, torch.Generator().manual_seed(F + T)
    x = torch.zeros((T, D))
    x[:, 0], x[:, 1] = 1.0, 2.0 ** -9

    def positive():
        return torch.randint(8, 16, (1, F, D), generator=g, dtype=torch.int8)

    def half(v):   # integers in 1 .. 7 in 4 bits
        return (v / 2).floor().clamp(1, 7) if bits == 4 else v.float()

    wg, wu, wd = half(positive()), half(positive()), half(positive())
    if sign == "any":
        wd *= 1 - 2 * torch.randint(0, 2, wd.shape, generator=g)
    w = [held(v, bits, 128, s) for v, s in ((wg, 2.0 ** -3), (wu, 2.0 ** -3), (wd, 2.0 ** -6))]
    x[:, 1] *= torch.arange(1, T + 1) / 256
    x = x.to(torch.bfloat16).cuda()
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    rows = [0, 1, T // 2, T - 1]
    ids[rows, 0] = 0
    y = tw.twell_moe_decode(x, None, *w, ids=ids, weights=torch.ones((T, k), device="cuda")).y
    g64, u64, d64 = (torch.from_numpy(values(v)[0]) for v in w)
    xd = x[rows].double().cpu()
    h = (xd @ g64.t()) * (xd @ u64.t())
    ref = h @ d64
    err = (y[rows].double().cpu() - ref).norm(dim=1) / ref.norm(dim=1)
    n = F / 16
    assert (err <= (8 + (n / 4 if sign == "same" else 0.6 * n ** 0.5)) * U).all(), err / U


@pytest.mark.parametrize("bits,size", [(4, 1.0), (16, 1.0), (16, 2.0 ** -65), (16, 2.0 ** -74)])
@pytest.mark.parametrize("act", ["relu", "silu"])
@pytest.mark.parametrize("T,F", [(1, 5), (3, 40), (20, 33)])
def test_infinities_of_wd(T, F, act, bits, size):
    """An infinity in W_d times an h that is not zero is one in y, whatever the number of
    neurons and however few bits h has, h of 2^-130 and 2^-148 among them.  (In 4 bits:
    of a scale, with codes of zero a NaN by the formula.)  Elsewhere y is as it was: parts of
    h are multiples of 2^-133, so that three may be 3 2^-133 off, and SiLU is good to 16 u."""
    D, g = 256, torch.Generator().manual_seed(T)
    x = torch.zeros((T, D))
    x[:, 0] = 1.0                                   # z and v are column 0 of the weights
    wg = torch.randint(1, 8, (1, F, D), generator=g).float()
    wu = wg.flip(1) * (1 - 2 * torch.randint(0, 2, (1, F, D), generator=g))
    wd = torch.randint(-7, 8, (1, F, D), generator=g).float()
    w = [held(wg, bits, 64, size), held(wu, bits, 64, size), held(wd, bits, 64)]
    if bits == 16:
        w[2][0, F - 1, 3] = float("inf")
        w[2][0, 2, 9] = -float("inf")
        w[2][0, 0, 11] = w[2][0, 1, 11] = float("inf")
    else:
        w[2].scale[0, F - 1, 0] = float("inf")
        w[2].scale[0, 2, 2] = -float("inf")
    x = x.to(torch.bfloat16).cuda()
    ids = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    y = tw.twell_moe_decode(x, None, *w, act=act, ids=ids,
                            weights=torch.ones((T, 1), device="cuda")).y
    with np.errstate(all="ignore"):
        g64, u64, d64 = (values(v)[0] for v in w)
        z, v = f64(x) @ g64.T, f64(x) @ u64.T
        h = (z if act == "relu" else z / (1 + np.exp(-z))) * v
        ref = (h[:, :, None] * d64).sum(1)
        tol = ((16 + F) * U * np.abs(h) + 3 * 2.0 ** -133) @ np.nan_to_num(np.abs(d64), posinf=0.0)
    got = f64(y)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    there = np.isinf(ref)
    assert there.any() and np.array_equal(got[there], ref[there])
    some = np.isfinite(ref)
    assert (np.abs(got[some] - ref[some]) <= tol[some] + 2.0 ** -149).all()
