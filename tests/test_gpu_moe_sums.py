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
