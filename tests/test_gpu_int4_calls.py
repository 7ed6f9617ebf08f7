"""Calls of the 4-bit and mixture-of-experts operators that leave to the caller what the
operators do not use, or that no kernel can take."""
import pytest
import torch

import activation_sparse_gated_gate_gb300 as tw
from tests._gpu import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def quantised(*shape, group, seed=0):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(shape, generator=g) / shape[-1] ** 0.5
    return tw.twell_quant_int4(w.cuda(), group=group, zero_points=True)


def unset_behind(q, value):
    """The same weights with anything in what is stored behind column K: codes, scales and zero
    points of the last block."""
    n, K = -(-q.K // q.group), q.K
    scale, zero = q.scale.clone(), q.zero.clone()
    scale[..., n:] = value
    zero[..., n:] = 255
    codes = tw.Int4(q.code, scale, zero, q.code.shape[-1] * 2, q.group).codes()
    codes[..., K:] = 13
    full = tw.Int4.of_codes(codes, scale, group=q.group)
    return tw.Int4(full.code, scale, zero, K, q.group)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("T", [1, 9, 40])
@pytest.mark.parametrize("K", [8, 31, 72, 164, 200, 1088])
def test_product_uses_nothing_behind_K(K, T, group, value):
    q = quantised(40, K, group=group)
    x = torch.randn((T, K), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    y = tw.twell_gemv_int4(x, q, dtype=torch.float32)
    other = unset_behind(q, value)
    assert not torch.equal(other.code, q.code)
    assert torch.equal(tw.twell_gemv_int4(x, other, dtype=torch.float32), y)
    assert torch.equal(tw.twell_dequant_int4(other), tw.twell_dequant_int4(q))


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("act", ["relu", "silu"])
@pytest.mark.parametrize("T,E,k,F,D", [(1, 4, 2, 20, 8), (3, 4, 2, 40, 72), (40, 4, 3, 50, 1088)])
def test_experts_use_nothing_behind_D(T, E, k, F, D, act, group, value):
    w = [quantised(E, F, D, group=group, seed=s) for s in range(3)]
    g = torch.Generator().manual_seed(1)
    x = (torch.randn((T, D), generator=g) + 0.5).to(torch.bfloat16).cuda()
    r = torch.randn((E, D), generator=g).cuda()
    y = tw.twell_moe_decode(x, r, *w, top_k=k, act=act).y
    other = [unset_behind(v, value) for v in w]
    assert torch.equal(tw.twell_moe_decode(x, r, *other, top_k=k, act=act).y, y)


def test_sizes_beyond_32_bits():
    """Sizes of which only the low 32 bits would reach the library are refused."""
    free, _ = torch.cuda.mem_get_info()
    if free < 180 << 30:
        pytest.skip("needs 180 GB")
    many = 2 ** 32 + 1
    x = torch.empty((many, 1), dtype=torch.bfloat16, device="cuda")
    q = tw.twell_quant_int4(torch.ones((1, 1), device="cuda"))
    y = torch.empty((many, 1), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        tw.twell_gemv_int4(x, q, out=y)
    wide = x.view(1, many)
    with pytest.raises(ValueError):
        tw.twell_quant_int4(wide)
    del y
    nb = (many + 127) // 128
    code = torch.empty((1, 64 * nb), dtype=torch.uint8, device="cuda")
    scale = torch.empty((1, nb), dtype=torch.bfloat16, device="cuda")
    long = tw.Int4(code, scale, None, many, 128)
    with pytest.raises(ValueError):
        tw.twell_dequant_int4(long)
    with pytest.raises(ValueError):
        tw.twell_gemv_int4(wide, long)
    del x, wide, code, scale, long
    x = torch.empty((many, 8), dtype=torch.bfloat16, device="cuda")
    y = torch.empty((many, 8), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((1, 8, 8), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        tw.twell_moe_decode(x[:1], None, *[x.view(1, many, 8)] * 3, ids=torch.zeros(
            (1, 1), dtype=torch.int32, device="cuda"), weights=torch.ones((1, 1), device="cuda"))
    ids = torch.zeros((many, 1), dtype=torch.int32, device="cuda")
    weights = ids.view(torch.float32)
    with pytest.raises(ValueError):
        tw.twell_moe_decode(x, None, w, w, w, ids=ids, weights=weights, y=y)
    with pytest.raises(ValueError):
        tw.twell_moe_decode(x[:1], w[0], w, w, w, top_k=many)
    for sizes in ((many, 8, 8, 1, 1), (1, many + 7, 8, 1, 1), (1, 8, many, 1, 1),
                  (1, 8, 8, many, 1), (1, 8, 8, 1, many)):
        assert tw.twell_moe_decode_workspace(*sizes) == 0


def test_workspace_size_is_asked_again(monkeypatch):
    """A size that the library could not tell is not kept for later calls."""
    g = torch.Generator().manual_seed(2)
    w = [torch.randn((3, 24, 40), generator=g).to(torch.bfloat16).cuda() for _ in range(3)]
    x, r = torch.ones((5, 40), dtype=torch.bfloat16, device="cuda"), torch.ones((3, 40), device="cuda")
    with monkeypatch.context() as m:
        m.setattr(tw, "twell_moe_decode_workspace", lambda *sizes: 0)
        with pytest.raises(tw.TwellError):
            tw.twell_moe_decode(x, r, *w, top_k=2)
    assert tw.twell_moe_decode(x, r, *w, top_k=2).y.isfinite().all()
