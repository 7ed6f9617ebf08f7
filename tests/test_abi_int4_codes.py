"""What ``Int4.of_codes`` takes of a checkpoint and what it refuses."""
import pytest
import torch

import activation_sparse_gated_gate_gb300 as tw


def taken(codes, zero=None):
    n = -(-codes.shape[-1] // 32)
    return tw.Int4.of_codes(codes, torch.ones((*codes.shape[:-1], n)), zero, group=32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("value", [3.4, 7.5, 14.99, 15.25, -0.5, float("nan"), float("inf")])
def test_only_integers(value, dtype):
    """Half-way zero points and codes that are no integers are not cut off."""
    if dtype is torch.bfloat16 and value == 14.99:
        value = 14.9375
    codes = torch.full((2, 40), 5.0, dtype=dtype)
    zero = torch.full((2, 2), 8.0, dtype=dtype)
    taken(codes, zero)
    zero[1, 1] = value
    with pytest.raises(ValueError):
        taken(codes, zero)
    codes[1, 39] = value
    with pytest.raises(ValueError):
        taken(codes)


@pytest.mark.parametrize("dtype", [torch.uint8, torch.int8, torch.int32, torch.int64,
                                   torch.float16, torch.float32])
def test_integers_of_any_type(dtype):
    g = torch.Generator().manual_seed(1)
    codes = torch.randint(0, 16, (3, 70), generator=g)
    zero = torch.randint(0, 16, (3, 3), generator=g)
    w = taken(codes.to(dtype), zero.to(dtype))
    assert torch.equal(w.codes(), codes.to(torch.uint8))
    assert torch.equal(w.zero[:, :3], zero.to(torch.uint8))
    none = taken(codes[:0].to(dtype), zero[:0].to(dtype))
    assert none.shape == (0, 70)


@pytest.mark.parametrize("dtype", [torch.uint8, torch.int32, torch.float32])
def test_range(dtype):
    codes = torch.zeros((2, 40), dtype=dtype)
    for bad in (16, 255 if dtype is torch.uint8 else -1):
        codes[0, 3] = bad
        with pytest.raises(ValueError):
            taken(codes)


def test_scales_round_to_bf16():
    s = torch.rand((2, 2), generator=torch.Generator().manual_seed(1)).to(torch.float16)
    w = tw.Int4.of_codes(torch.zeros((2, 64), dtype=torch.uint8), s, group=32)
    assert torch.equal(w.scale[:, :2], s.to(torch.bfloat16))
    assert ((w.scale[:, :2].double() - s.double()).abs() <= 2.0 ** -8 * s.double()).all()
