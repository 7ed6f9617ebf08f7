"""Host-side checks of the 4-bit and mixture-of-experts entry points (bad calls are rejected
before any device work, empty ones do nothing), and the stored order of 4-bit codes."""
import ctypes
import os

import numpy as np
import pytest
import torch

import activation_sparse_gated_gate_gb300 as tw

OK, INVALID, UNSUPPORTED, CUDA = 0, 1, 2, 3
P = 0x10000  # aligned, never dereferenced
BF16, F32 = 0, 1


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(tw.LIB_PATH):
        from activation_sparse_gated_gate_gb300 import build
        build.build()
    return tw.lib()


def int4(rows=8, K=64, group=32, code=P, scale=P, zero=P):
    return tw._INT4.pack(rows, K, group, code or 0, scale or 0, zero or 0)


BAD_INT4 = [dict(rows=-1), dict(K=0), dict(K=-5), dict(group=16), dict(group=0), dict(group=256),
            dict(code=None), dict(scale=None), dict(code=P + 8), dict(scale=P + 4),
            dict(zero=P + 2), dict(scale=P + 2, group=64), dict(zero=P + 1, group=64),
            dict(scale=P + 1, group=128)]


@pytest.mark.parametrize("bad", BAD_INT4)
def test_descriptors(lib, bad):
    w = int4(**bad)
    K = bad.get("K", 64)
    assert lib.twell_quant_int4(P, BF16, max(K, 64), w, None) == INVALID
    assert lib.twell_dequant_int4(w, P, BF16, max(K, 64), None) == INVALID
    assert lib.twell_gemv_int4(P, max(K, 64), w, 3, P, BF16, 8, None) == INVALID


def test_no_descriptor(lib):
    assert lib.twell_quant_int4(P, BF16, 64, None, None) == INVALID
    assert lib.twell_dequant_int4(None, P, BF16, 64, None) == INVALID
    assert lib.twell_gemv_int4(P, 64, None, 3, P, BF16, 8, None) == INVALID


@pytest.mark.parametrize("bad", [dict(src=None), dict(src=P + 1), dict(type=2), dict(type=-1),
                                 dict(ld=63), dict(ld=0), dict(src=P + 2, type=F32)])
def test_quant_rejects(lib, bad):
    a = {**dict(src=P, type=BF16, ld=64), **bad}
    assert lib.twell_quant_int4(a["src"], a["type"], a["ld"], int4(), None) == INVALID
    assert lib.twell_dequant_int4(int4(), a["src"], a["type"], a["ld"], None) == INVALID


@pytest.mark.parametrize("bad", [dict(x=None), dict(x=P + 1), dict(ldx=63), dict(T=-1),
                                 dict(y=None), dict(y=P + 1), dict(y_type=5), dict(ldy=7),
                                 dict(y=P + 2, y_type=F32)])
def test_gemv_rejects(lib, bad):
    a = {**dict(x=P, ldx=64, w=int4(), T=3, y=P, y_type=BF16, ldy=8), **bad}
    assert lib.twell_gemv_int4(*a.values(), None) == INVALID


def test_empty_and_limits(lib):
    none = int4(rows=0, code=None, scale=None, zero=None)
    assert lib.twell_quant_int4(None, BF16, 64, none, None) == OK
    assert lib.twell_dequant_int4(none, None, BF16, 64, None) == OK
    assert lib.twell_gemv_int4(None, 0, none, 3, None, BF16, 0, None) == OK
    assert lib.twell_gemv_int4(None, 0, int4(), 0, None, BF16, 0, None) == OK
    assert lib.twell_gemv_int4(P, 64, int4(rows=2 ** 31), 3, P, BF16, 2 ** 31, None) == UNSUPPORTED
    assert lib.twell_gemv_int4(P, 64, int4(), 2 ** 21, P, BF16, 8, None) == UNSUPPORTED


class Experts:
    """``twell_experts_t`` and the descriptors that it points at."""

    def __init__(self, E=4, F=32, D=64, bits=16, gate=P, up=P, down=P, extra=0, **kw):
        self.q = [ctypes.create_string_buffer(int4(**{**dict(rows=E * F, K=D), **(kw.get(n) or {})}))
                  for n in ("gate4", "up4", "down4")]
        at = [ctypes.addressof(b) for b in self.q]
        p = [gate or 0, up or 0, down or 0]
        fields = (*p, extra, 0, 0) if bits == 16 else (extra, 0, 0, *at)
        for i, n in enumerate(("gate4", "up4", "down4")):
            if n in kw and kw[n] is None:
                fields = (*fields[:3 + i], 0, *fields[4 + i:])
        self.bytes = tw._EXPERTS.pack(E, F, D, *fields)


def moe(lib, experts=None, **kw):
    e = experts or Experts()
    a = {**dict(x=P, T=3, router=P, router_type=BF16, w=e.bytes, top_k=2, act=0, renormalise=1,
                ids=P, weights=P, y=P, y_type=F32, ws=P, ws_bytes=1 << 30), **kw}
    return lib.twell_moe_decode(*a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(top_k=0), dict(top_k=5), dict(act=2), dict(act=-1), dict(router_type=2),
    dict(y_type=2), dict(x=None), dict(x=P + 2), dict(ids=None), dict(ids=P + 2),
    dict(weights=None), dict(weights=P + 1), dict(y=None), dict(y=P + 8), dict(ws=None),
    dict(ws=P + 8), dict(router=P + 4), dict(w=None)])
def test_moe_rejects(lib, bad):
    assert moe(lib, **bad) == INVALID


@pytest.mark.parametrize("bad", [
    dict(E=0), dict(F=0), dict(D=0), dict(D=60), dict(D=-8), dict(gate=None), dict(up=None),
    dict(down=None), dict(gate=P + 8), dict(down=P + 2), dict(extra=P),
    dict(bits=4, extra=P), dict(bits=4, up4=None), dict(bits=4, gate4=dict(rows=127)),
    dict(bits=4, up4=dict(K=32)), dict(bits=4, down4=dict(group=64)),
    dict(bits=4, up4=dict(code=P + 8)), dict(bits=4, gate4=dict(rows=-1))])
def test_moe_rejects_experts(lib, bad):
    assert moe(lib, Experts(**bad)) == INVALID


def test_moe_empty_and_limits(lib):
    assert moe(lib, T=0, x=None, y=None, ids=None, weights=None, ws=None) == OK
    assert moe(lib, T=257) == UNSUPPORTED
    assert moe(lib, T=200, top_k=11, router=None) == UNSUPPORTED
    assert moe(lib, Experts(E=40), top_k=33) == UNSUPPORTED
    assert moe(lib, Experts(E=513)) == UNSUPPORTED
    assert moe(lib, Experts(D=16392)) == UNSUPPORTED
    assert moe(lib, Experts(E=512, F=1 << 18)) == UNSUPPORTED
    for sizes in ((3, 60, 32, 4, 2), (-1, 64, 32, 4, 2), (3, 64, 0, 4, 2), (3, 64, 32, 0, 2),
                  (3, 64, 32, 4, 0), (257, 64, 32, 4, 2), (3, 64, 32, 513, 2)):
        assert lib.twell_moe_decode_workspace(*sizes) == 0


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("K", [1, 8, 31, 128, 200, 384])
def test_stored_order(K, group):
    """Column 32 i + 8 c + 2 n + o of a block is nibble n of the 16 bits at byte
    8 (2 c + o) + 2 i."""
    g = torch.Generator().manual_seed(K)
    codes = torch.randint(0, 16, (3, K), generator=g, dtype=torch.uint8)
    n = -(-K // group)
    scale = torch.rand((3, n), generator=g)
    zero = torch.randint(0, 16, (3, n), generator=g)
    w = tw.Int4.of_codes(codes, scale, zero, group)
    assert w.shape == (3, K) and w.code.shape == (3, 64 * -(-K // 128))
    raw = w.code.numpy()
    for k in range(-(-K // 128) * 128):
        b, r = divmod(k, 128)
        i, c, m, o = r // 32, r // 8 % 4, r // 2 % 4, r % 2
        at = 64 * b + 8 * (2 * c + o) + 2 * i
        bits = raw[:, at].astype(np.int64) | raw[:, at + 1].astype(np.int64) << 8
        want = codes[:, k].numpy() if k < K else 8
        assert ((bits >> (4 * m) & 15) == want).all()
    assert torch.equal(w.codes(), codes)
    held = w.scale.shape[1]
    assert held == -(-K // 128) * (128 // group)
    assert torch.equal(w.scale[:, :n], scale.to(torch.bfloat16)) and not w.scale[:, n:].any()
    assert torch.equal(w.zero[:, :n], zero.to(torch.uint8)) and (w.zero[:, n:] == 8).all()


@pytest.mark.parametrize("bad", [
    dict(codes=torch.full((2, 64), 16)), dict(codes=torch.full((2, 64), -1)), dict(group=48),
    dict(scale=torch.ones(2, 3)), dict(zero=torch.full((2, 2), 16)), dict(zero=torch.ones(2, 1))])
def test_of_codes_rejects(bad):
    a = {**dict(codes=torch.zeros((2, 64), dtype=torch.int64), scale=torch.ones(2, 2), zero=None,
                group=32), **bad}
    with pytest.raises(ValueError):
        tw.Int4.of_codes(**a)


def test_binding_needs_the_gpu():
    w = torch.zeros((4, 64))
    q = tw.Int4.of_codes(torch.zeros((4, 64), dtype=torch.uint8), torch.ones(4, 1), group=64)
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    for call in (lambda: tw.twell_quant_int4(w), lambda: tw.twell_dequant_int4(q),
                 lambda: tw.twell_gemv_int4(x, q), lambda: tw.twell_gemv_int4(x, w),
                 lambda: tw.twell_moe_decode(x, None, w, w, w)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        tw.twell_quant_int4(w, group=100)
