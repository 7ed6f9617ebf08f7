"""Host-side argument checks of the norm, quantisation and 8-bit product entry
points: bad calls are rejected before any device work, empty ones do nothing."""
import ctypes
import os

import pytest

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


NORM = dict(x=P, x_type=BF16, ldx=64, r=P, r_type=F32, ldr=64, w=P, w_type=F32, T=4, D=64,
            eps=1e-6, total=P, ldt=64, y=P, ldy=64, q=P, ldq=64, scale=P, rstd=P, stream=None)


def norm(lib, **kw):
    return lib.twell_rms_norm(*{**NORM, **kw}.values())


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(D=0), dict(eps=-1.0), dict(eps=float("nan")), dict(x_type=2), dict(w_type=-1),
    dict(r_type=7), dict(x=None), dict(w=None), dict(r=None), dict(total=None), dict(scale=None),
    dict(q=None), dict(y=None, q=None, scale=None), dict(ldx=63), dict(ldr=0), dict(ldt=10),
    dict(ldy=63), dict(ldq=63), dict(x=P + 1), dict(y=P + 1), dict(total=P + 2), dict(scale=P + 2),
    dict(rstd=P + 1), dict(w=P + 2)])
def test_norm_rejects(lib, bad):
    assert norm(lib, **bad) == INVALID


def test_norm_limits(lib):
    big = {k: 20000 for k in ("D", "ldx", "ldr", "ldt", "ldy", "ldq")}
    assert norm(lib, **big) == UNSUPPORTED
    assert norm(lib, T=0, x=None, y=None) == OK


BWD = dict(total=P, type=F32, ld=64, w=P, w_type=F32, rstd=P, dy=P, dy_type=BF16, lddy=64,
           dtotal=P, lddt=64, T=4, D=64, dx=P, lddx=64, dw=P, ws=P, ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(D=0), dict(type=3), dict(w_type=9), dict(dy_type=-2), dict(dw=None),
    dict(total=None), dict(w=None), dict(rstd=None), dict(dy=None), dict(dx=None), dict(ws=None),
    dict(ld=63), dict(lddy=63), dict(lddt=63), dict(lddx=63), dict(dw=P + 2), dict(total=P + 2),
    dict(dy=P + 1)])
def test_norm_bwd_rejects(lib, bad):
    assert lib.twell_rms_norm_bwd(*{**BWD, **bad}.values()) == INVALID


@pytest.mark.parametrize("off", [4, 8, 12])
def test_norm_bwd_rejects_a_workspace_off_16_bytes(lib, off):
    # its partial sums are stored 16 bytes at a time
    assert lib.twell_rms_norm_bwd(*{**BWD, "ws": P + off}.values()) == INVALID


def test_norm_bwd_workspace(lib):
    assert tw.twell_rms_norm_bwd_workspace(-1, 64) == 0
    assert tw.twell_rms_norm_bwd_workspace(4, 0) == 0
    assert tw.twell_rms_norm_bwd_workspace(4, 20000) == 0
    assert tw.twell_rms_norm_bwd_workspace(1, 64) >= 64 * 4
    assert tw.twell_rms_norm_bwd_workspace(16384, 2304) >= 2304 * 4


QUANT = dict(src=P, type=BF16, ld=64, R=4, C=64, block=1, q=P, ldq=64, scale=P, qt=P, ldqt=16,
             scale_t=P, stream=None)


@pytest.mark.parametrize("bad", [
    dict(R=-1), dict(C=-1), dict(block=2), dict(type=2), dict(src=None), dict(src=P + 1),
    dict(q=None), dict(scale=None), dict(qt=None), dict(scale_t=None), dict(ld=63), dict(ldq=63),
    dict(ldqt=3), dict(scale=P + 1), dict(q=None, scale=None, qt=None, scale_t=None)])
def test_quant_rejects(lib, bad):
    assert lib.twell_quant_fp8(*{**QUANT, **bad}.values()) == INVALID


def test_quant_empty(lib):
    assert lib.twell_quant_fp8(*{**QUANT, "R": 0}.values()) == OK
    assert lib.twell_quant_fp8(*{**QUANT, "C": 0}.values()) == OK


GEMM = dict(a=P, lda=64, sa=P, b=P, ldb=64, sb=P, block=128, M=4, N=256, K=64, c=P, c_type=BF16,
            ldc=256, status=P, stream=None)


@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(N=-1), dict(K=0), dict(block=64), dict(c_type=2), dict(a=None), dict(b=None),
    dict(sa=None), dict(sb=None), dict(c=None), dict(a=P + 8), dict(b=P + 4), dict(sa=P + 2),
    dict(lda=72), dict(ldb=48), dict(lda=60), dict(ldc=255), dict(c=P + 1)])
def test_gemm_rejects(lib, bad):
    assert lib.twell_gemm_fp8(*{**GEMM, **bad}.values()) == INVALID


def test_gemm_empty(lib):
    assert lib.twell_gemm_fp8(*{**GEMM, "M": 0, "a": None}.values()) == OK
    assert lib.twell_gemm_fp8(*{**GEMM, "N": 0, "c": None}.values()) == OK


@pytest.mark.parametrize("big", [dict(M=2**31 - 1), dict(N=2**31 - 1, ldc=2**31),
                                 dict(M=2**31 - 255), dict(N=2**31 - 255, ldc=2**31)])
def test_gemm_limits(lib, big):
    # tiles past them would not be numbered in 32 bits
    assert lib.twell_gemm_fp8(*{**GEMM, **big}.values()) == UNSUPPORTED


@pytest.mark.parametrize("T,F", [(2**31 - 1, 128), (1, 2**31 - 128), (2**24, 2**14)])
def test_gate_limits(lib, T, F):
    s = tw.TwellStruct(T, F, 128, 8, P, P, P, P, 16, P, P, P, None)
    assert gate(lib, s, T=T, F=F) == UNSUPPORTED


def gate(lib, s=None, **kw):
    s = tw.TwellStruct(4, 256, 128, 8, P, P, P, P, 16, P, P, P, None) if s is None else s
    args = dict(xq=P, ldx=64, sx=P, wq=P, ldw=64, sw=P, T=4, D=64, F=256, out=ctypes.byref(s),
                z=None, status=P, stream=None)
    return lib.twell_gate_pack_fp8(*{**args, **kw}.values())


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(T=5), dict(D=0), dict(F=200), dict(F=384), dict(xq=None), dict(wq=None),
    dict(sx=None), dict(sw=None), dict(xq=P + 8), dict(ldw=72), dict(ldx=32), dict(out=None),
    dict(z=P + 4)])
def test_gate_rejects(lib, bad):
    assert gate(lib, **bad) == INVALID


def test_gate_empty(lib):
    s = tw.TwellStruct(0, 256, 128, 8, None, None, None, None, 0, None, None, None, None)
    assert gate(lib, s, T=0, xq=None) == OK


def test_valid_calls_without_a_gpu_report_it(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("has a GPU")
    for code in (norm(lib), lib.twell_rms_norm_bwd(*BWD.values()),
                 lib.twell_quant_fp8(*QUANT.values()), lib.twell_gemm_fp8(*GEMM.values()),
                 gate(lib)):
        assert code in (CUDA, UNSUPPORTED)
