"""Refusals of the operators around the dense products: checked on the host, before any device work."""
import pytest
import torch

import software_pipelined_tiled_gb300 as sptg

OK = 1 << 20        # a 16-byte aligned address that is never dereferenced on these paths
ARG, ALIGN = -1, -2
F16, BF16, S8, E4M3 = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    sptg.build()
    return sptg.load()


def test_norm_refusals(lib):
    def call(rows=2, cols=64, it=BF16, ot=S8, x=OK, ldx=64, r=OK, ldr=64, w=OK, eps=1e-6, h=OK,
             ldh=64, y=OK, ldy=64, s=OK):
        return lib.sptg_add_rms_norm(rows, cols, it, ot, x, ldx, r, ldr, w, eps, h, ldh, y, ldy, s, None)

    for bad in (dict(it=S8), dict(it=77), dict(ot=F16), dict(ot=-1), dict(rows=-1), dict(cols=-1),
                dict(rows=1 << 31), dict(cols=(1 << 31) - 1, ldx=1 << 31, ldr=1 << 31, ldh=1 << 31,
                                         ldy=1 << 31), dict(eps=0.0), dict(eps=-1e-6), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(x=None), dict(r=None), dict(w=None), dict(h=None),
                dict(y=None), dict(s=None), dict(ldx=63), dict(ldr=63), dict(ldh=63), dict(ldy=63)):
        assert call(**bad) == ARG, bad
    for bad in (dict(x=OK + 1), dict(r=OK + 1), dict(w=OK + 1), dict(h=OK + 1), dict(s=OK + 2),
                dict(ot=BF16, y=OK + 1, s=None)):
        assert call(**bad) == ALIGN, bad
    assert call(rows=0, x=None, y=None) == 0 and call(cols=0, x=None) == 0


def test_w4_refusals(lib):
    def call(M=2, N=8, K=128, g=64, xt=BF16, ot=BF16, x=OK, ldx=128, xs=None, c=OK, ldw=64, s=OK,
             z=None, y=OK, ldy=8):
        return lib.sptg_gemm_w4(M, N, K, g, xt, ot, x, ldx, xs, c, ldw, s, z, y, ldy, None)

    for bad in (dict(xt=F16), dict(ot=S8), dict(ot=9), dict(xt=9), dict(M=-1), dict(N=1 << 31),
                dict(N=(1 << 31) - 128, ldy=1 << 31),
                dict(K=-128), dict(g=16), dict(g=0), dict(K=160, ldx=160, ldw=80), dict(x=None),
                dict(c=None), dict(s=None), dict(y=None), dict(xt=S8, xs=None), dict(xs=OK),
                dict(ldx=127), dict(ldw=63), dict(ldy=7)):
        assert call(**bad) == ARG, bad
    for bad in (dict(x=OK + 8), dict(c=OK + 8), dict(s=OK + 1), dict(y=OK + 1), dict(ldx=130),
                dict(ldw=72), dict(xt=S8, xs=OK + 2)):
        assert call(**bad) == ALIGN, bad
    assert call(M=0, x=None) == 0 and call(N=0, c=None) == 0


def test_grouped_refusals(lib):
    def y(E=2, T=4, N=16, K=16, d=3, o=OK, x=OK, ldx=16, w=OK, out=OK, ldo=16):
        return lib.sptg_grouped_gemm(E, T, N, K, d, o, x, ldx, w, out, ldo, None)

    def dx(E=2, T=4, N=16, K=16, d=3, o=OK, x=OK, ldx=16, w=OK, out=OK, ldo=16):
        return lib.sptg_grouped_gemm_dx(E, T, N, K, d, o, x, ldx, w, out, ldo, None)

    def dw(E=2, T=4, N=16, K=16, d=3, o=OK, x=OK, ldx=16, w=OK, ldw=16, out=OK):
        return lib.sptg_grouped_gemm_dw(E, T, N, K, d, o, x, ldx, w, ldw, out, None)

    for f in (y, dx, dw):
        for bad in (dict(d=2), dict(d=50), dict(E=-1), dict(T=-1), dict(N=-8), dict(K=1 << 31),
                    dict(T=(1 << 31) - 1),
                    dict(E=1025), dict(o=None), dict(x=None), dict(w=None), dict(out=None),
                    dict(ldx=8)):
            assert f(**bad) == ARG, (f.__name__, bad)
        for bad in (dict(x=OK + 8), dict(w=OK + 8), dict(out=OK + 8), dict(o=OK + 2), dict(ldx=20),
                    dict(N=12), dict(K=12)):
            assert f(**bad) == ALIGN, (f.__name__, bad)
    assert y(ldo=8) == ARG and dx(ldo=8) == ARG and dw(ldw=8) == ARG
    assert y(ldo=20) == ALIGN and dx(ldo=20) == ALIGN and dw(ldw=20) == ALIGN
    assert y(T=0, x=None) == 0 and y(N=0, w=None) == 0 and dx(K=0) == 0 and dw(E=0, o=None) == 0


def test_python_refuses_host_tensors_and_mixed_types():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        sptg.add_rms_norm(x, x, x[0])
    with pytest.raises(ValueError, match="CUDA"):
        sptg.gemm_w4(x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        sptg.grouped_gemm(x, x[None], torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        sptg.grouped_gemm_dw(x, x, torch.zeros(2, dtype=torch.int32))
