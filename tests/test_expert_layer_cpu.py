"""Refusals of the operators around an expert layer: checked on the host, before any device work."""
import pytest
import torch

import software_pipelined_tiled_gb300 as sptg

OK = 1 << 20        # a 16-byte aligned address that is never dereferenced on these paths
ARG, ALIGN = -1, -2
F16, BF16, S8, F32 = 0, 1, 2, 4
BIG = (1 << 31) - 4096
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    sptg.build()
    return sptg.load()


def test_route_refusals(lib):
    def call(T=2, E=16, top=4, t=F32, l=OK, ld=16, b=OK, sig=0, g=4, tg=2, gb=2, rn=1, sc=1.0, w=OK, x=OK):
        return lib.sptg_route_experts(T, E, top, t, l, ld, b, sig, g, tg, gb, rn, sc, w, x, None)

    for bad in (dict(t=S8), dict(t=3), dict(t=5), dict(t=-1), dict(T=-1), dict(T=1 << 31), dict(T=BIG, top=2), dict(E=-4),
                dict(E=1028, ld=1028), dict(top=0), dict(top=17, E=64, ld=64), dict(top=9), dict(E=3, g=1, tg=1, top=4),
                dict(g=0), dict(g=5), dict(g=-1), dict(E=64, ld=64, g=64), dict(tg=0), dict(tg=5), dict(top=5, tg=1),
                dict(gb=0), dict(gb=3), dict(sig=2), dict(sig=-1), dict(rn=2), dict(sc=INF), dict(sc=NAN),
                dict(l=None), dict(w=None), dict(x=None), dict(ld=15)):
        assert call(**bad) == ARG, bad
    for bad in (dict(l=OK + 2), dict(t=F16, l=OK + 1), dict(b=OK + 2), dict(w=OK + 1), dict(x=OK + 2)):
        assert call(**bad) == ALIGN, bad
    assert call(T=0, l=None, w=None, x=None) == 0


def test_route_dlogits_refusals(lib):
    def call(T=2, E=16, top=4, t=F32, l=OK, ld=16, x=OK, dw=OK, sig=0, rn=1, sc=1.0, dl=OK, ldd=16):
        return lib.sptg_route_experts_dlogits(T, E, top, t, l, ld, x, dw, sig, rn, sc, dl, ldd, None)

    for bad in (dict(t=S8), dict(T=-1), dict(E=1025), dict(top=0), dict(top=17), dict(sig=3), dict(rn=-1), dict(sc=NAN),
                dict(l=None), dict(x=None), dict(dw=None), dict(dl=None), dict(ld=15), dict(ldd=15)):
        assert call(**bad) == ARG, bad
    for bad in (dict(l=OK + 2), dict(x=OK + 2), dict(dw=OK + 1), dict(dl=OK + 2)):
        assert call(**bad) == ALIGN, bad
    assert call(T=0, l=None) == 0


def test_dispatch_refusals(lib):
    def call(T=2, C=16, top=4, E=8, t=BF16, x=OK, ldx=16, e=OK, s=OK, lds=16, p=OK, o=OK):
        return lib.sptg_dispatch_rows(T, C, top, E, t, x, ldx, e, s, lds, p, o, None)

    for bad in (dict(t=S8), dict(t=F32), dict(T=-1), dict(T=1 << 31), dict(C=-1), dict(C=1 << 31), dict(top=0),
                dict(top=-1), dict(T=BIG, top=2), dict(E=-1), dict(E=1025), dict(x=None), dict(e=None),
                dict(s=None), dict(p=None), dict(o=None), dict(ldx=15), dict(lds=15)):
        assert call(**bad) == ARG, bad
    for bad in (dict(x=OK + 1), dict(e=OK + 2), dict(s=OK + 1), dict(p=OK + 2), dict(o=OK + 1)):
        assert call(**bad) == ALIGN, bad


def test_combine_refusals(lib):
    def call(T=2, C=16, top=4, R=8, t=BF16, y=OK, ldy=16, p=OK, w=OK, b=OK, ldb=16, o=OK, ldo=16):
        return lib.sptg_combine_rows(T, C, top, R, t, y, ldy, p, w, b, ldb, o, ldo, None)

    for bad in (dict(t=S8), dict(t=F32), dict(T=-1), dict(C=1 << 31), dict(top=0), dict(T=BIG, top=2), dict(R=-1),
                dict(R=1 << 31), dict(y=None), dict(p=None), dict(o=None), dict(ldy=15), dict(ldb=15), dict(ldo=15)):
        assert call(**bad) == ARG, bad
    for bad in (dict(y=OK + 1), dict(p=OK + 2), dict(w=OK + 2), dict(b=OK + 1), dict(o=OK + 1)):
        assert call(**bad) == ALIGN, bad
    assert call(T=0, y=None, o=None) == 0 and call(C=0, y=None, ldy=0) == 0


def test_combine_grad_refusals(lib):
    def call(T=2, C=16, top=4, R=8, t=BF16, d=OK, ldd=16, y=OK, ldy=16, p=OK, w=OK, dy=OK, lddy=16, dw=OK):
        return lib.sptg_combine_rows_grad(T, C, top, R, t, d, ldd, y, ldy, p, w, dy, lddy, dw, None)

    for bad in (dict(t=S8), dict(T=-1), dict(C=-1), dict(top=0), dict(R=1 << 31), dict(d=None), dict(y=None), dict(p=None),
                dict(dy=None), dict(w=None), dict(ldd=15), dict(ldy=15), dict(lddy=15)):
        assert call(**bad) == ARG, bad
    for bad in (dict(d=OK + 1), dict(y=OK + 1), dict(p=OK + 2), dict(w=OK + 2), dict(dy=OK + 1), dict(dw=OK + 2)):
        assert call(**bad) == ALIGN, bad
    assert call(T=0, d=None, dy=None) == 0


def test_gate_norm_refusals(lib):
    def call(T=2, C=16, t=BF16, y=OK, ldy=16, r=OK, ldr=16, w1=OK, g=OK, k=3, ldg=16, a=1.0, w2=OK, eps=1e-6, h=OK,
             ldh=16, v=OK, ldv=16, cfg=None):
        return lib.sptg_gate_add_rms_norm(T, C, t, y, ldy, r, ldr, w1, g, k, ldg, a, w2, eps, h, ldh, v, ldv, None, cfg)

    for bad in (dict(t=S8), dict(t=F32), dict(T=-1), dict(C=1 << 31), dict(k=-1), dict(k=4), dict(eps=0.0), dict(eps=NAN),
                dict(eps=INF), dict(a=INF), dict(a=NAN), dict(y=None), dict(r=None), dict(g=None), dict(w2=None),
                dict(h=None), dict(v=None), dict(ldy=15), dict(ldr=15), dict(ldg=15), dict(k=2, ldg=0), dict(ldh=15),
                dict(ldv=15)):
        assert call(**bad) == ARG, bad
    for bad in (dict(y=OK + 1), dict(r=OK + 1), dict(w1=OK + 1), dict(g=OK + 1), dict(w2=OK + 1), dict(h=OK + 1),
                dict(v=OK + 1)):
        assert call(**bad) == ALIGN, bad
    assert call(T=0, y=None) == 0 and call(C=0, y=None) == 0
    for bad in bad_configs():
        assert call(cfg=bad) == ARG


def bad_configs():
    out = []
    for name, value in (("timeout_ms", -1), ("inject_stall", 2), ("inject_stall", -1)):
        out.append(sptg.Config())
        setattr(out[-1], name, value)
    return out


def test_gate_norm_grad_refusals(lib):
    size = lib.sptg_gate_add_rms_norm_grad_workspace(2, 16)
    assert size >= 2 * 2 * 16 * 4
    for rows, cols in ((0, 16), (16, 0), (-1, 4), (1 << 31, 4)):
        assert lib.sptg_gate_add_rms_norm_grad_workspace(rows, cols) == 0

    def call(T=2, C=16, t=BF16, dh=OK, lddh=16, dv=OK, lddv=16, y=OK, ldy=16, r=OK, ldr=16, w1=OK, g=OK, k=3, ldg=16,
             a=1.0, w2=OK, eps=1e-6, dy=OK, lddy=16, dr=OK, lddr=16, dg=OK, lddg=16, dw2=OK, dw1=OK, ot=F32, ws=OK,
             n=size, cfg=None):
        return lib.sptg_gate_add_rms_norm_grad(T, C, t, dh, lddh, dv, lddv, y, ldy, r, ldr, w1, g, k, ldg, a, w2, eps, dy,
                                               lddy, dr, lddr, dg, lddg, dw2, dw1, ot, ws, n, None, cfg)

    for bad in (dict(t=S8), dict(T=-1), dict(C=1 << 31), dict(k=4), dict(eps=-1.0), dict(a=NAN), dict(ot=F16), dict(ot=S8),
                dict(y=None), dict(r=None), dict(g=None), dict(w2=None), dict(dy=None), dict(dr=None), dict(dg=None),
                dict(dw2=None), dict(dw1=None), dict(ws=None), dict(n=size - 1), dict(lddh=15), dict(lddv=15),
                dict(ldy=15), dict(ldr=15), dict(ldg=15), dict(k=2, ldg=0), dict(lddy=15), dict(lddr=15), dict(lddg=15),
                dict(k=1, dg=None), dict(k=2, ldg=1, dg=None), dict(T=0, dw2=None), dict(C=0, k=2, dg=None)):
        assert call(**bad) == ARG, bad
    for bad in (dict(dh=OK + 1), dict(dv=OK + 1), dict(y=OK + 1), dict(r=OK + 1), dict(w1=OK + 1), dict(g=OK + 1),
                dict(w2=OK + 1), dict(dy=OK + 1), dict(dr=OK + 1), dict(dg=OK + 1), dict(dw2=OK + 2),
                dict(dw1=OK + 2), dict(k=1, dg=OK + 2), dict(ws=OK + 8)):
        assert call(**bad) == ALIGN, bad
    for bad in bad_configs():
        assert call(cfg=bad) == ARG


def test_python_refuses_bad_tensors():
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    for bad in (lambda: sptg.route_experts(x, 2), lambda: sptg.route_experts_dlogits(x, x, ids),
                lambda: sptg.dispatch_rows(x, ids, 4), lambda: sptg.dispatch_rows_dx(x, ids),
                lambda: sptg.combine_rows(x, ids), lambda: sptg.combine_rows_grad(x, x, ids),
                lambda: sptg.gate_add_rms_norm(x, x, x[0]), lambda: sptg.gate_add_rms_norm_grad(x, x, x, x, x[0])):
        with pytest.raises(ValueError):
            bad()
