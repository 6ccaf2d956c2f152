"""Refusals of the gradients around an expert layer that a later entry point added: checked on the host."""
import pytest

import software_pipelined_tiled_gb300 as sptg

OK = 1 << 20        # a 16-byte aligned address that is never dereferenced on these paths
ARG, ALIGN = -1, -2
S8, BF16 = 2, 1


@pytest.fixture(scope="module")
def lib():
    sptg.build()
    return sptg.load()


def test_combine_grad_ex_refusals(lib):
    def call(T=2, C=16, top=4, R=8, t=BF16, d=OK, ldd=16, y=OK, ldy=16, p=OK, w=OK, dy=OK, lddy=16, dw=OK, zero=1):
        return lib.sptg_combine_rows_grad_ex(T, C, top, R, t, d, ldd, y, ldy, p, w, dy, lddy, dw, zero, None)

    for bad in (dict(zero=2), dict(zero=-1), dict(t=S8), dict(T=-1), dict(C=-1), dict(top=0), dict(R=1 << 31), dict(R=-1),
                dict(d=None), dict(y=None), dict(p=None), dict(dy=None), dict(w=None), dict(ldd=15), dict(ldy=15),
                dict(lddy=15), dict(T=0, dy=None), dict(T=0, lddy=15)):
        assert call(**bad) == ARG, bad
    for bad in (dict(d=OK + 1), dict(y=OK + 1), dict(p=OK + 2), dict(w=OK + 2), dict(dy=OK + 1), dict(dw=OK + 2),
                dict(T=0, dy=OK + 1)):
        assert call(**bad) == ALIGN, bad
    assert call(T=0, R=0, d=None, y=None, p=None, dy=None) == 0 and call(C=0, dw=None) == 0
    assert call(T=0, zero=0, d=None, dy=None) == 0
