"""Unusual sizes of the operators around the dense products: settled on the host, before any device work."""
import pytest

import software_pipelined_tiled_gb300 as sptg

OK = 1 << 20  # a 16-byte aligned address that is never dereferenced on these paths
ARG = -1
BF16_BF16 = 3


@pytest.fixture(scope="module")
def lib():
    sptg.build()
    return sptg.load()


@pytest.mark.parametrize("e,n,k", [(16, 1 << 30, 1 << 30), (1024, 1 << 30, 1 << 30), (64, 1 << 28, 1 << 30),
                                   (5, 1 << 30, (1 << 31) - 4096)])
def test_grouped_dw_of_more_elements_than_64_bits_count(lib, e, n, k):
    """The product of the three sizes passes 2^64; for the first three its low 64 bits are zero."""
    assert lib.sptg_grouped_gemm_dw(e, 4, n, k, BF16_BF16, OK, OK, n, OK, k, OK, None) == ARG
    assert "tiles" in sptg.last_error()
