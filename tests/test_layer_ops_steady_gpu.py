"""The 4-bit kernels past their first stages: rings that wrap, barriers that turn, segments that follow each other.

Small products are cut along K until a CTA has a stage or three; these are wide enough to leave a CTA
more stages than its ring holds, in every type of x, group size and number of rows.

Bounds, derived before the first run: each value as in test_layer_ops_gpu.  In the mean, rounding an exact
value to nearest is off by the unit in the last place over sqrt(12), that is at most 2 u / sqrt(12) =
0.577 u of the value (u: unit roundoff); the sums' own errors are far below that, so the root mean square
error stays within 0.6 u of the root mean square result.  One group, column or stage that is lost,
repeated or taken from another place is many times that.
"""
import pytest
import torch

import software_pipelined_tiled_gb300 as sptg
from test_layer_ops_gpu import BF16, E4M3, F16, S8, U, assert_close, gen, w4_inputs, w4_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    torch.cuda.synchronize()
    assert sptg.device_error() == 0


def chosen():
    """The numbers of the last call's choice of kernel."""
    return {k: int(v) for k, v in (f.split("=") for f in sptg.last_config().split() if "=" in f)
            if v.isdigit()}


def close_in_the_mean(y, ref):
    err, size = ((t.double().square().mean().sqrt()) for t in (y.double() - ref, ref))
    assert err <= 0.6 * U[y.dtype] * size, f"rms error {float(err / size / U[y.dtype]):.3f} u"


# stages of K past the ring's ten at most; rows of weights a CTA from 80 to 128; scales and zero points
# read a lane's groups at a time (K a multiple of 256) and one by one
@pytest.mark.parametrize("m", [16, 32, 64])
@pytest.mark.parametrize("xdtype", [BF16, F16, S8, E4M3])
@pytest.mark.parametrize("n,k,group,zeros", [(18001, 4128, 32, True), (18000, 5120, 32, False),
                                             (14300, 4160, 64, False), (18001, 4352, 64, True),
                                             (18000, 4224, 128, True), (15000, 8192, 128, False),
                                             (11800, 4096, 128, True)])
def test_w4_tiles_of_many_stages(n, k, group, zeros, m, xdtype):
    g = gen(n + m)
    dtype = xdtype if xdtype in (BF16, F16) else (BF16 if m == 32 else F16)
    x, codes, scales, z, xs = w4_inputs(g, m, n, k, group, dtype, xdtype, zeros)
    y = sptg.gemm_w4(x, codes, scales, z, x_scales=xs)
    c = chosen()
    assert -(-k // 256) // c["splits"] > c["stages"] and c["x_rows"] >= 16
    ref, S = w4_reference(x, codes, scales, z, xs)
    assert_close(y, ref, S, k)
    close_in_the_mean(y, ref)
    for _ in range(5):
        assert torch.equal(y, sptg.gemm_w4(x, codes, scales, z, x_scales=xs))


# K in two segments and more, after each of which x is loaded anew, and more stages than a warp's ring
# holds; segments that end in the middle of the last one
@pytest.mark.parametrize("m", [1, 5, 8])
@pytest.mark.parametrize("xdtype", [BF16, F16, S8, E4M3])
@pytest.mark.parametrize("n,k,group,zeros", [(18001, 24608, 32, True), (18000, 20480, 32, False),
                                             (8200, 24640, 64, False), (18001, 16640, 64, True),
                                             (18000, 16512, 128, True), (32768, 8192, 128, False)])
def test_w4_streams_of_many_segments(n, k, group, zeros, m, xdtype):
    g = gen(n + m)
    dtype = xdtype if xdtype in (BF16, F16) else (BF16 if m == 5 else F16)
    x, codes, scales, z, xs = w4_inputs(g, m, n, k, group, dtype, xdtype, zeros)
    y = sptg.gemm_w4(x, codes, scales, z, x_scales=xs)
    c = chosen()
    stages = -(-(-(-k // 256)) // c["splits"])
    assert c["x_rows"] == 8 and stages > 2 * c["stages"]
    if m > 1:
        assert stages > c["segment"]
    ref, S = w4_reference(x, codes, scales, z, xs)
    assert_close(y, ref, S, k)
    close_in_the_mean(y, ref)
    for _ in range(5):
        assert torch.equal(y, sptg.gemm_w4(x, codes, scales, z, x_scales=xs))
