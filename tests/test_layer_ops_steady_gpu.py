"""The layer operators past their first stages: rings that wrap, barriers that turn, segments that follow each other.

Small products with 4-bit weights are cut along K until a CTA has a stage or three; these are wide enough
to leave a CTA more stages than its ring holds, in every type of x, group size and number of rows.  Every
operator gives the same bits when it is called again.

Bounds, derived before the first run: each value as in test_layer_ops_gpu.  In the mean, rounding an exact
value to nearest is off by the unit in the last place over sqrt(12), that is at most 2 u / sqrt(12) =
0.577 u of the value (u: unit roundoff); the sums' own errors are far below that, so the root mean square
error stays within 0.6 u of the root mean square result.  One group, column or stage that is lost,
repeated or taken from another place is many times that.
"""
import pytest
import torch

import software_pipelined_tiled_gb300 as sptg
from test_layer_ops_gpu import (BF16, E4M3, F16, F32, S8, U, assert_close, gen, offsets_of, rand, w4_inputs,
                                w4_reference)

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


# the same bits on every call, for the operators whose kernels hand work from warp to warp
def _again(f, *args, **kw):
    first = f(*args, **kw)
    for _ in range(5):
        for a, b in zip(*((t if isinstance(t, tuple) else (t,)) for t in (first, f(*args, **kw)))):
            if a is not None:
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("out_dtype", [E4M3, S8, None])
@pytest.mark.parametrize("rows,cols", [(1, 4096), (700, 4096), (333, 5000), (1900, 8192), (16384, 8192), (3, 5001)])
def test_norm_gives_the_same_bits_on_every_call(rows, cols, out_dtype):
    g = gen(rows)
    _again(sptg.add_rms_norm, rand(g, rows, cols), rand(g, rows, cols), rand(g, cols), out_dtype=out_dtype)


# the sizes of a decoding step, of a prompt's ragged experts, and of rows that fill whole tiles and do not
@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("sizes,n,k", [([3, 0, 9, 1, 0, 0, 12, 0, 7], 4096, 2048), ([300, 0, 1025, 17, 700], 1048, 1160),
                                       ([256, 512, 1000, 1024], 2048, 2048)])
def test_grouped_gives_the_same_bits_on_every_call(sizes, n, k, out_dtype):
    g = gen(n)
    t, off = sum(sizes), offsets_of(sizes)
    X, W, dY = rand(g, t, k), rand(g, len(sizes), n, k), rand(g, t, n)
    _again(sptg.grouped_gemm, X, W, off, out_dtype=out_dtype)
    _again(sptg.grouped_gemm_dx, dY, W, off, out_dtype=out_dtype)
    _again(sptg.grouped_gemm_dw, dY, X, off, out_dtype=out_dtype)


# K cut over a cluster's CTAs
@pytest.mark.parametrize("m", [1, 8, 16, 33, 64])
@pytest.mark.parametrize("xdtype", [BF16, S8])
def test_w4_in_clusters_gives_the_same_bits_on_every_call(m, xdtype):
    x, codes, scales, z, xs = w4_inputs(gen(m), m, 4096, 8192, 128, BF16, xdtype, True)
    _again(sptg.gemm_w4, x, codes, scales, z, x_scales=xs)
    assert chosen()["splits"] > 1


# widths of dW's last tile of columns, in steps of 8, past one and past two tiles
@pytest.mark.parametrize("cols", [104, 112, 120, 136, 144, 232, 360, 368, 2056])
def test_grouped_dw_of_every_width(cols):
    g = gen(cols)
    off, o = offsets_of([70, 33, 0, 128]), [0, 70, 103, 103, 231]
    X, dY = rand(g, 231, cols), rand(g, 231, 136)
    dw = sptg.grouped_gemm_dw(dY, X, off, out_dtype=F32)
    for e in range(4):
        d, x = dY[o[e]:o[e + 1]].double(), X[o[e]:o[e + 1]].double()
        assert_close(dw[e], d.t() @ x, d.abs().t() @ x.abs(), o[e + 1] - o[e])
