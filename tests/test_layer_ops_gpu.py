"""The operators around the dense products against plain implementations in 64 bits.

Bounds, derived before the first run (u: unit roundoff of the output type,
2^-11 for binary16, 2^-8 for bfloat16, 0 for float32; S: the sum of the
products' magnitudes):

* products: a sum of n terms kept in 32 bits is off by at most (n + 16) 2^-23 S
  (each addition and each scaling at most one unit in the last place, by
  truncation at worst), and the result is rounded once more: u |ref|.
* norm: the sum of squares of n values is off by at most (n + 16) 2^-24 of
  itself, its reciprocal root by half of that; each quantised value lies within
  half a step of the exact one, plus those errors.
"""
import numpy as np
import pytest
import torch

import software_pipelined_tiled_gb300 as sptg

pytestmark = pytest.mark.gpu

BF16, F16, F32, S8, E4M3 = (torch.bfloat16, torch.float16, torch.float32, torch.int8,
                            torch.float8_e4m3fn)
U = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 0.0}
TINY = {BF16: 0.0, F16: 2.0 ** -25, F32: 0.0}  # half the smallest binary16 number


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    torch.cuda.synchronize()
    assert sptg.device_error() == 0


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def rand(g, *shape, dtype=BF16, std=1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * std).to(dtype)


def assert_close(got, ref, S, terms):
    u, tiny = U[got.dtype], TINY[got.dtype]
    e = (terms + 16) * 2.0 ** -23 * S
    bound = e + u * (ref.abs() + e) + tiny
    err = (got.double() - ref).abs()
    assert torch.isfinite(got.double()).all()
    assert (err <= bound).all(), f"max err/bound {float((err / bound.clamp(min=1e-300)).max()):.3f}"


# ------------------------------------------------------------------ the norm
def norm_reference(x, r, w, eps):
    t = x.double() + r.double()
    rstd = 1.0 / torch.sqrt((t * t).sum(1, keepdim=True) / t.shape[1] + eps)
    return t, t * rstd * w.double()


def check_norm(x, r, w, out_dtype, eps=1e-6, **kw):
    rows, cols = x.shape
    # the call may write h over x or r: the reference comes first
    t, v = norm_reference(x, r, w, eps)
    h, y, scales = sptg.add_rms_norm(x, r, w, eps=eps, out_dtype=out_dtype, **kw)
    torch.cuda.synchronize()
    u = U[x.dtype]
    # the 32-bit sum itself is off by half a unit of 32 bits
    assert ((h.double() - t).abs() <= u * t.abs() * (1 + 2.0 ** -10) + TINY[x.dtype]).all()
    rel = (cols + 32) * 2.0 ** -24
    if out_dtype == x.dtype:
        assert scales is None
        assert ((y.double() - v).abs() <= (u * (1 + rel) + rel) * v.abs() + TINY[x.dtype]).all()
        return
    top = 127.0 if out_dtype == S8 else 448.0
    a = v.abs().amax(1)
    assert ((scales.double() - a / top).abs() <= rel * a / top).all()
    q = y.float().double()
    exact = torch.where(a[:, None] > 0, v / (a[:, None] / top).clamp(min=1e-300), 0.0)
    half = (torch.full_like(exact, 0.5) if out_dtype == S8
            else torch.maximum(exact.abs() * 2.0 ** -4, torch.full_like(exact, 2.0 ** -10)))
    assert q.abs().max() <= top
    assert ((q - exact).abs() <= half * (1 + 2.0 ** -10) + 2 * rel * exact.abs()).all()


@pytest.mark.parametrize("out_dtype", [S8, E4M3, None])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8), (3, 7), (5, 64), (2, 1000), (9, 1024),
                                       (3, 1032), (1, 4096), (4, 4104), (2, 8192), (3, 8200),
                                       (2, 16384), (2, 16392), (1, 32768), (1, 32776), (2, 5001)])
def test_norm(rows, cols, dtype, out_dtype):
    g = gen(rows * 131 + cols)
    x, r = rand(g, rows, cols, dtype=dtype), rand(g, rows, cols, dtype=dtype, std=3.0)
    w = 1 + rand(g, cols, dtype=dtype, std=0.2)
    check_norm(x, r, w, out_dtype or dtype)


@pytest.mark.parametrize("out_dtype", [S8, E4M3, BF16])
def test_norm_strided_rows_and_in_place(out_dtype):
    g = gen(7)
    big_x, big_r = rand(g, 6, 300), rand(g, 6, 300)
    w = rand(g, 96)
    for off in (0, 8, 3):  # 16-byte aligned slices, and one that is not
        x, r = big_x[:, off:off + 96].clone(), big_r[:, off:off + 96]
        keep = big_r.clone()
        check_norm(x, r, w, out_dtype, h=r)  # h written over residual
        # nothing outside the slice changed
        mask = torch.ones(300, dtype=torch.bool, device="cuda")
        mask[off:off + 96] = False
        assert torch.equal(big_r[:, mask], keep[:, mask])
        xs = big_x[:, off:off + 96]
        check_norm(xs, r.clone(), w, out_dtype, h=xs)
    wide = torch.zeros(6, 200, dtype=out_dtype, device="cuda")
    check_norm(rand(g, 6, 96), rand(g, 6, 96), w, out_dtype, y=wide[:, 16:112])
    assert float(wide[:, :16].float().abs().sum()) == 0
    assert float(wide[:, 112:].float().abs().sum()) == 0


@pytest.mark.parametrize("cols", [64, 65, 5000])
@pytest.mark.parametrize("out_dtype", [S8, E4M3])
def test_norm_rows_of_zeros_infinities_and_nan(cols, out_dtype):
    g = gen(11)
    x, r, w = rand(g, 8, cols), rand(g, 8, cols), rand(g, cols)
    x[1], r[1] = 0, 0
    x[2, cols // 2] = float("inf")
    x[3, cols - 1] = float("nan")
    r[4] = -x[4]
    x[5, 0] = float("-inf")
    x[6], r[6] = 3e38, 0  # the sum of squares passes 32 bits
    w[3] = 0
    h, y, s = sptg.add_rms_norm(x, r, w, out_dtype=out_dtype)
    y = y.float()
    for row in (1, 4, 6):
        assert float(s[row]) == 0 and not y[row].any()
    for row in (2, 3, 5):
        assert torch.isnan(s[row]) and not y[row].any()
    torch.testing.assert_close(h.float(), (x.float() + r.float()).to(BF16).float(), rtol=0, atol=0,
                               equal_nan=True)
    fine = torch.tensor([0, 7], device="cuda")
    check_norm(x[fine], r[fine], w, out_dtype)


def test_norm_of_no_rows_and_no_columns():
    w = torch.ones(64, dtype=F16, device="cuda")
    e = torch.empty(0, 64, dtype=F16, device="cuda")
    h, y, s = sptg.add_rms_norm(e, e, w, out_dtype=S8)
    assert h.shape == (0, 64) and y.shape == (0, 64) and s.shape == (0,)
    e = torch.empty(3, 0, dtype=F16, device="cuda")
    sptg.add_rms_norm(e, e, w[:0], out_dtype=S8)


# ------------------------------------------------------------ 4-bit weights
def w4_inputs(g, m, n, k, group, dtype, xdtype, zeros):
    codes = torch.randint(0, 256, (n, k // 2), device="cuda", generator=g, dtype=torch.uint8)
    scales = (torch.rand(n, k // group, device="cuda", generator=g) * 0.02 + 1e-3).to(dtype)
    z = (torch.randint(0, 16, (n, k // group), device="cuda", generator=g, dtype=torch.uint8)
         if zeros else None)
    xs = None
    if xdtype in (S8, E4M3):
        xs = torch.rand(m, device="cuda", generator=g) * 0.01 + 1e-3
        x = torch.randint(-127, 128, (m, k), device="cuda", generator=g)
        x = x.to(S8) if xdtype == S8 else (x.float() * 3.5).to(E4M3)
    else:
        x = rand(g, m, k, dtype=xdtype)
    return x, codes, scales, z, xs


def w4_reference(x, codes, scales, z, xs):
    n, half = codes.shape
    group = 2 * half // scales.shape[1]
    w = torch.stack([codes & 15, codes >> 4], 2).reshape(n, 2 * half).double()
    w = w - (8.0 if z is None else z.double().repeat_interleave(group, 1))
    w = w * scales.double().repeat_interleave(group, 1)
    xd = x.float().double()
    if xs is not None:
        xd = xd * xs.double()[:, None]
    return xd @ w.t(), xd.abs() @ w.abs().t()


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("xdtype", [BF16, F16, S8, E4M3])
@pytest.mark.parametrize("m,n,k,group", [(1, 1, 32, 32), (1, 128, 128, 128), (3, 130, 256, 64),
                                         (8, 257, 288, 32), (9, 100, 512, 128), (16, 1000, 1088, 64),
                                         (17, 64, 2080, 32), (33, 300, 640, 128), (64, 129, 4096, 64),
                                         (65, 96, 384, 32), (130, 200, 1024, 128),
                                         (2, 4096, 4096, 128), (5, 40, 8192, 32)])
def test_w4(m, n, k, group, xdtype, zeros):
    g = gen(m * 7 + n + k)
    dtype = xdtype if xdtype in (BF16, F16) else (BF16 if m % 2 else F16)
    x, codes, scales, z, xs = w4_inputs(g, m, n, k, group, dtype, xdtype, zeros)
    ref, S = w4_reference(x, codes, scales, z, xs)
    y = sptg.gemm_w4(x, codes, scales, z, x_scales=xs)
    assert y.dtype == dtype and y.shape == (m, n)
    assert_close(y, ref, S, k)


def test_w4_strided_x_codes_and_out():
    g = gen(3)
    m, n, k = 5, 70, 128
    x, codes, scales, z, _ = w4_inputs(g, m, n, k, 64, F16, F16, True)
    ref, S = w4_reference(x, codes, scales, z, None)
    xw = torch.full((m, 3 * k), float("nan"), dtype=F16, device="cuda")
    xw[:, k:2 * k] = x
    cw = torch.full((n, 256), 255, dtype=torch.uint8, device="cuda")
    cw[:, 64:128] = codes
    out = torch.full((m, n + 9), 7.0, dtype=F16, device="cuda")
    sptg.gemm_w4(xw[:, k:2 * k], cw[:, 64:128], scales, z, out=out[:, 3:3 + n])
    assert_close(out[:, 3:3 + n], ref, S, k)
    assert (out[:, :3] == 7).all() and (out[:, 3 + n:] == 7).all()


def test_w4_infinite_and_nan_rows_stay_in_their_rows():
    g = gen(5)
    x, codes, scales, z, _ = w4_inputs(g, 12, 140, 512, 128, BF16, BF16, False)
    clean = sptg.gemm_w4(x, codes, scales, z)
    x[3, 100] = float("inf")
    x[11, 511] = float("nan")
    y = sptg.gemm_w4(x, codes, scales, z)
    keep = torch.tensor([i for i in range(12) if i not in (3, 11)], device="cuda")
    assert torch.equal(y[keep], clean[keep])
    assert torch.isnan(y[11]).all() and not torch.isfinite(y[3]).any()


def test_w4_empty():
    g = gen(6)
    x, codes, scales, z, _ = w4_inputs(g, 4, 64, 128, 128, BF16, BF16, False)
    assert sptg.gemm_w4(x[:0], codes, scales).shape == (0, 64)
    assert sptg.gemm_w4(x, codes[:0], scales[:0]).shape == (4, 0)
    y = sptg.gemm_w4(x[:, :0], codes[:, :0], scales[:, :0])
    assert y.shape == (4, 64) and not y.any()


def test_w4_same_bits_on_every_call():
    g = gen(8)
    x, codes, scales, z, _ = w4_inputs(g, 7, 520, 4096, 64, F16, F16, True)
    first = sptg.gemm_w4(x, codes, scales, z)
    for _ in range(5):
        assert torch.equal(first, sptg.gemm_w4(x, codes, scales, z))


# ------------------------------------------------------------------ experts
def offsets_of(sizes, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(sizes)]), dtype=torch.int32,
                        device="cuda")


SIZES = [
    [1], [0], [5, 0, 3], [0, 0, 17, 1, 0], [64, 64], [63, 65, 128, 1], [300, 0, 513, 31, 33],
    [97, 112, 113, 160], [0] * 40 + [7] + [0] * 30, [1] * 70, [1100], [16, 15, 48, 47, 49],
]


@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "-".join(map(str, s))[:24])
@pytest.mark.parametrize("n,k", [(8, 8), (264, 72), (520, 328), (128, 640)])
def test_grouped(sizes, n, k, dtype, out_dtype):
    g = gen(sum(sizes) * 3 + n + k)
    e, t = len(sizes), sum(sizes)
    X, W, dY = rand(g, t, k, dtype=dtype), rand(g, e, n, k, dtype=dtype), rand(g, t, n, dtype=dtype)
    off = offsets_of(sizes)
    y = sptg.grouped_gemm(X, W, off, out_dtype=out_dtype)
    dx = sptg.grouped_gemm_dx(dY, W, off, out_dtype=out_dtype)
    dw = sptg.grouped_gemm_dw(dY, X, off, out_dtype=out_dtype)
    assert y.shape == (t, n) and dx.shape == (t, k) and dw.shape == (e, n, k)
    a = 0
    for i, r in enumerate(sizes):
        x, w, d = X[a:a + r].double(), W[i].double(), dY[a:a + r].double()
        assert_close(y[a:a + r], x @ w.t(), x.abs() @ w.abs().t(), k)
        assert_close(dx[a:a + r], d @ w, d.abs() @ w.abs(), n)
        assert_close(dw[i], d.t() @ x, d.abs().t() @ x.abs(), r)
        a += r


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_grouped_infinities_and_nan_stay_in_their_experts(dtype):
    """Rows that share a tile or a chunk of the sum with another expert's rows never see its values."""
    g = gen(2)
    sizes, n, k = [5, 33, 70, 2], 136, 72
    X, W, dY = rand(g, 110, k, dtype=dtype), rand(g, 4, n, k, dtype=dtype), rand(g, 110, n, dtype=dtype)
    off = offsets_of(sizes)
    clean = [sptg.grouped_gemm(X, W, off), sptg.grouped_gemm_dx(dY, W, off),
             sptg.grouped_gemm_dw(dY, X, off)]
    for i, bad in ((1, float("inf")), (3, float("nan"))):
        a = int(off[i])
        X[a:a + sizes[i]] = bad
        dY[a:a + sizes[i]] = bad
        W[i] = bad
    y, dx, dw = (sptg.grouped_gemm(X, W, off), sptg.grouped_gemm_dx(dY, W, off),
                 sptg.grouped_gemm_dw(dY, X, off))
    for i in (0, 2):
        rows = slice(int(off[i]), int(off[i + 1]))
        assert torch.equal(y[rows], clean[0][rows])
        assert torch.equal(dx[rows], clean[1][rows])
        assert torch.equal(dw[i], clean[2][i])
    for i in (1, 3):
        rows = slice(int(off[i]), int(off[i + 1]))
        assert not torch.isfinite(y[rows]).any() and not torch.isfinite(dw[i]).any()


def test_grouped_rows_of_no_expert_are_zero():
    g = gen(4)
    X, W, dY = rand(g, 400, 64), rand(g, 3, 72, 64), rand(g, 400, 72)
    X[:37], X[337:], dY[:37], dY[337:] = (float("nan"),) * 4
    off = offsets_of([100, 0, 200], first=37)
    y, dx = sptg.grouped_gemm(X, W, off), sptg.grouped_gemm_dx(dY, W, off)
    dw = sptg.grouped_gemm_dw(dY, X, off)
    for out in (y, dx):
        assert not out[:37].any() and not out[337:].any()
        assert torch.isfinite(out).all()
    assert torch.isfinite(dw).all() and not dw[1].any()
    x, d, w = X[37:137].double(), dY[37:137].double(), W[0].double()
    assert_close(y[37:137], x @ w.t(), x.abs() @ w.abs().t(), 64)
    assert_close(dw[0], d.t() @ x, d.abs().t() @ x.abs(), 100)


def test_grouped_strided_rows():
    g = gen(9)
    sizes, n, k = [50, 3, 90], 80, 96
    off = offsets_of(sizes)
    Xw, dYw, W = rand(g, 143, 3 * k), rand(g, 143, 2 * n), rand(g, 3, n, k)
    X, dY = Xw[:, k:2 * k], dYw[:, n:]
    Yw = torch.full((143, n + 16), 7.0, dtype=F32, device="cuda")
    sptg.grouped_gemm(X, W, off, out=Yw[:, 8:8 + n])
    assert torch.equal(Yw[:, 8:8 + n], sptg.grouped_gemm(X.contiguous(), W, off, out_dtype=F32))
    assert (Yw[:, :8] == 7).all() and (Yw[:, 8 + n:] == 7).all()
    assert torch.equal(sptg.grouped_gemm_dx(dY, W, off),
                       sptg.grouped_gemm_dx(dY.contiguous(), W, off))
    assert torch.equal(sptg.grouped_gemm_dw(dY, X, off),
                       sptg.grouped_gemm_dw(dY.contiguous(), X.contiguous(), off))


def test_grouped_empty():
    W = torch.ones(3, 64, 72, dtype=BF16, device="cuda")
    off = offsets_of([0, 0, 0])
    X, dY = torch.empty(0, 72, dtype=BF16, device="cuda"), torch.empty(0, 64, dtype=BF16, device="cuda")
    assert sptg.grouped_gemm(X, W, off).shape == (0, 64)
    assert sptg.grouped_gemm_dx(dY, W, off).shape == (0, 72)
    dw = sptg.grouped_gemm_dw(dY, X, off)
    assert dw.shape == (3, 64, 72) and not dw.any()
    off = offsets_of([4, 0, 1])
    y = sptg.grouped_gemm(torch.empty(5, 0, dtype=BF16, device="cuda"), W[:, :, :0].contiguous(), off)
    assert y.shape == (5, 64) and not y.any()


@pytest.mark.parametrize("bad", [[-5, 10, 20, 30], [0, 25, 10, 30], [0, 10, 20, 5000], [40, 60, 50, 90]])
def test_grouped_offsets_out_of_range_touch_nothing_else(bad):
    """The kernels clamp the offsets; the guard zones around the outputs stay as they were."""
    g = gen(10)
    X, W, dY = rand(g, 64, 64), rand(g, 3, 64, 64), rand(g, 64, 64)
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    for call, rows in ((lambda o: sptg.grouped_gemm(X, W, off, out=o), 64),
                       (lambda o: sptg.grouped_gemm_dx(dY, W, off, out=o), 64),
                       (lambda o: sptg.grouped_gemm_dw(dY, X, off, out=o), 192)):
        guard = torch.full((rows + 128, 64), 7.0, dtype=BF16, device="cuda")
        o = guard[64:64 + rows]
        call(o if rows == 64 else o.view(3, 64, 64))
        assert (guard[:64] == 7).all() and (guard[64 + rows:] == 7).all()


def test_grouped_gradients_against_differences():
    """f = sum(G * Y) is linear in X and in W: a central difference along any direction is exact.

    Small integers keep every product and sum exact in 32 bits, so the two
    sides are equal, not merely close."""
    g = gen(12)
    sizes, n, k = [19, 0, 40, 70], 48, 56
    off = offsets_of(sizes)

    def ints(*shape):
        return torch.randint(-3, 4, shape, device="cuda", generator=g).to(BF16)

    X, W, G, dX, dW = ints(129, k), ints(4, n, k), ints(129, n), ints(129, k), ints(4, n, k)

    def f(x, w):
        return float((sptg.grouped_gemm(x, w, off, out_dtype=F32).double() * G.double()).sum())

    gx = sptg.grouped_gemm_dx(G, W, off, out_dtype=F32)
    gw = sptg.grouped_gemm_dw(G, X, off, out_dtype=F32)
    assert (f(X + dX, W) - f(X - dX, W)) / 2 == float((gx.double() * dX.double()).sum())
    assert (f(X, W + dW) - f(X, W - dW)) / 2 == float((gw.double() * dW.double()).sum())


def test_grouped_many_experts():
    g = gen(13)
    sizes = [(i * 7) % 5 for i in range(1024)]
    off = offsets_of(sizes)
    t = sum(sizes)
    X, W, dY = rand(g, t, 64), rand(g, 1024, 16, 64), rand(g, t, 16)
    e = torch.repeat_interleave(torch.arange(1024, device="cuda"), torch.tensor(sizes, device="cuda"))
    y, dx = sptg.grouped_gemm(X, W, off, out_dtype=F32), sptg.grouped_gemm_dx(dY, W, off, out_dtype=F32)
    Xd, Wd, dd = X.double(), W.double()[e], dY.double()
    assert_close(y, torch.einsum("tk,tnk->tn", Xd, Wd), torch.einsum("tk,tnk->tn", Xd.abs(), Wd.abs()), 64)
    assert_close(dx, torch.einsum("tn,tnk->tk", dd, Wd), torch.einsum("tn,tnk->tk", dd.abs(), Wd.abs()), 16)
    dw = sptg.grouped_gemm_dw(dY, X, off, out_dtype=F32)
    ref = torch.zeros(1024, 16, 64, dtype=torch.float64, device="cuda")
    ref.index_add_(0, e, dd[:, :, None] * Xd[:, None, :])
    mag = torch.zeros_like(ref).index_add_(0, e, dd.abs()[:, :, None] * Xd.abs()[:, None, :])
    assert_close(dw, ref, mag, 4)


# ------------------------------------------------------- streams and capture
def test_on_another_stream_and_in_a_graph():
    g = gen(14)
    x, r, w = rand(g, 4, 512), rand(g, 4, 512), rand(g, 512)
    _, codes, scales, z, _ = w4_inputs(g, 4, 256, 512, 64, BF16, BF16, True)
    W, off = rand(g, 2, 64, 512), offsets_of([1, 3])

    def step():
        h, q, s = sptg.add_rms_norm(x, r, w, out_dtype=S8)
        y = sptg.gemm_w4(q, codes, scales, z, x_scales=s)
        z16 = sptg.grouped_gemm(h, W, off)
        return h, q, s, y, z16, sptg.grouped_gemm_dx(z16, W, off), sptg.grouped_gemm_dw(z16, h, off)

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    side.wait_stream(torch.cuda.current_stream())
    y = sptg.gemm_w4(x, codes, scales, z, stream=side)
    side.synchronize()
    assert torch.equal(y, sptg.gemm_w4(x, codes, scales, z))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caught = step()
    x.copy_(rand(g, 4, 512))
    off.copy_(offsets_of([4, 0]))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(step(), caught):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ----------------------------------------------------------------- refusals
def test_python_refusals():
    g = gen(15)
    x, w = rand(g, 4, 64), rand(g, 64)
    for bad in (dict(out_dtype=F16), dict(out_dtype=F32), dict(h=rand(g, 4, 65)),
                dict(y=torch.empty(4, 64, dtype=S8, device="cuda"), scales=torch.empty(3, device="cuda")),
                dict(scales=torch.empty(4, device="cuda")), dict(h=x.t().contiguous().t())):
        with pytest.raises(ValueError):
            sptg.add_rms_norm(x, x, w, **bad)
    with pytest.raises(ValueError):
        sptg.add_rms_norm(x.float(), x.float(), w.float())
    with pytest.raises(ValueError):
        sptg.add_rms_norm(x, x.half(), w)
    with pytest.raises(ValueError):
        sptg.add_rms_norm(x, x, w.cpu())
    with pytest.raises(sptg.SptgError) as e:
        sptg.add_rms_norm(x, x, w, eps=0.0)
    assert e.value.status == -1
    x, codes, scales, z, _ = w4_inputs(g, 4, 16, 128, 64, BF16, BF16, True)
    q = torch.zeros(4, 128, dtype=S8, device="cuda")
    one = torch.ones(4, device="cuda")
    for args, kw in (((x.half(), codes, scales), {}), ((x, codes.int(), scales), {}),
                     ((x, codes, scales[:8]), {}), ((x, codes[:, :32], scales), {}),
                     ((x, codes, scales, z[:8]), {}), ((x, codes, scales, z.float()), {}),
                     ((x, codes, scales), dict(x_scales=one)), ((q, codes, scales), {}),
                     ((q, codes, scales), dict(x_scales=one[:3])),
                     ((x, codes, scales), dict(out=torch.empty(4, 15, dtype=BF16, device="cuda"))),
                     ((x, codes, scales[:, :0]), {})):
        with pytest.raises(ValueError):
            sptg.gemm_w4(*args, **kw)
    with pytest.raises(sptg.SptgError) as e:  # groups of 16
        sptg.gemm_w4(x, codes, torch.ones(16, 8, dtype=BF16, device="cuda"))
    assert e.value.status == -1
    X, W, off = rand(g, 8, 64), rand(g, 2, 32, 64), offsets_of([3, 5])
    for args, kw in (((X.half(), W, off), {}), ((X, W, off.long()), {}), ((X, W, off[:2]), {}),
                     ((X, W.transpose(1, 2), off), {}), ((X[:, :32], W, off), {}),
                     ((X, W, off.cpu()), {}), ((X, W, off), dict(out_dtype=F16)),
                     ((X, W, off), dict(out=torch.empty(8, 64, dtype=BF16, device="cuda")))):
        with pytest.raises(ValueError):
            sptg.grouped_gemm(*args, **kw)
    with pytest.raises(ValueError):
        sptg.grouped_gemm_dx(X, W, off)
    with pytest.raises(ValueError):
        sptg.grouped_gemm_dw(X, X[:7], off)
    with pytest.raises(sptg.SptgError) as e:  # rows of 60 values are not a multiple of 16 bytes
        sptg.grouped_gemm(rand(g, 8, 60), rand(g, 2, 32, 60), off)
    assert e.value.status == -2


# --------------------------------------------------------------- the example
def test_example_layer():
    """The operators together, against a float32 version, and the experts' gradients against autograd.

    The bounds: int8 rows carry a relative error of about 1/127/sqrt(12) of their
    largest value (4 to 5 times their root mean square), 0.3 % to 1 % of the
    projection that they enter, and each of the four bfloat16 roundings on the
    way 0.2 %; 2 % of the result's norm holds them together.  The gradients see
    roundings alone: 1 %."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    r = example.main(["--rows", "37", "--hidden", "512", "--inner", "384", "--experts", "8"])
    assert r["distance"] < 0.02
    kept, layer = r["kept"], r["layer"]
    up, down = (layer[n].float().requires_grad_() for n in ("up", "down"))
    rows = kept["sorted_rows"].float().requires_grad_()
    off, out = kept["offsets"].tolist(), []
    for e in range(8):
        s = slice(off[e], off[e + 1])
        out.append(torch.nn.functional.silu(rows[s] @ up[e].t()) @ down[e].t())
    (torch.cat(out) * kept["out"].float()[kept["rows"]] * kept["weight"][:, None]).sum().backward()
    for name, ref in (("up", up.grad), ("down", down.grad), ("rows", rows.grad)):
        got = r["grads"][name].float()
        assert float((got - ref).norm() / ref.norm()) < 0.01, name


# the choices of kernel that row counts make, at widths that fill and do not fill their threads
@pytest.mark.parametrize("out_dtype", [S8, E4M3, None])
@pytest.mark.parametrize("rows,cols", [(700, 4096), (650, 3000), (1400, 4104), (1500, 5000),
                                       (930, 8192), (460, 16384), (470, 12000), (300, 2048), (33, 520)])
def test_norm_of_many_rows(rows, cols, out_dtype):
    g = gen(rows + cols)
    dtype = BF16 if rows % 2 else F16
    x, r = rand(g, rows, cols, dtype=dtype), rand(g, rows, cols, dtype=dtype, std=3.0)
    w = 1 + rand(g, cols, dtype=dtype, std=0.2)
    check_norm(x, r, w, out_dtype or dtype)
    check_norm(x, r, w, out_dtype or dtype, h=r)  # in place


# Long sums with a 32-bit output. All terms are positive, so every rounding toward zero adds up: a
# part of 512 takes 32 steps of the tensor core, each rounding its running sum at most twice by a unit
# of 2^-23; with the running sum growing evenly that is 32 units of 2^-23 of the part. The parts are
# rounded to nearest as they are added: half a unit each, twelve parts at most.
@pytest.mark.parametrize("length", [900, 1024, 1025, 4100, 6000])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_grouped_long_sums_in_32_bits(length, dtype):
    g = gen(length)
    bound = 32 * 2.0 ** -23 + 12 * 2.0 ** -24
    n, k, sizes = 72, 200, [3, length, 20]
    t = sum(sizes)
    off = offsets_of(sizes)

    def positive(*shape):
        return (torch.rand(*shape, device="cuda", generator=g) + 0.5).to(dtype)

    X, dY = positive(t, k), positive(t, n)
    dw = sptg.grouped_gemm_dw(dY, X, off, out_dtype=F32)
    ref = dY[3:3 + length].double().t() @ X[3:3 + length].double()
    assert ((dw[1].double() - ref).abs() <= bound * ref).all()
    long_k = length // 8 * 8
    for rows in (20, 300):
        off = offsets_of([rows, rows])
        X, W = positive(2 * rows, long_k), positive(2, n, long_k)
        y = sptg.grouped_gemm(X, W, off, out_dtype=F32)
        ref = torch.cat([X[:rows].double() @ W[0].double().t(), X[rows:].double() @ W[1].double().t()])
        assert ((y.double() - ref).abs() <= bound * ref).all()
        dY, W = positive(2 * rows, long_k), positive(2, long_k, n)
        dx = sptg.grouped_gemm_dx(dY, W, off, out_dtype=F32)
        ref = torch.cat([dY[:rows].double() @ W[0].double(), dY[rows:].double() @ W[1].double()])
        assert ((dx.double() - ref).abs() <= bound * ref).all()


# Offsets past 32 bits: the last rows of tensors of more than 2^31 elements.
def test_norm_past_two_to_the_31():
    rows, cols = (1 << 31) // 8192 + 40, 8192
    x = torch.zeros(rows, cols, device="cuda", dtype=BF16)
    r = torch.zeros(rows, cols, device="cuda", dtype=BF16)
    g = gen(31)
    x[-30:], r[-30:], w = rand(g, 30, cols), rand(g, 30, cols), rand(g, cols)
    h, y, scales = sptg.add_rms_norm(x, r, w, out_dtype=S8)
    assert (scales[:-30] == 0).all()
    # check_norm's bounds
    t, v = norm_reference(x[-30:], r[-30:], w, 1e-6)
    rel, a = (cols + 32) * 2.0 ** -24, v.abs().amax(1)
    assert ((h[-30:].double() - t).abs() <= U[BF16] * t.abs() * (1 + 2.0 ** -10)).all()
    assert ((scales[-30:].double() - a / 127.0).abs() <= rel * a / 127.0).all()
    exact = v / (a[:, None] / 127.0)
    assert ((y[-30:].double() - exact).abs() <= 0.5 * (1 + 2.0 ** -10) + 2 * rel * exact.abs()).all()


@pytest.mark.parametrize("m", [1, 16])
def test_w4_past_two_to_the_31(m):
    g = gen(m)
    k, group = 8192, 128
    n = (1 << 32) // k + 200  # more than 2^31 bytes of codes
    codes = torch.zeros(n, k // 2, device="cuda", dtype=torch.uint8)
    scales = torch.zeros(n, k // group, device="cuda", dtype=BF16)
    x, c, s, _, _ = w4_inputs(g, m, 150, k, group, BF16, BF16, False)
    codes[-150:], scales[-150:] = c, s
    y = sptg.gemm_w4(x, codes, scales)
    ref, S = w4_reference(x, c, s, None, None)
    assert_close(y[:, -150:], ref, S, k)
    assert (y[:, :-150] == 0).all()


def test_grouped_past_two_to_the_31():
    g = gen(5)
    e, n, k = 36, 8192, 8192
    W = torch.zeros(e, n, k, device="cuda", dtype=BF16)
    W[-1] = rand(g, n, k, std=0.05)
    off = offsets_of([0] * (e - 1) + [40])
    X, dY = rand(g, 40, k), rand(g, 40, n)
    y, dx = sptg.grouped_gemm(X, W, off), sptg.grouped_gemm_dx(dY, W, off)
    w = W[-1].double()
    assert_close(y, X.double() @ w.t(), X.double().abs() @ w.abs().t(), k)
    assert_close(dx, dY.double() @ w, dY.double().abs() @ w.abs(), n)
    del W, w
    dw = sptg.grouped_gemm_dw(dY, X, off)
    assert (dw[:-1] == 0).all()
    assert_close(dw[-1], dY.double().t() @ X.double(), dY.double().abs().t() @ X.double().abs(), 40)
