"""The operators around the dense products where a call is unusual: their waits, their edges and their sizes."""
import threading

import pytest
import torch

import software_pipelined_tiled_gb300 as sptg
from test_layer_ops_gpu import (BF16, E4M3, F16, F32, S8, assert_close, check_norm, gen, offsets_of, rand,
                                w4_inputs, w4_reference)

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


# ------------------------------------------------------------------ the norm
WARP_2, WARP_4, BLOCK_2, BLOCK_4, RING, ANY = range(6)  # its kernels, by last_config's kind


@pytest.mark.parametrize("out_dtype", [S8, E4M3, None])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("cols", [4104, 4352, 5128, 6144, 8192, 16384])
def test_norm_ring_has_as_many_blocks_as_the_gpu_holds(cols, dtype, out_dtype):
    """Rows are dealt out to all blocks from the start: one that waits for an SM makes the call longer."""
    x = torch.ones(3000, cols, dtype=dtype, device="cuda")
    sptg.add_rms_norm(x, x, x[0], out_dtype=out_dtype)
    c, sms = chosen(), torch.cuda.get_device_properties(0).multi_processor_count
    assert c["kind"] == RING and c["grid"] % sms == 0
    per_sm, registers = c["grid"] // sms, -(-c["regs"] // 8) * 8  # handed out in eights

    # an SM's registers lie in four parts of 16384, and a warp in one of them; of its 228 KB of shared
    # memory, 1 KB a block are the system's
    warps = 4 * (16384 // (32 * registers))

    def fits(n):
        return n * c["threads"] // 32 <= warps and n * (c["smem"] + 1024 + 1024) <= 228 * 1024
    assert fits(per_sm) and not fits(per_sm + 1)


@pytest.mark.parametrize("out_dtype", [S8, E4M3, None])
@pytest.mark.parametrize("rows,cols,kind", [(40, 512, WARP_2), (33, 520, WARP_4), (300, 2048, BLOCK_2),
                                            (20, 4096, BLOCK_2), (700, 4096, BLOCK_4), (650, 3000, BLOCK_4),
                                            (300, 6144, BLOCK_2), (1900, 4104, RING), (1500, 5000, RING),
                                            (1500, 6144, RING), (930, 8192, RING), (470, 12000, RING),
                                            (460, 16384, RING), (5, 16392, ANY), (700, 4095, ANY)])
def test_norm_by_each_of_its_kernels(rows, cols, kind, out_dtype):
    g = gen(rows + cols)
    dtype = BF16 if rows % 20 else F16
    x, r = rand(g, rows, cols, dtype=dtype), rand(g, rows, cols, dtype=dtype, std=3.0)
    w = 1 + rand(g, cols, dtype=dtype, std=0.2)
    check_norm(x, r, w, out_dtype or dtype)
    assert chosen()["kind"] == kind
    check_norm(x, r, w, out_dtype or dtype, h=r)  # in place


@pytest.mark.parametrize("out_dtype", [S8, BF16])
def test_norm_wait_that_runs_out_is_reported_and_the_context_survives(out_dtype):
    # each block's second row never arrives: its wait runs out after 100 ms, nothing is copied behind
    # it, and what was in flight lands before the block leaves
    g = gen(50)
    x, r, w = rand(g, 2500, 8192), rand(g, 2500, 8192), rand(g, 8192)
    cfg = sptg.Config()
    cfg.timeout_ms, cfg.inject_stall = 100, 1
    sptg.add_rms_norm(x, r, w, out_dtype=out_dtype, config=cfg)
    assert chosen()["kind"] == RING
    assert sptg.device_error() == -5
    assert sptg.device_error() == 0  # the word was cleared
    check_norm(x, r, w, out_dtype)
    assert chosen()["kind"] == RING


def test_norm_config_refusals():
    x = rand(gen(51), 2, 64)
    for bad in (dict(timeout_ms=-1), dict(inject_stall=2), dict(inject_stall=-1)):
        cfg = sptg.Config()
        for k, v in bad.items():
            setattr(cfg, k, v)
        with pytest.raises(sptg.SptgError) as e:
            sptg.add_rms_norm(x, x, x[0], config=cfg)
        assert e.value.status == -1


@pytest.mark.parametrize("out_dtype", [S8, E4M3, BF16])
@pytest.mark.parametrize("rows,cols", [(5, 64), (5, 1024), (3, 3000), (640, 4096), (4, 65), (2, 16392),
                                       (2000, 8192)])
def test_norm_of_rows_whose_products_with_the_weight_pass_32_bits(rows, cols, out_dtype):
    g = gen(rows + cols)
    x, r, w = rand(g, rows, cols), rand(g, rows, cols, std=3.0), rand(g, cols, std=3e30)
    x[1::2] *= 1e10  # about 1e41 with the weight, 1e31 when normalised
    check_norm(x, r, w, out_dtype)
    if out_dtype != BF16:
        x[1, cols // 2], x[0, 0] = float("inf"), float("nan")
        s = sptg.add_rms_norm(x, r, w, out_dtype=out_dtype)[2]
        assert torch.isnan(s[:2]).all() and torch.isfinite(s[2:]).all()
        x[0, 0], x[1, cols // 2] = 1.0, 1.0
        w[5] = float("inf")
        assert torch.isnan(sptg.add_rms_norm(x, r, w, out_dtype=out_dtype)[2]).all()


@pytest.mark.parametrize("out_dtype", [S8, E4M3])
def test_norm_of_rows_without_columns_has_scales_of_zero(out_dtype):
    e = torch.empty(3, 0, dtype=F16, device="cuda")
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        s = torch.full((3,), 7.0, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        assert sptg.add_rms_norm(e, e, e[0], out_dtype=out_dtype, scales=s, stream=stream)[2] is s
        own = sptg.add_rms_norm(e, e, e[0], out_dtype=out_dtype, stream=stream)[2]
        side.synchronize()
        assert (s == 0).all() and (own == 0).all()


# ------------------------------------------------------------ 4-bit weights
@pytest.mark.parametrize("group,block", [(32, 32), (128, 64)])
def test_w4_of_more_rows_than_a_grid_is_high(group, block):
    m, n = block * 65535 + 33, 16
    g = gen(group)
    x, codes, scales, z, _ = w4_inputs(g, m, n, group, group, BF16, BF16, True)
    y = sptg.gemm_w4(x, codes, scales, z)
    assert chosen()["launches"] == 2
    for a in (slice(0, 100), slice(m // 2, m // 2 + 100), slice(m - 200, m)):
        ref, S = w4_reference(x[a], codes, scales, z, None)
        assert_close(y[a], ref, S, group)
    assert torch.equal(y[-65:], sptg.gemm_w4(x[-65:], codes, scales, z))


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("xdtype", [BF16, F16, S8, E4M3])
@pytest.mark.parametrize("m,n,k,group", [(1, 300, 4096, 128), (3, 4100, 8192, 64), (5, 70, 2080, 32),
                                         (8, 1000, 8192, 128), (16, 300, 4096, 64), (40, 200, 2048, 32)])
def test_w4_weights_at_their_zero_points_add_nothing(m, n, k, group, xdtype, zeros):
    """All codes equal their zero points: 0.  One code a row that does not: its product alone, rounded once."""
    g = gen(m + n)
    dtype = xdtype if xdtype in (BF16, F16) else BF16
    x, _, scales, z, xs = w4_inputs(g, m, n, k, group, dtype, xdtype, zeros)
    if xdtype in (BF16, F16):
        x = x.abs() * 100  # of one sign, so that nothing cancels that should not be there
    code = (torch.full((n, k), 8, dtype=torch.uint8, device="cuda") if z is None
            else z.repeat_interleave(group, 1))
    codes = code[:, 0::2] | code[:, 1::2] << 4
    assert not sptg.gemm_w4(x, codes, scales, z, x_scales=xs).any()
    at = torch.randint(0, k, (n,), device="cuda", generator=g)
    rows = torch.arange(n, device="cuda")
    old = code[rows, at].int()
    code[rows, at] = torch.where(old < 15, old + 1, old - 1).to(torch.uint8)
    codes = code[:, 0::2] | code[:, 1::2] << 4
    one = torch.where(old < 15, 1.0, -1.0) * scales[rows, at // group].float()
    want = x[:, at].float() * one  # exact in 32 bits
    if xs is not None:
        want = want * xs[:, None]
    assert torch.equal(sptg.gemm_w4(x, codes, scales, z, x_scales=xs), want.to(dtype))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("m,n,k,group", [(1, 70, 256, 64), (4, 300, 8192, 128), (8, 130, 2080, 32),
                                         (12, 140, 512, 128)])
def test_w4_rows_with_infinities_give_what_the_formula_gives(m, n, k, group, zeros, dtype):
    g = gen(m + n)
    x, codes, scales, z, _ = w4_inputs(g, m, n, k, group, dtype, dtype, zeros)
    clean = sptg.gemm_w4(x, codes, scales, z)
    inf = float("inf")
    x[0, 100] = inf
    if m > 1:
        x[1, 5], x[1, k - 1] = -inf, -inf
        x[2, 7], x[2, 200] = inf, -inf
        x[3, k // 2] = float("nan")
    y = sptg.gemm_w4(x, codes, scales, z)
    w = torch.stack([codes & 15, codes >> 4], 2).reshape(n, k).double()
    w = w - (8.0 if z is None else z.double().repeat_interleave(group, 1))
    w = w * scales.double().repeat_interleave(group, 1)
    for i in range(min(m, 4)):
        bad = ~torch.isfinite(x[i])
        ref = (x[i, bad].double()[None] * w[:, bad]).sum(1)  # what is finite beside them changes nothing
        assert torch.equal(torch.isnan(y[i]), torch.isnan(ref))
        fine = ~torch.isnan(ref)
        assert torch.equal(y[i].double()[fine], ref[fine])
    assert torch.equal(y[4:], clean[4:])


# ----------------------------------------------------------- one after another
@pytest.mark.parametrize("m", [1, 7, 33])
def test_operands_written_by_the_call_before(m):
    """Weights, scales and zero points that the previous call on the stream has just written.

    A kernel starts while the one before it ends; the same calls one at a time give the same bits."""
    n, k, group = 520, 4096, 64
    groups = k // group

    def steps(wait):
        g = gen(52)
        x, codes = rand(g, m, k), torch.randint(0, 256, (n, k // 2), device="cuda", generator=g,
                                                dtype=torch.uint8)
        weight, row = torch.empty(k, dtype=BF16, device="cuda"), rand(g, 1, k)
        scales, zeros = torch.empty(n, groups, dtype=BF16, device="cuda"), torch.empty(n, groups, dtype=S8, device="cuda")
        ones, none = torch.ones(k, dtype=BF16, device="cuda"), torch.zeros(n, groups, dtype=BF16, device="cuda")
        kept = []
        for _ in range(12):
            a, b = rand(g, n, groups), rand(g, n, groups)
            sptg.add_rms_norm(row, rand(g, 1, k), ones, h=row, y=weight[None])
            wait()
            h, y, _ = sptg.add_rms_norm(x, x, weight)
            wait()
            sptg.add_rms_norm(a, none, ones[:groups], y=zeros)
            wait()
            kept += [y, sptg.gemm_w4(x, codes, a, zeros.view(torch.uint8))]
            wait()
            sptg.add_rms_norm(b, none, ones[:groups], y=scales)
            wait()
            kept.append(sptg.gemm_w4(x, codes, scales, zeros.view(torch.uint8)))
            wait()
        torch.cuda.synchronize()
        return kept

    for a, b in zip(steps(torch.cuda.synchronize), steps(lambda: None)):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ experts
@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [[0, 40, 10, 64], [0, 90, 20, 30], [30, 10, 50, 40], [-7, -3, 200, 60], [70, 0, 0, 0],
                                 [0, 300, 7, 250] * 20, [5, 0] * 40])
def test_grouped_offsets_that_decrease_are_raised(bad, out_dtype):
    g = gen(len(bad) + bad[1])
    t, n, k, e = 290, 72, 136, len(bad) - 1
    X, W, dY = rand(g, t, k), rand(g, e, n, k), rand(g, t, n)
    raw = torch.tensor(bad, dtype=torch.int32)
    off, good = raw.cuda(), torch.cummax(raw.clamp(0, t), 0).values.cuda()
    for call, args in ((sptg.grouped_gemm, (X, W)), (sptg.grouped_gemm_dx, (dY, W)), (sptg.grouped_gemm_dw, (dY, X))):
        for _ in range(3):
            assert torch.equal(call(*args, off, out_dtype=out_dtype), call(*args, good, out_dtype=out_dtype))
    y = sptg.grouped_gemm(X, W, off, out_dtype=out_dtype)
    assert not y[:int(good[0])].any() and not y[int(good[-1]):].any()


@pytest.mark.parametrize("out_dtype", [None, F32])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_grouped_gemm_in_automatic_differentiation(dtype, out_dtype):
    """Against the formula in 64 bits, by the bounds of a product (the gradient of Y is exact in 16 bits)."""
    g = gen(31)
    sizes, n, k = [19, 0, 40, 70], 48, 56
    off, o = offsets_of(sizes), [0, 19, 19, 59, 129]
    X, W, G = rand(g, 135, k, dtype=dtype), rand(g, 4, n, k, dtype=dtype), rand(g, 135, n, dtype=dtype)
    for t in (X, W):
        t.requires_grad_()
    y = sptg.grouped_gemm(X, W, off, out_dtype=out_dtype)
    assert torch.equal(y, sptg.grouped_gemm(X.detach(), W.detach(), off, out_dtype=out_dtype))
    y.backward(G.to(y.dtype))
    assert X.grad.dtype == dtype and W.grad.dtype == dtype
    x, w, d = X.detach().double(), W.detach().double(), G.double()
    for e in range(4):
        r = slice(o[e], o[e + 1])
        assert_close(X.grad[r], d[r] @ w[e], d[r].abs() @ w[e].abs(), n)
        assert_close(W.grad[e], d[r].t() @ x[r], d[r].abs().t() @ x[r].abs(), o[e + 1] - o[e])
    assert not X.grad[129:].any()  # rows of no expert
    assert torch.equal(X.grad, sptg.grouped_gemm_dx(G, W.detach(), off))
    assert torch.equal(W.grad, sptg.grouped_gemm_dw(G, X.detach(), off))


def test_grouped_gemm_gradients_in_unusual_graphs():
    g = gen(33)
    off = offsets_of([30, 2, 0, 68])
    X, W = rand(g, 100, 64).requires_grad_(), rand(g, 4, 32, 64).requires_grad_()
    ones = torch.ones(100, 32, dtype=BF16, device="cuda")
    want = sptg.grouped_gemm_dx(ones, W.detach(), off), sptg.grouped_gemm_dw(ones, X.detach(), off)
    sptg.grouped_gemm(X, W, off).sum().backward()  # an expanded gradient, strides of zero
    assert torch.equal(X.grad, want[0]) and torch.equal(W.grad, want[1])
    wide = torch.ones(100 * 32 + 1, dtype=BF16, device="cuda")[1:].view(100, 32)  # not 16-byte aligned
    gx, = torch.autograd.grad(sptg.grouped_gemm(X, W.detach(), off), X, wide)
    assert torch.equal(gx, want[0])
    gw, = torch.autograd.grad(sptg.grouped_gemm(X.detach(), W, off), W, ones)
    assert torch.equal(gw, want[1])
    with torch.no_grad():
        assert not sptg.grouped_gemm(X, W, off).requires_grad
        sptg.grouped_gemm(X, W, off, out=torch.empty_like(ones))
    with pytest.raises(ValueError):
        sptg.grouped_gemm(X, W, off, out=torch.empty_like(ones))
    with pytest.raises(ValueError):
        sptg.grouped_gemm(X, W, off[:3])
    gx, = torch.autograd.grad(sptg.grouped_gemm(X, W, off), X, ones, create_graph=True)
    with pytest.raises(RuntimeError):  # the gradient has no derivative of its own
        gx.sum().backward()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        side.wait_stream(torch.cuda.current_stream())
        y = sptg.grouped_gemm(X, W, off, stream=stream)
        torch.cuda.current_stream().wait_stream(side)
        gx, gw = torch.autograd.grad(y, (X, W), ones)
        assert torch.equal(gx, want[0]) and torch.equal(gw, want[1])


# ------------------------------------------------------------------- streams
def _operators(g):
    """name: (operator, its tensors, other arguments)."""
    t, n, k, e = 4096, 1024, 2048, 4
    off = offsets_of([1000, 0, 3000, 96])
    X, W, dY = rand(g, t, k), rand(g, e, n, k), rand(g, t, n)
    w4x, codes, scales, z, xs = w4_inputs(g, 256, 4096, 4096, 64, BF16, S8, True)
    return {"norm": (sptg.add_rms_norm, [rand(g, t, k), rand(g, t, k), rand(g, k)], dict(out_dtype=S8)),
            "w4": (lambda x, c, s, z, xs, **kw: sptg.gemm_w4(x, c, s, z, x_scales=xs, **kw),
                   [w4x, codes, scales, z, xs], {}),
            "y": (sptg.grouped_gemm, [X, W, off], {}), "dx": (sptg.grouped_gemm_dx, [dY, W, off], {}),
            "dw": (sptg.grouped_gemm_dw, [dY, X, off], {})}


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["norm", "w4", "y", "dx", "dw"])
def test_tensors_dropped_after_a_call_on_another_stream_stay_as_they_are(name, raw):
    """The stream is still busy with something else when the inputs are dropped and their memory is asked for."""
    f, args, kw = _operators(gen(60))[name]
    want = f(*args, **kw)
    side = torch.cuda.Stream()
    copies = [a.clone() for a in args]
    sizes = [a.numel() * a.element_size() for a in args]
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)  # some 20 ms
    got = f(*copies, stream=side.cuda_stream if raw else side, **kw)
    del copies
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes]
    side.synchronize()
    for a, b in zip(*((want, got) if isinstance(got, tuple) else ((want,), (got,)))):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    del junk


@pytest.mark.parametrize("name", ["norm", "w4", "w4 row", "y", "dx", "dw", "gemm", "gemm skinny", "gemm int8"])
def test_first_call_of_a_host_thread(name):
    """A thread that has made no CUDA call of its own: one of a pool, or automatic differentiation's."""
    g = gen(61)
    if name.startswith("gemm"):
        dtype, m = (S8, 256) if name == "gemm int8" else (BF16, 64 if "skinny" in name else 256)
        A, B = (torch.randint(-9, 9, (r, 512), device="cuda", generator=g).to(dtype) for r in (m, 384))
        f, args, kw = sptg.gemm, [A, B], {}
    else:
        f, args, kw = _operators(g)[name.split()[0]]
        if name == "w4 row":
            args = [a[:1] if a is args[0] or a is args[4] else a for a in args]
    want, got = f(*args, **kw), []
    # new addresses, so that no tensor map of theirs is at hand
    copies = [a.clone() for a in args]
    torch.cuda.synchronize()

    def work():
        try:
            got.append(f(*copies, **kw))
        except Exception as e:  # reported below, on the main thread
            got.append(e)

    thread = threading.Thread(target=work)
    thread.start()
    thread.join()
    torch.cuda.synchronize()
    assert not isinstance(got[0], Exception), got[0]
    for a, b in zip(*((want, got[0]) if isinstance(want, tuple) else ((want,), (got[0],)))):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_host_threads_on_streams_of_their_own():
    """Every operator at the same time as the others, and as the dense product, gives the bits that it gives alone."""
    g = gen(62)
    calls = [(f, args, kw) for f, args, kw in _operators(g).values()]
    x, codes, scales, z, xs = w4_inputs(g, 5, 4096, 4096, 64, F16, F16, True)
    calls.append((sptg.gemm_w4, [x, codes, scales, z], {}))
    x, codes, scales, z, xs = w4_inputs(g, 16, 1000, 4096, 128, BF16, BF16, False)  # two blocks to an SM would fit
    calls.append((sptg.gemm_w4, [x, codes, scales, z], {}))
    calls.append((sptg.gemm, [rand(g, 512, 2048), rand(g, 768, 2048)], {}))
    alone = [f(*args, **kw) for f, args, kw in calls]
    torch.cuda.synchronize()
    results = {}

    def work(t):
        try:
            stream, out = torch.cuda.Stream(), []
            with torch.cuda.stream(stream):
                for rep in range(8):
                    for j in range(len(calls)):
                        i = (j + t + rep) % len(calls)  # threads interleave different kernels
                        f, args, kw = calls[i]
                        out.append((i, f(*args, **kw)))
            stream.synchronize()
            results[t] = out
        except Exception as e:  # reported below, on the main thread
            results[t] = e

    threads = [threading.Thread(target=work, args=(t,)) for t in range(4)]
    for thread in threads:
        thread.start()
    for thread in threads:
        thread.join()
    torch.cuda.synchronize()
    for t in range(4):
        assert not isinstance(results[t], Exception), results[t]
        for i, got in results[t]:
            for a, b in zip(*((v if isinstance(v, tuple) else (v,)) for v in (alone[i], got))):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i
