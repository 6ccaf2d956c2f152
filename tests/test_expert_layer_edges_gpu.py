"""The operators around an expert layer where a call is unusual: each of their kernels, sizes past 32 bits, streams,
threads, graphs, waits, and a run of all of them together."""
import threading

import pytest
import torch

import software_pipelined_tiled_gb300 as sptg
from test_expert_layer_gpu import (BF16, F16, F32, I32, INF, UNIT, assert_within, check_dispatch, check_gate_norm,
                                   check_route, combine_reference, distance, dlogits_reference, gate_norm_reference,
                                   gate_of, gen, rand)
from test_layer_ops_edges_gpu import chosen

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    torch.cuda.synchronize()
    assert sptg.device_error() == 0


# ------------------------------------------------------------------- routing
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("e,top,groups,lanes,per", [(64, 8, 1, 8, 8), (50, 8, 8, 8, 8), (128, 8, 1, 8, 16), (96, 6, 4, 8, 16),
                                                    (128, 16, 1, 16, 8), (256, 8, 8, 32, 8), (136, 3, 1, 32, 8),
                                                    (96, 4, 32, 32, 8), (512, 10, 1, 32, 16), (1024, 16, 16, 32, 32),
                                                    (1023, 4, 3, 32, 64)])
def test_route_by_each_of_its_kernels_in_several_turns(e, top, groups, lanes, per, dtype):
    g = gen(e + top)
    rows = 20011
    logits, bias = rand(g, rows, e, dtype=dtype, std=1.5), rand(g, e, dtype=F32, std=0.05)
    how = dict(groups=groups, top_groups=max(1, groups // 2 + 1) if groups > 1 else 1)
    if e == 50:
        how = dict()  # 50 experts in 8 groups is no division: one group, in parts of 8
    for scores in ("sigmoid", "softmax"):
        check_route(logits, top, scores=scores, bias=bias, **how)
        check_route(logits, top, scores=scores, renormalize=False, **how)
    c = chosen()
    assert (c["lanes"], c["per"]) == (lanes, per) and c["turns"] == lanes // (8 if top <= 8 else 16)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_route_of_rows_whose_picks_lie_within_a_few_units_of_each_other(scores):
    """Logits in steps of one unit and biases that undo most of it: keys that 32 bits cannot tell apart, many to a lane."""
    g = gen(70)
    rows, e = 500, 256
    steps = torch.randint(0, 64, (rows, e), device="cuda", generator=g)
    logits = (0.5 + steps * 2.0 ** -24).float()
    bias = -(torch.randint(0, 8, (e,), device="cuda", generator=g) * 2.0 ** -27).float()
    for groups, top_groups in ((1, 1), (8, 3)):
        for b in (None, bias):
            check_route(logits, 8, bias=b, scores=scores, groups=groups, top_groups=top_groups)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_route_of_logits_from_a_product_just_launched(dtype):
    """The router's kernel starts under the product's end and must not read its output before."""
    g = gen(71)
    x, w = rand(g, 4096, 2048), rand(g, 128, 2048, std=2048 ** -0.5)
    want = None
    for _ in range(5):
        logits = sptg.gemm(x, w, out_dtype=F32 if dtype == F32 else BF16).to(dtype)
        got = sptg.route_experts(logits, 8)
        if want is None:
            torch.cuda.synchronize()
            want = sptg.route_experts(logits, 8)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------- rows to experts and back
@pytest.mark.parametrize("rows,top,e,kernel", [(256, 8, 64, "dispatch_small"), (512, 8, 64, "dispatch_small"),
                                               (513, 8, 64, "dispatch"), (257, 8, 64, "dispatch_small"),
                                               (4096, 1, 1024, "dispatch_small"), (4097, 1, 1024, "dispatch"),
                                               (70001, 3, 200, "dispatch"), (2048, 1, 1024, "dispatch_small"),
                                               (1, 2048, 33, "dispatch_small"), (1, 4096, 33, "dispatch_small"),
                                               (3, 5000, 7, "dispatch")])
def test_dispatch_by_each_of_its_kernels(rows, top, e, kernel):
    g = gen(rows + top)
    experts = torch.randint(-1, e + 1, (rows, top), device="cuda", generator=g, dtype=I32)
    for cols in (8, 3):
        x = rand(g, rows, cols)
        _, places, _ = check_dispatch(x, experts, e)
        assert f"kernel={kernel} " in sptg.last_config()
        flat = places.reshape(-1).long()
        assert torch.equal(torch.sort(flat).values, torch.arange(rows * top, device="cuda"))


@pytest.mark.parametrize("cols", [2048, 2047])
def test_rows_past_32_bits_of_elements(cols):
    """600000 rows of 8 places: sorted rows of some 9.8e9 elements, offsets past 2^32."""
    g = gen(72)
    rows, top, e = 600_000, 8, 64
    x = rand(g, rows, cols)
    experts = torch.randint(0, e, (rows, top), device="cuda", generator=g, dtype=I32)
    y, places, offsets = sptg.dispatch_rows(x, experts, e)
    assert y.numel() > 2 ** 32 and int(offsets[-1]) == rows * top
    some = torch.cat([torch.arange(50, device="cuda"), torch.randint(0, rows, (200,), device="cuda", generator=g),
                      torch.arange(rows - 50, rows, device="cuda")])
    for j in range(top):
        assert torch.equal(y[places[some, j].long()], x[some])
    weights = torch.rand(rows, top, device="cuda", generator=g)
    out = sptg.combine_rows(y, places, weights)
    want = x[some].double() * weights[some].double().sum(1, keepdim=True)
    # (eight products and additions of the same value)
    assert_within(out[some], want, 10 * UNIT * want.abs())
    del out
    dout = rand(g, rows, cols)
    dy, dweights = sptg.combine_rows_grad(dout, y, places, weights)
    for j in (0, top - 1):
        want = dout[some].double() * weights[some, j, None].double()
        assert_within(dy[places[some, j].long()], want, UNIT * want.abs())
    p = x[some].double() * dout[some].double()
    assert_within(dweights[some, 3], p.sum(1), (cols / 128 + 16) * UNIT * p.abs().sum(1))


# ---------------------------------------------------------- the end of a block
RING, SHIFTED, ANY = 2, 3, 4              # forward kernels, by last_config's kind (0 and 1: a row to a block)
GRAD_RING, GRAD_SHIFTED, GRAD_ANY = range(3)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("kind", ["none", "cols", "rows", "full"])
@pytest.mark.parametrize("rows,cols,forward,backward", [
    (8000, 1000, RING, GRAD_RING), (1900, 4096, RING, GRAD_RING), (2500, 2056, RING, GRAD_RING), (950, 8192, RING, GRAD_RING),
    (2000, 512, 0, GRAD_RING), (460, 16384, RING, GRAD_ANY), (1000, 8200, RING, GRAD_ANY), (900, 4097, SHIFTED, GRAD_SHIFTED),
    (1000, 777, SHIFTED, GRAD_SHIFTED), (310, 8191, SHIFTED, GRAD_SHIFTED), (40, 16375, SHIFTED, GRAD_ANY),
    (40, 16377, ANY, GRAD_ANY), (5, 16392, ANY, GRAD_ANY)])
def test_gate_norm_by_each_of_its_kernels(rows, cols, forward, backward, kind, dtype):
    g = gen(rows + cols)
    y, x = rand(g, rows, cols, dtype=dtype), rand(g, rows, cols, dtype=dtype, std=2.0)
    w2, gate = 1 + rand(g, cols, dtype=dtype, std=0.2), gate_of(g, kind, rows, cols, dtype)
    dh, dv = rand(g, rows, cols, dtype=dtype), rand(g, rows, cols, dtype=dtype)
    for w1 in (rand(g, cols, dtype=dtype), None):
        check_gate_norm(y, x, w2, w1, gate, dh=dh, dv=dv)
        assert chosen()["kind"] == forward
        sptg.gate_add_rms_norm_grad(dh, dv, y, x, w2, w1, gate)
        assert chosen()["kind"] == backward
    check_gate_norm(y, x, w2, w2, gate, dv=dv)
    check_gate_norm(y, x, w2, w2, gate, dh=dh)
    ref = gate_norm_reference(y, x, w2, None, gate, 0.75, 1e-5)
    h, v = sptg.gate_add_rms_norm(y, x, w2, gate=gate, alpha=0.75, eps=1e-5, h=x)  # in place
    assert_within(h, ref["h"][0], (cols / 128 + 128) * UNIT * ref["h"][1])
    assert_within(v, ref["v"][0], (cols / 128 + 128) * UNIT * ref["v"][1])


@pytest.mark.parametrize("kind", ["none", "cols", "rows", "full"])
@pytest.mark.parametrize("rows,cols,forward", [
    (3000, 4097, SHIFTED), (8000, 1001, SHIFTED), (2000, 5003, SHIFTED), (1000, 8189, SHIFTED), (480, 12289, SHIFTED),
    (470, 16377, ANY), (5000, 1, SHIFTED), (5000, 7, SHIFTED), (5000, 9, SHIFTED), (5000, 21, SHIFTED), (9000, 129, SHIFTED),
    (700, 8190, SHIFTED)])
def test_gate_norm_of_many_rows_off_16_byte_boundaries(rows, cols, forward, kind):
    g = gen(rows * 3 + cols)
    w2, gate = 1 + rand(g, cols, std=0.2), gate_of(g, kind, rows, cols, BF16)
    for pitches in ((0, 0, 0, 0), (3, 0, 6, 1)):  # all rows a shift alike; each operand with its own
        y, x, dh, dv = (rand(g, rows, cols + k + (k > 3))[:, k:cols + k] for k in pitches)
        for w1 in (rand(g, cols), None):
            check_gate_norm(y, x, w2, w1, gate, dh=dh, dv=dv)
            assert chosen()["kind"] == forward
            sptg.gate_add_rms_norm_grad(dh, dv, y, x, w2, w1, gate)
            assert chosen()["kind"] == (GRAD_SHIFTED if cols <= 8192 else GRAD_ANY)
        check_gate_norm(y, x, w2, w2, gate, dv=dv)
        wide = rand(g, rows, cols + 5)
        inside, ref = wide[:, 2:cols + 2], gate_norm_reference(y, wide[:, 2:cols + 2], w2, w2, gate, 0.75, 1e-5)
        before = wide.clone()
        h, v = sptg.gate_add_rms_norm(y, inside, w2, w2, gate, alpha=0.75, eps=1e-5, h=inside)  # in place
        assert_within(h, ref["h"][0], (cols / 128 + 128) * UNIT * ref["h"][1])
        assert_within(v, ref["v"][0], (cols / 128 + 128) * UNIT * ref["v"][1])
        assert torch.equal(wide[:, :2], before[:, :2]) and torch.equal(wide[:, cols + 2:], before[:, cols + 2:])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("kind", ["none", "cols", "rows", "full"])
@pytest.mark.parametrize("rows,cols,parts", [(1, 8200, 2), (2, 16384, 2), (300, 16384, 2), (3, 16392, 4), (160, 32768, 4),
                                             (5, 32776, 8), (40, 65536, 8), (3, 65544, 1), (3, 16385, 1)])
def test_gate_norm_gradients_of_rows_that_a_cluster_shares(rows, cols, parts, kind, dtype):
    g = gen(rows + cols)
    y, x = rand(g, rows, cols, dtype=dtype), rand(g, rows, cols, dtype=dtype, std=2.0)
    w2, gate = 1 + rand(g, cols, dtype=dtype, std=0.2), gate_of(g, kind, rows, cols, dtype)
    dh, dv = rand(g, rows, cols, dtype=dtype), rand(g, rows, cols, dtype=dtype)
    for w1 in (rand(g, cols, dtype=dtype), None):
        check_gate_norm(y, x, w2, w1, gate, dh=dh, dv=dv)
        check_gate_norm(y, x, w2, w1, gate, dv=dv, out_dtype=dtype)
        check_gate_norm(y, x, w2, w1, gate, dh=dh)
        first = sptg.gate_add_rms_norm_grad(dh, dv, y, x, w2, w1, gate)
        assert chosen()["kind"] == GRAD_ANY and chosen()["parts"] == parts
        again = sptg.gate_add_rms_norm_grad(dh, dv, y, x, w2, w1, gate)
        assert all(a is b or torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("rows,cols,kind", [(3000, 4097, GRAD_SHIFTED), (500, 16384, GRAD_ANY), (200, 40000, GRAD_ANY)])
def test_gate_norm_gradients_waits_that_run_out_are_reported(rows, cols, kind):
    g = gen(77)
    y, x, w = rand(g, rows, cols), rand(g, rows, cols), rand(g, cols)
    cfg = sptg.Config()
    cfg.timeout_ms, cfg.inject_stall = 100, 1
    sptg.gate_add_rms_norm_grad(y, x, y, x, w, w, config=cfg)
    assert chosen()["kind"] == kind
    assert sptg.device_error() == -5
    assert sptg.device_error() == 0
    check_gate_norm(y, x, w, w, None, dh=x, dv=y)


def test_gate_norm_waits_that_run_out_are_reported_and_the_context_survives():
    # each block's second row never arrives: its wait runs out after 100 ms, nothing is copied behind
    # it, and what was in flight lands before the block leaves
    g = gen(73)
    y, x, w = rand(g, 2500, 4096), rand(g, 2500, 4096), rand(g, 4096)
    cfg = sptg.Config()
    cfg.timeout_ms, cfg.inject_stall = 100, 1
    sptg.gate_add_rms_norm(y, x, w, w, config=cfg)
    assert chosen()["kind"] == RING
    assert sptg.device_error() == -5
    sptg.gate_add_rms_norm_grad(y, x, y, x, w, w, config=cfg)
    assert chosen()["kind"] == GRAD_RING
    assert sptg.device_error() == -5
    assert sptg.device_error() == 0  # the word was cleared
    check_gate_norm(y, x, w, w, None, dh=x, dv=y)


def test_gate_norm_past_32_bits_of_elements():
    g = gen(74)
    rows, cols = 1_100_000, 4096
    y, x, w = rand(g, rows, cols), rand(g, rows, cols), rand(g, cols)
    gate = rand(g, rows, 1)
    h, v = sptg.gate_add_rms_norm(y, x, w, w, gate)
    assert h.numel() > 2 ** 32
    for s in (slice(0, 40), slice(rows // 2, rows // 2 + 40), slice(rows - 40, rows)):
        ref = gate_norm_reference(y[s], x[s], w, w, gate[s], 1.0, 1e-6)
        assert_within(h[s], ref["h"][0], 160 * UNIT * ref["h"][1])
        assert_within(v[s], ref["v"][0], 160 * UNIT * ref["v"][1])
    del h, v
    dy, dx, dw2, dw1, dgate = sptg.gate_add_rms_norm_grad(x, y, y, x, w, w, gate, out_dtype=F32)
    for s in (slice(0, 40), slice(rows - 40, rows)):
        ref = gate_norm_reference(y[s], x[s], w, w, gate[s], 1.0, 1e-6, x[s], y[s])
        assert_within(dy[s], ref["y"][0], 160 * UNIT * ref["y"][1])
        assert_within(dx[s], ref["residual"][0], 160 * UNIT * ref["residual"][1])
        assert_within(dgate[s], ref["gate"][0], 230 * UNIT * ref["gate"][1])
    assert torch.isfinite(dw1).all() and torch.isfinite(dw2).all()


# ----------------------------------------------------------- all together
def layer_weights(g, hidden=256, inner=192, experts=16):
    return {"router": rand(g, experts, hidden, std=hidden ** -0.5), "up": rand(g, experts, inner, hidden, std=hidden ** -0.5),
            "down": rand(g, experts, hidden, inner, std=inner ** -0.5), "post": rand(g, hidden, std=0.3),
            "next": 1 + rand(g, hidden, std=0.1), "gate": rand(g, hidden, std=0.5),
            "bias": rand(g, experts, dtype=F32, std=0.02)}


def layer(w, x, residual, logits, stream=None):
    """An expert layer's forward half with the block's end; all calls on one stream."""
    kw = {} if stream is None else dict(stream=stream)
    experts = w["up"].shape[0]
    weights, ids = sptg.route_experts(logits, 4, bias=w["bias"], scores="sigmoid", groups=4, top_groups=2, scale=1.5, **kw)
    rows, places, offsets = sptg.dispatch_rows(x, ids, experts, **kw)
    u = sptg.grouped_gemm(rows, w["up"], offsets, **kw)
    d = sptg.grouped_gemm(u, w["down"], offsets, **kw)
    out = sptg.combine_rows(d, places, weights, base=x, **kw)
    h, v = sptg.gate_add_rms_norm(out, residual, w["next"], block_weight=w["post"], gate=w["gate"], alpha=0.5, **kw)
    return h, v, ids, weights


def layer_inputs(g, rows=300, hidden=256, experts=16):
    return rand(g, rows, hidden), rand(g, rows, hidden), rand(g, rows, experts, dtype=F32)


def plain_layer(w, x, residual, logits, ids):
    """The same in 64 bits, with the given choice of experts."""
    s = torch.sigmoid(logits)
    c = torch.gather(s, 1, ids.long())
    weights = 1.5 * c / c.sum(1, keepdim=True)
    out = x
    for j in range(ids.shape[1]):
        e = ids[:, j].long()
        u = torch.einsum("th,tih->ti", x, w["up"][e])
        out = out + weights[:, j, None] * torch.einsum("ti,thi->th", u, w["down"][e])
    n = out * torch.rsqrt(out.square().mean(1, keepdim=True) + 1e-6) * w["post"]
    h = 0.5 * residual + w["gate"] * n
    return h, h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * w["next"]


@pytest.mark.parametrize("rows", [1, 37, 300])
def test_a_layer_and_its_gradients_against_64_bits(rows):
    """Five bfloat16 roundings lie between inputs and outputs, and as many again on the way back: 3 % of a norm."""
    g = gen(80 + rows)
    w = layer_weights(g)
    x, residual, logits = layer_inputs(g, rows)
    names = ["up", "down", "post", "next", "gate"]
    leaves = [t.clone().requires_grad_() for t in (x, residual, logits)]
    params = {k: (v.clone().requires_grad_() if k in names else v) for k, v in w.items()}
    h, v, ids, _ = layer(params, *leaves)
    dh, dv = rand(g, *h.shape), rand(g, *h.shape)
    grads = torch.autograd.grad((h, v), leaves + [params[k] for k in names], (dh, dv))
    exact = [t.detach().double().requires_grad_() for t in leaves]
    wide = {k: (v.detach().double().requires_grad_() if k in names else v.double()) for k, v in params.items()}
    ref = plain_layer(wide, *exact, ids)
    ref_grads = torch.autograd.grad(ref, exact + [wide[k] for k in names], (dh.double(), dv.double()))
    for got, want in zip((h, v) + grads, ref + ref_grads):
        assert got.shape == want.shape
        assert float((got.detach().double() - want.detach()).norm() / want.detach().norm()) < 0.03


def test_a_layer_on_streams_and_threads_of_its_own_gives_the_same_bits():
    g = gen(90)
    w, inputs = layer_weights(g), layer_inputs(g)
    want = layer(w, *inputs)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        side.wait_stream(torch.cuda.current_stream())
        got = layer(w, *inputs, stream=stream)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    results = {}

    def work(t):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                results[t] = [layer(w, *inputs) for _ in range(10)]
            stream.synchronize()
        except Exception as e:  # reported below, on the main thread
            results[t] = e

    threads = [threading.Thread(target=work, args=(t,)) for t in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for t in range(4):
        assert not isinstance(results[t], Exception), results[t]
        for got in results[t]:
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_tensors_dropped_after_a_layer_on_another_stream():
    """The stream is still busy with something else when the inputs are dropped and their memory is asked for."""
    g = gen(91)
    w, inputs = layer_weights(g), layer_inputs(g, 4000)
    want = layer(w, *inputs)
    side = torch.cuda.Stream()
    copies = [t.clone() for t in inputs]
    sizes = [t.numel() * t.element_size() for t in inputs]
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)  # some 20 ms
    got = layer(w, *copies, stream=side)
    del copies
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del junk


@pytest.mark.parametrize("rows", [1, 700])
def test_a_layer_and_its_gradients_in_graphs(rows):
    """Two graphs captured from one pool, replayed in turn on new inputs.  (No other graph of the same leaves is alive
    meanwhile: PyTorch would let the stream of its nodes join the capture.)"""
    g = gen(92)
    w = layer_weights(g)
    sets = [layer_inputs(g, rows) for _ in range(3)]
    names = ["up", "down", "post", "next", "gate"]
    params = {k: (v.clone().requires_grad_() if k in names else v) for k, v in w.items()}

    def step(x, residual, logits):
        leaves = [t.detach().requires_grad_() for t in (x, residual, logits)]
        h, v, ids, weights = layer(params, *leaves)
        grads = torch.autograd.grad((h, v), leaves + [params[k] for k in names], (residual, x))
        return (h.detach(), v.detach(), ids, weights.detach()) + grads

    want = [step(*s) for s in sets]
    static = [t.clone() for t in sets[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*static)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs, pool = [], [], None
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            outs.append(step(*static))
        pool = graph.pool()
        graphs.append(graph)
    for i in (1, 2, 0, 2):
        for a, b in zip(static, sets[i]):
            a.copy_(b)
        for graph, out in zip(graphs, outs):
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))


def test_the_same_bits_on_every_call():
    g = gen(93)
    rows, cols = 3000, 1024
    logits, bias = rand(g, rows, 256, dtype=F32), rand(g, 256, dtype=F32, std=0.05)
    weights, ids = sptg.route_experts(logits, 8, bias=bias, scores="sigmoid", groups=8, top_groups=4)
    x, dout, w = rand(g, rows, cols), rand(g, rows, cols), rand(g, cols)
    y, places, _ = sptg.dispatch_rows(x, ids, 256)

    def calls():
        yield from sptg.route_experts(logits, 8, bias=bias, scores="sigmoid", groups=8, top_groups=4)
        yield sptg.route_experts_dlogits(weights, logits, ids, scores="sigmoid")
        yield from sptg.dispatch_rows(x, ids, 256)
        yield sptg.combine_rows(y, places, weights)
        yield from sptg.combine_rows_grad(dout, y, places, weights)
        yield from sptg.gate_add_rms_norm(x, dout, w, w, w)
        yield from sptg.gate_add_rms_norm_grad(dout, x, x, dout, w, w, w, out_dtype=F32)

    first = list(calls())
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(calls(), first))


# ------------------------------------------------------ automatic differentiation
def test_gradients_of_some_inputs_and_odd_gradients():
    g = gen(94)
    w, (x, residual, logits) = layer_weights(g), layer_inputs(g, 50)
    # some inputs only, one of the two outputs only
    for which in range(5):
        tensors = [x, residual, w["next"], w["post"], w["gate"]]
        leaf = tensors[which] = tensors[which].clone().requires_grad_()
        h, v = sptg.gate_add_rms_norm(*tensors)
        want = sptg.gate_add_rms_norm_grad(residual, None, *[t.detach() for t in tensors])[which]
        if which != 2:
            assert torch.equal(torch.autograd.grad(h, leaf, residual, retain_graph=True)[0], want)
        want = sptg.gate_add_rms_norm_grad(residual, x, *[t.detach() for t in tensors])[which]
        # a gradient of a type and strides that the kernels do not take
        odd = torch.stack([x.float(), x.float()], 2)[:, :, 0]
        assert torch.equal(torch.autograd.grad((h, v), leaf, (residual, odd.to(BF16)))[0], want)
    leaf = logits.clone().requires_grad_()
    weights, ids = sptg.route_experts(leaf, 4)
    ones = torch.ones(1, device="cuda").expand(50, 4)
    assert float(torch.autograd.grad(weights, leaf, ones, retain_graph=True)[0].abs().max()) < 1e-6  # they sum to 1
    with pytest.raises(ValueError):
        sptg.route_experts(leaf, 4, weights=torch.empty(50, 4, device="cuda"))
    with pytest.raises(ValueError):
        sptg.dispatch_rows(x.clone().requires_grad_(), ids, 16, out=torch.empty(200, 256, dtype=BF16, device="cuda"))
    with torch.no_grad():
        assert not sptg.route_experts(leaf, 4)[0].requires_grad
    grad, = torch.autograd.grad(weights, leaf, ones, create_graph=True)
    with pytest.raises(RuntimeError):  # the gradient has no derivative of its own
        grad.sum().backward()


@pytest.mark.parametrize("rows,cols", [(700, 4097), (200, 16384)])
def test_gradients_of_cut_and_of_shared_rows_in_a_graph(rows, cols):
    """Captured, replayed with new inputs, and beside the same call on another stream."""
    g = gen(96)
    w = rand(g, cols)
    y, x, dh, dv = (rand(g, rows, cols) for _ in range(4))
    places = torch.randperm(2 * rows, device="cuda", generator=g).to(I32).reshape(rows, 2)
    weights, sorted_rows = torch.rand(rows, 2, device="cuda", generator=g), rand(g, 2 * rows, cols)

    def calls(**kw):
        return (*sptg.gate_add_rms_norm_grad(dh, dv, y, x, w, w, w, out_dtype=F32, **kw),
                *sptg.combine_rows_grad(dh, sorted_rows, places, weights, **kw))

    calls()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = calls()
    side = torch.cuda.Stream()
    for _ in range(2):
        for t in (y, x, dh, dv):
            t.copy_(rand(g, rows, cols))
        torch.cuda.synchronize()
        graph.replay()
        beside = calls(stream=side)
        torch.cuda.synchronize()
        want = calls()
        assert all(torch.equal(a, b) and torch.equal(c, b) for a, b, c in zip(out, want, beside))


def test_rows_without_a_place_get_no_gradient():
    g = gen(95)
    places = torch.randperm(40, device="cuda", generator=g)[:24].to(I32).reshape(8, 3)
    weights = torch.rand(8, 3, device="cuda", generator=g)
    for cols in (64, 65):
        y, dout = rand(g, 40, cols), rand(g, 8, cols)
        torch.full_like(y, 3.0)  # (what the allocator hands out next)
        leaf = y.clone().requires_grad_()
        dy, = torch.autograd.grad(sptg.combine_rows(leaf, places, weights), leaf, dout)
        want = torch.zeros(40, cols, dtype=torch.float64, device="cuda")
        want[places.flatten().long()] = (weights[:, :, None].double() * dout[:, None].double()).reshape(24, cols)
        assert_within(dy, want, UNIT * want.abs())
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        on_side = sptg.combine_rows_grad(dout, y, places, weights, stream=side)[0]
        side.synchronize()
        assert torch.equal(on_side, dy)


def test_python_refusals_on_the_gpu():
    x, ids = torch.zeros(4, 16, dtype=BF16, device="cuda"), torch.zeros(4, 2, dtype=I32, device="cuda")
    w = x[0].clone()
    for bad in (lambda: sptg.route_experts(x.double(), 2), lambda: sptg.route_experts(x, 2, scores="tanh"),
                lambda: sptg.route_experts(x.t(), 2), lambda: sptg.route_experts(x[:1].expand(4, 16), 2),
                lambda: sptg.route_experts(x, 2, bias=w), lambda: sptg.route_experts(x, 2, bias=torch.zeros(16)),
                lambda: sptg.route_experts_dlogits(x, x, ids), lambda: sptg.dispatch_rows(x.float(), ids, 4),
                lambda: sptg.dispatch_rows(x, ids.long(), 4), lambda: sptg.dispatch_rows(x, ids[:3], 4),
                lambda: sptg.dispatch_rows(x, ids[0], 4), lambda: sptg.combine_rows(x, ids.long()),
                lambda: sptg.combine_rows(x, ids, torch.zeros(4, 2, dtype=BF16, device="cuda")),
                lambda: sptg.combine_rows(x, ids, base=x[:3]), lambda: sptg.combine_rows_grad(x, x, ids, dweights=w),
                lambda: sptg.gate_add_rms_norm(x, x, x), lambda: sptg.gate_add_rms_norm(x, x.half(), w),
                lambda: sptg.gate_add_rms_norm(x, x, w, gate=w[:5]), lambda: sptg.gate_add_rms_norm(x, x, w, gate=x[:3]),
                lambda: sptg.gate_add_rms_norm(x, x, w, gate=x[:, :1].float()),
                lambda: sptg.gate_add_rms_norm(x, x, w, gate=w.expand(4, 16)),
                lambda: sptg.gate_add_rms_norm_grad(x, x, x, x, w, out_dtype=torch.float16)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: sptg.route_experts(x, 17), lambda: sptg.route_experts(x, 2, groups=3),
                lambda: sptg.route_experts(x, 9, groups=2, top_groups=1), lambda: sptg.route_experts(x, 0),
                lambda: sptg.dispatch_rows(x, ids, 1025), lambda: sptg.gate_add_rms_norm(x, x, w, eps=0.0),
                lambda: sptg.gate_add_rms_norm(x, x, w, alpha=INF)):
        with pytest.raises(sptg.SptgError):
            bad()
