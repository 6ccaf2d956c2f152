"""Gradients of the operators around an expert layer in calls that a training run may make: entries that were dropped,
a configuration, tangents, one row, and a million rows."""
import pytest
import torch
import torch.autograd.forward_ad as forward_ad

import software_pipelined_tiled_gb300 as sptg
from test_expert_layer_gpu import BF16, F16, F32, I32, NAN, UNIT, assert_within, gate_norm_reference, gen, rand
from test_layer_ops_edges_gpu import chosen

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    torch.cuda.synchronize()
    assert sptg.device_error() == 0


# ------------------------------------------------------- entries that were dropped
def dropped_places(g, rows, top, share, y_rows=None):
    """A permutation's first places, some of them outside of y's rows."""
    y_rows = rows * top if y_rows is None else y_rows
    places = torch.randperm(max(y_rows, rows * top), device="cuda", generator=g)[:rows * top].to(I32).reshape(rows, top)
    outside = torch.tensor([-1, -(1 << 31), y_rows, (1 << 31) - 1], dtype=torch.int64, device="cuda").to(I32)
    some = outside[torch.randint(0, 4, (rows, top), device="cuda", generator=g)]
    return torch.where(torch.rand(rows, top, device="cuda", generator=g) < share, some, places)


def dy_reference(dout, places, weights, y_rows):
    """(One product of 32 bits a value; rows without a place are 0.)"""
    want = torch.zeros(y_rows, dout.shape[1], dtype=torch.float64, device="cuda")
    t, j = ((places >= 0) & (places < y_rows)).nonzero(as_tuple=True)
    w = 1.0 if weights is None else weights[t, j, None].double()
    want[places[t, j].long()] = dout[t].double() * w
    return want


def poison(*likes):
    """What the allocator hands out next for tensors like these."""
    for t in [torch.full_like(x, NAN) for x in likes]:
        del t


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rows,top,cols", [(1, 1, 8), (8, 3, 64), (8, 3, 65), (40, 2, 1024), (531, 6, 2056), (333, 1, 1031),
                                           (1500, 8, 1025), (2600, 7, 1152), (9000, 2, 520), (20011, 3, 16)])
@pytest.mark.parametrize("share", [0.0, 0.05, 0.6, 1.0])
def test_rows_of_dropped_entries_get_no_gradient(share, rows, top, cols, dtype):
    g = gen(rows + top)
    y, dout = rand(g, rows * top, cols, dtype=dtype), rand(g, rows, cols, dtype=dtype)
    places = dropped_places(g, rows, top, share)
    for weights in (torch.rand(rows, top, device="cuda", generator=g), None):
        want = dy_reference(dout, places, weights, rows * top)
        leaf = y.clone().requires_grad_()
        out = sptg.combine_rows(leaf, places, weights)
        poison(y)
        dy, = torch.autograd.grad(out, leaf, dout)
        assert_within(dy, want, UNIT * want.abs())
        poison(y)
        dy, dweights = sptg.combine_rows_grad(dout, y, places, weights)
        assert_within(dy, want, UNIT * want.abs())
        if weights is not None:
            assert not dweights[(places < 0) | (places >= rows * top)].any()
            poison(y)
            assert torch.equal(sptg.combine_rows_grad(dout, y, places, weights, need_weights=False)[0], dy)
        given = torch.full_like(y, 7.0)  # a given dy's rows without a place are left as they were
        sptg.combine_rows_grad(dout, y, places, weights, dy=given)
        named = torch.zeros(rows * top, dtype=torch.bool, device="cuda")
        named[places[(places >= 0) & (places < rows * top)].long()] = True
        assert (given[~named] == 7.0).all() and torch.equal(given[named], dy[named])


@pytest.mark.parametrize("y_rows", [5000, 7000, 90000])
@pytest.mark.parametrize("cols", [1024, 2049, 24])
def test_rows_without_a_place_beside_dropped_entries(cols, y_rows):
    g = gen(cols + y_rows)
    places = dropped_places(g, 1500, 4, 0.1, y_rows)
    y, dout = rand(g, y_rows, cols), rand(g, 1500, cols)
    weights = torch.rand(1500, 4, device="cuda", generator=g)
    poison(y)
    dy, _ = sptg.combine_rows_grad(dout, y, places, weights)
    want = dy_reference(dout, places, weights, y_rows)
    assert_within(dy, want, UNIT * want.abs())
    poison(y[:300])
    none, _ = sptg.combine_rows_grad(dout[:0], y[:300], places[:0], weights[:0])  # no rows at all
    assert none.shape == (300, cols) and not none.any()


@pytest.mark.parametrize("rows,cols", [(600, 1024), (600, 1027), (600, 80), (600, 81)])
def test_dropped_entries_in_a_graph_and_on_another_stream(rows, cols):
    g = gen(21)
    y, dout, weights = rand(g, rows * 4, cols), rand(g, rows, cols), torch.rand(rows, 4, device="cuda", generator=g)
    places = dropped_places(g, rows, 4, 0.2)

    def calls(**kw):
        return sptg.combine_rows_grad(dout, y, places, weights, **kw)

    calls()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = calls()
    side = torch.cuda.Stream()
    for seed in range(3):
        places.copy_(dropped_places(gen(seed), rows, 4, 0.3 * seed))
        out[0].fill_(NAN)
        torch.cuda.synchronize()
        graph.replay()
        beside = calls(stream=side)
        torch.cuda.synchronize()
        want = dy_reference(dout, places, weights, rows * 4)
        assert_within(out[0], want, UNIT * want.abs())
        assert torch.equal(beside[0], out[0]) and torch.equal(beside[1], out[1])


@pytest.mark.parametrize("off,cols", [(0, 1024), (8, 96), (3, 1024), (0, 97)])
def test_zeros_in_a_gradient_of_strided_rows(off, cols):
    """By the C entry, which takes dy: rows without a place get zeros, what lies beside the rows is left as it was."""
    g = gen(22)
    rows, top = 300, 4
    wide = torch.full((rows * top, 1100), 7.0, dtype=BF16, device="cuda")
    y, dout = rand(g, rows * top, cols), rand(g, rows, cols)
    weights, places = torch.rand(rows, top, device="cuda", generator=g), dropped_places(g, rows, top, 0.3)
    want = dy_reference(dout, places, weights, rows * top)
    dy = wide[:, off:off + cols]
    rc = sptg.load().sptg_combine_rows_grad_ex(
        rows, cols, top, rows * top, 1, dout.data_ptr(), cols, y.data_ptr(), cols, places.data_ptr(), weights.data_ptr(),
        dy.data_ptr(), 1100, None, 1, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert_within(dy, want, UNIT * want.abs())
    assert (wide[:, :off] == 7.0).all() and (wide[:, off + cols:] == 7.0).all()


@pytest.mark.parametrize("rows,top,cols", [(1, 1, 8), (1, 3, 1024), (700, 3, 1024), (701, 3, 1031), (2051, 1, 512)])
@pytest.mark.parametrize("at", [1, 2, 3])
def test_dropped_entries_of_places_at_any_address(at, rows, top, cols):
    g = gen(23 + rows)
    y, dout = rand(g, rows * top, cols), rand(g, rows, cols)
    places = torch.zeros(rows * top + 8, dtype=I32, device="cuda")[at:at + rows * top].view(rows, top)
    places.copy_(dropped_places(g, rows, top, 0.2))
    want = dy_reference(dout, places, None, rows * top)
    poison(y)
    assert_within(sptg.combine_rows_grad(dout, y, places)[0], want, UNIT * want.abs())


# ------------------------------------------------------- a configuration
def test_a_configuration_holds_where_gradients_are_asked_for():
    g = gen(31)
    y, x, w = rand(g, 2500, 4096), rand(g, 2500, 4096), rand(g, 4096)
    leaf = y.clone().requires_grad_()
    bad = sptg.Config()
    bad.timeout_ms = -1
    with pytest.raises(sptg.SptgError):
        sptg.gate_add_rms_norm(leaf, x, w, w, config=bad)
    # (as in test_expert_layer_edges_gpu: each block's second row never arrives, and the waits for it run out)
    cfg = sptg.Config()
    cfg.timeout_ms, cfg.inject_stall = 100, 1
    h, v = sptg.gate_add_rms_norm(leaf, x, w, w, config=cfg)
    assert chosen()["kind"] == 2 and sptg.device_error() == -5
    cfg.inject_stall = 0  # the backward call has what the forward call was given
    torch.autograd.grad((h, v), leaf, (x, y))
    assert sptg.device_error() == -5  # (reported by a thread of automatic differentiation's, to the same word)
    fine = sptg.Config()
    fine.timeout_ms = 1000
    got = torch.autograd.grad(sptg.gate_add_rms_norm(leaf, x, w, w, config=fine), leaf, (x, y))[0]
    assert torch.equal(got, sptg.gate_add_rms_norm_grad(x, y, y, x, w, w)[0])


# ------------------------------------------------------- forward mode
def test_tangents_are_refused_not_dropped():
    g = gen(41)
    x, residual, w, gate = rand(g, 8, 16), rand(g, 8, 16), rand(g, 16), rand(g, 8, 1)
    logits, weights = rand(g, 8, 4, dtype=F32), torch.rand(8, 2, device="cuda", generator=g)
    _, ids = sptg.route_experts(logits, 2)
    y, places, offsets = sptg.dispatch_rows(x, ids, 4)
    W = rand(g, 4, 24, 16)
    calls = ((lambda l: sptg.route_experts(l, 2), (logits,)), (lambda x: sptg.dispatch_rows(x, ids, 4), (x,)),
             (lambda y, w, b: sptg.combine_rows(y, places, w, base=b), (y, weights, x)),
             (lambda *t: sptg.gate_add_rms_norm(*t), (x, residual, w, w, gate)),
             (lambda X, W: sptg.grouped_gemm(X, W, offsets), (y, W)))
    for call, tensors in calls:
        plain = call(*tensors)
        for i, t in enumerate(tensors):
            with forward_ad.dual_level():
                dual = forward_ad.make_dual(t, torch.ones_like(t))
                mixed = tensors[:i] + (dual,) + tensors[i + 1:]
                with pytest.raises(NotImplementedError):
                    call(*mixed)
                with torch.no_grad(), pytest.raises(NotImplementedError):
                    call(*mixed)
                again = call(*tensors)  # tensors without tangents pass
        for a, b in zip(again if isinstance(again, tuple) else (again,), plain if isinstance(plain, tuple) else (plain,)):
            assert torch.equal(a, b)


# ------------------------------------------------------- types
def test_type_of_a_column_gates_gradient():
    """Of C values: out_dtype for any number of rows.  1 x C with one row is the gate with a value an element."""
    g = gen(51)
    w = rand(g, 64)
    for rows in (1, 2):
        y, x = rand(g, rows, 64), rand(g, rows, 64)
        grads = sptg.gate_add_rms_norm_grad(x, y, y, x, w, w, w, out_dtype=F32)
        assert grads[4].dtype == F32 and grads[4].shape == (64,)
        wide = sptg.gate_add_rms_norm_grad(x, y, y, x, w, w, w[None], out_dtype=F32)[4]
        assert wide.shape == (1, 64) and wide.dtype == (BF16 if rows == 1 else F32)
        assert torch.equal(wide[0].to(BF16), grads[4].to(BF16))


def test_gate_norm_sums_past_32_bits_of_elements():
    """1.1 million rows: the sums over all of them against 64 bits, chunk by chunk.  Nothing cancels (inputs are positive) and
    gradients grow with the row, so that rows left out, taken twice or taken for others would show.  The bound counts an
    addition in 32 bits for each row of a block (at least 152 blocks) and for each block, and check_gate_norm's roundings
    of a term: 1e-3 of the sum of magnitudes."""
    g = gen(52)
    rows, cols = 1_100_000, 4096
    y, x, dh, dv = (rand(g, rows, cols).abs_() for _ in range(4))
    w2, w1, gate = (rand(g, cols).abs_() for _ in range(3))
    by_row = (1 + torch.arange(rows, device="cuda") * 8 // rows).to(BF16)[:, None]
    dh.mul_(by_row)
    dv.mul_(by_row)
    grads = sptg.gate_add_rms_norm_grad(dh, dv, y, x, w2, w1, gate, out_dtype=F32)[2:]
    assert y.numel() > 2 ** 32
    names = ("weight", "block_weight", "gate")
    sums = {k: [torch.zeros(cols, dtype=torch.float64, device="cuda") for _ in range(2)] for k in names}
    for at in range(0, rows, 20000):
        s = slice(at, min(rows, at + 20000))
        ref = gate_norm_reference(y[s], x[s], w2, w1, gate, 1.0, 1e-6, dh[s], dv[s])
        for k in names:
            for total, part in zip(sums[k], ref[k]):
                total += part
        del ref
    for k, got in zip(names, grads):
        want, mag = sums[k]
        assert want.abs().sum() > 0.2 * mag.sum()
        assert_within(got, want, (cols / 128 + 128 + rows / 152 + 456) * UNIT * mag)
