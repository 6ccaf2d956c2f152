"""The operators around an expert layer against plain implementations in 64 bits.

Bounds, derived before the first run (u: unit roundoff of the output type, 2^-8
for bfloat16, 2^-11 for binary16, 0 for float32; one unit of 32 bits: 2^-23):

* experts, places, offsets, dispatched rows: equal.
* weights: exponentials, logarithms and divisions of up to 2 units each, the
  sum over the experts (at most 64 additions in a row), and the rounding of a
  logit's distance d from the largest, which the exponential turns into a
  relative error of d / 2 units: (64 + d) units of the weight.
* logits' gradients: the same relative error of each product in it, so
  (64 + d) units of s (|g| + sum |g| s), and the output's rounding.
* sums of rows: one rounding for each product and addition, (top + 2) units of
  the sum of magnitudes; the weights' gradients: columns / 128 additions in a row,
  16 more between threads, so (columns / 128 + 16) units of the magnitudes.
* norms: up to three sums follow one another, each with at most columns / 512 + 48
  additions in a row, and a dozen roundings an element: (columns / 128 + 128)
  units of the formula evaluated with the magnitudes of all its terms, and the
  output's rounding; for sums over rows as many units more as rows are added up
  in a row (rows / 128 + 64).
"""
import pytest
import torch

import software_pipelined_tiled_gb300 as sptg

pytestmark = pytest.mark.gpu

BF16, F16, F32, I32 = torch.bfloat16, torch.float16, torch.float32, torch.int32
U = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 0.0}
TINY = {BF16: 2.0 ** -133, F16: 2.0 ** -25, F32: 2.0 ** -126}  # (around zero)
UNIT = 2.0 ** -23
INF, NAN = float("inf"), float("nan")


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    torch.cuda.synchronize()
    assert sptg.device_error() == 0


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def rand(g, *shape, dtype=BF16, std=1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * std).to(dtype)


def assert_within(got, ref, error):
    """got within `error` of ref before its rounding."""
    u, tiny = U[got.dtype], TINY[got.dtype]
    off = (got.double() - ref).abs()
    bound = error + u * (ref.abs() + error) + tiny
    assert got.shape == ref.shape
    assert (off <= bound).all(), f"max error / bound {float((off / bound).max()):.3f}"


# ------------------------------------------------------------------- routing
def route_reference(logits, top, bias=None, scores="softmax", groups=1, top_groups=1, group_best=2,
                    renormalize=True, scale=1.0):
    """Scores, the experts and their weights; picks one by one, -infinity never."""
    z = logits.double()
    t, e = z.shape
    if scores == "sigmoid":
        s = 1 / (1 + torch.exp(-z))
    else:
        s = torch.exp(z - z.amax(1, keepdim=True).clamp(min=-1e300))
        s = s / s.sum(1, keepdim=True).clamp(min=1e-300)
    plain = bias is None or not bias.any()
    key = s + bias.double() if bias is not None else s
    if plain and (groups == 1 or group_best == 1):
        key = z
    key = torch.where(z == -INF, z, key)
    if bias is not None:
        key = torch.where(bias.double()[None, :] == -INF, torch.full_like(key, -INF), key)
    if groups > 1:
        m = key.reshape(t, groups, -1)
        b = m.sort(dim=2, descending=True).values[:, :, :group_best]
        b = torch.where((b == -INF) & (torch.arange(b.shape[2], device=b.device) > 0), torch.zeros_like(b), b).sum(2)
        rank = ((b[:, None, :] > b[:, :, None])
                | ((b[:, None, :] == b[:, :, None])
                   & (torch.arange(groups, device=b.device)[None, None, :] < torch.arange(groups, device=b.device)[None, :, None]))
                ).sum(2)
        key = torch.where((rank < top_groups)[:, :, None], m, torch.full_like(m, -INF)).reshape(t, e)
    order = torch.sort(key, dim=1, descending=True, stable=True)
    experts, dead = order.indices[:, :top].clone(), order.values[:, :top] == -INF
    w = torch.gather(s, 1, experts).masked_fill(dead, 0.0)
    if renormalize and scores == "sigmoid":  # (in logarithms: scores may all be tiny)
        zl = torch.gather(z, 1, experts)
        w = torch.softmax(torch.nn.functional.logsigmoid(zl).masked_fill(dead, -INF), 1).nan_to_num(0.0)
    elif renormalize:
        w = torch.softmax(torch.gather(z, 1, experts).masked_fill(dead, -INF), 1).nan_to_num(0.0)
    return s, w * scale, torch.where(dead, torch.full_like(experts, -1), experts).to(I32)


def distance(logits):
    """The largest distance of a finite logit of a row from the row's largest."""
    z = logits.double()
    least = torch.where(z == -INF, torch.full_like(z, INF), z).amin(1, keepdim=True)
    return (z.amax(1, keepdim=True) - least).clamp(min=0.0).nan_to_num(0.0)


def check_route(logits, top, stream=None, **how):
    _, w, experts = route_reference(logits, top, **how)
    weights, chosen = sptg.route_experts(logits, top, **how)
    assert weights.dtype == F32 and chosen.dtype == I32
    assert torch.equal(chosen, experts)
    assert_within(weights, w, (64 + distance(logits)) * UNIT * w)
    return weights, chosen


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("scores,biased,renormalize", [("softmax", False, True), ("softmax", True, False),
                                                       ("sigmoid", True, True), ("sigmoid", False, False)])
@pytest.mark.parametrize("rows,e,top,groups,top_groups,group_best", [
    (1, 1, 1, 1, 1, 2), (1, 64, 8, 1, 1, 2), (7, 8, 2, 1, 1, 1), (33, 60, 4, 1, 1, 2), (5, 61, 7, 1, 1, 2),
    (257, 128, 8, 1, 1, 2), (100, 160, 6, 8, 3, 2), (64, 256, 8, 8, 4, 2), (31, 256, 16, 32, 5, 1),
    (12, 384, 8, 1, 1, 2), (9, 512, 10, 8, 2, 1), (3, 1024, 16, 16, 8, 2), (6, 999, 3, 3, 2, 2),
    (4, 32, 4, 32, 4, 2), (2, 9, 9, 3, 3, 2), (1000, 40, 8, 5, 2, 1)])
def test_route(rows, e, top, groups, top_groups, group_best, scores, biased, renormalize, dtype):
    g = gen(rows + 31 * e + top)
    logits = rand(g, rows, e, dtype=dtype, std=1.5)
    bias = rand(g, e, dtype=F32, std=0.05) if biased else None
    check_route(logits, top, bias=bias, scores=scores, groups=groups, top_groups=top_groups,
                group_best=group_best, renormalize=renormalize, scale=2.5 if biased else 1.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top_groups,group_best", [(1, 1, 2), (8, 4, 2), (8, 3, 1)])
@pytest.mark.parametrize("kind", ["zero bias", "steps", "equal rows", "neighbours", "zeros"])
def test_route_decides_ties_and_close_calls_as_exact_arithmetic_does(kind, groups, top_groups, group_best,
                                                                     scores, dtype):
    g = gen(5)
    logits = rand(g, 2000, 128, dtype=dtype)
    if kind == "zero bias":
        bias = torch.zeros(128, device="cuda")
    elif kind == "steps":  # as a balance of loads moves them
        bias = torch.randint(-3, 4, (128,), device="cuda", generator=g).float() * 0.001
    elif kind == "equal rows":
        logits = logits[:, :1].expand(2000, 128).contiguous()
        bias = torch.randint(0, 2, (128,), device="cuda", generator=g).float() * 0.01
    elif kind == "zeros":  # rows of padding
        logits[::3] = 0
        bias = torch.randint(-1, 2, (128,), device="cuda", generator=g).float() * 0.001
    else:  # logits that lie closer than the roundings of their scores
        logits = (1.0 + torch.randint(0, 40, (2000, 128), device="cuda", generator=g) * 2.0 ** -22).to(dtype)
        bias = torch.randint(0, 3, (128,), device="cuda", generator=g).float() * 2.0 ** -24
    check_route(logits, 8, bias=bias, scores=scores, groups=groups, top_groups=top_groups, group_best=group_best)
    check_route(logits, 8, scores=scores, groups=groups, top_groups=top_groups, group_best=group_best)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (8, 4)])
def test_route_of_masked_experts(groups, top_groups, biased, renormalize, scores):
    g = gen(6)
    e = 64
    logits = rand(g, 40, e, dtype=F32)
    logits[:20] = torch.where(torch.rand(20, e, device="cuda", generator=g) < 0.9, torch.full_like(logits[:20], -INF),
                              logits[:20])
    logits[20] = -INF
    logits[21, 1:] = -INF
    logits[22] = torch.finfo(F32).min  # the lowest value is a value
    logits[23, :60] = torch.finfo(F32).min
    logits[24] = -120.0 - torch.arange(e, device="cuda") * 0.5  # scores that 32 bits hold no more
    bias = rand(g, e, dtype=F32, std=0.05) if biased else None
    how = dict(bias=bias, scores=scores, groups=groups, top_groups=top_groups, renormalize=renormalize)
    if biased:
        bias[3], bias[40:44] = -INF, -INF
    rows = torch.arange(40, device="cuda")
    if not biased and groups > 1:  # (sums of scores that are all zero in 64 bits too are ties there only)
        rows = rows[(rows != 23) & (rows != 22)]
    weights, chosen = check_route(logits[rows].contiguous(), 8, **how)
    assert (chosen[20] == -1).all() and not weights[20].any()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_route_of_infinities_and_nan(scores, dtype):
    g = gen(7)
    logits = rand(g, 8, 200, dtype=dtype)
    logits[1, 7], logits[2, 199], logits[4, 5] = NAN, NAN, INF
    for bias in (None, rand(g, 200, dtype=F32, std=0.01)):
        weights, chosen = sptg.route_experts(logits, 4, bias=bias, scores=scores)
        bad = [1, 2, 4] if scores == "softmax" else [1, 2]
        assert torch.isnan(weights[bad]).all()
        assert torch.equal(chosen[bad], torch.arange(4, dtype=I32, device="cuda").expand(len(bad), 4))
        fine = [r for r in range(8) if r not in bad and r != 4]
        assert torch.isfinite(weights[fine]).all()
        if scores == "sigmoid":
            assert int(chosen[4, 0]) == 5 and torch.isfinite(weights[4]).all()
    bias[9] = NAN
    assert torch.isnan(sptg.route_experts(logits, 4, bias=bias, scores=scores)[0]).all()


def test_route_of_strided_logits_into_given_outputs():
    g = gen(8)
    wide = rand(g, 50, 300, dtype=F32)
    for off, e in ((0, 128), (4, 128), (3, 101)):
        logits = wide[:, off:off + e]
        _, w, experts = route_reference(logits, 5)
        weights = torch.full((50, 5), NAN, device="cuda")
        chosen = torch.full((50, 5), -7, dtype=I32, device="cuda")
        got = sptg.route_experts(logits, 5, weights=weights, experts=chosen)
        assert got[0] is weights and got[1] is chosen and torch.equal(chosen, experts)
        assert_within(weights, w, 80 * UNIT * w)
    assert sptg.route_experts(wide[:0], 4)[0].shape == (0, 4)


def dlogits_reference(dweights, logits, experts, scores="softmax", renormalize=True, scale=1.0):
    """The formula's derivative, and the sum of its terms' magnitudes."""
    z, live = logits.double(), experts >= 0
    at = experts.clamp(min=0).long()
    g = dweights.double() * scale * live
    if scores == "sigmoid":
        s = 1 / (1 + torch.exp(-z))
    else:
        s = torch.softmax(z, 1).nan_to_num(0.0)
    c = torch.gather(s, 1, at) * live
    u = c
    if renormalize:
        zc = torch.gather(z, 1, at)
        u = torch.softmax((torch.nn.functional.logsigmoid(zc) if scores == "sigmoid" else zc)
                          .masked_fill(~live, -INF), 1).nan_to_num(0.0)
    dot, mag = (g * u).sum(1, keepdim=True), (g * u).abs().sum(1, keepdim=True)
    rest = 1 / (1 + torch.exp(torch.gather(z, 1, at))) if scores == "sigmoid" else 1.0
    zero = torch.zeros_like(z)
    if renormalize:
        return (zero.scatter_add(1, at, (g - dot) * u * rest * live),
                zero.scatter_add(1, at, (g.abs() + mag) * u * rest * live))
    if scores == "sigmoid":
        return zero.scatter_add(1, at, g * c * rest), zero.scatter_add(1, at, (g * c * rest).abs())
    return (zero.scatter_add(1, at, g * c) - s * dot, zero.scatter_add(1, at, (g * c).abs()) + s * mag)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("rows,e,top", [(1, 64, 8), (3, 1, 1), (50, 61, 5), (129, 256, 8), (7, 1000, 16), (9, 1024, 2)])
def test_route_dlogits(rows, e, top, renormalize, scores, dtype):
    g = gen(rows + e)
    logits, dweights = rand(g, rows, e, dtype=dtype, std=1.5), rand(g, rows, top, dtype=F32)
    if e >= top + 3:
        logits[0, 2:] = -INF  # fewer experts than places
        logits[rows // 2, 1] = -INF
    how = dict(scores=scores, renormalize=renormalize)
    experts = sptg.route_experts(logits, top, scale=1.5, **how)[1]
    ref, mag = dlogits_reference(dweights, logits, experts, scale=1.5, **how)
    got = sptg.route_experts_dlogits(dweights, logits, experts, scale=1.5, **how)
    assert got.dtype == dtype
    assert_within(got, ref, (64 + distance(logits)) * UNIT * mag)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_dlogits_of_experts_named_twice_and_out_of_range(renormalize, scores):
    g = gen(9)
    logits, dweights = rand(g, 4, 32, dtype=F32), rand(g, 4, 4, dtype=F32)
    experts = torch.tensor([[3, 3, 5, 7], [0, 1, -1, 32], [31, 31, 31, 31], [-5, 1 << 30, -1, -1]],
                           dtype=I32, device="cuda")
    known = torch.where((experts < 0) | (experts >= 32), torch.full_like(experts, -1), experts)
    ref, mag = dlogits_reference(dweights, logits, known, scores=scores, renormalize=renormalize)
    got = sptg.route_experts_dlogits(dweights, logits, experts, scores=scores, renormalize=renormalize)
    assert_within(got, ref, 80 * UNIT * mag)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradient_against_differences(renormalize, scores):
    """Central differences of the 64-bit formula, the choice held fixed (step 1e-4: error of order 1e-8)."""
    g = gen(10)
    logits, dweights = rand(g, 5, 24, dtype=F32), rand(g, 5, 4, dtype=F32)
    leaf = logits.clone().requires_grad_()
    weights, experts = sptg.route_experts(leaf, 4, scores=scores, renormalize=renormalize, scale=2.0)
    assert not experts.requires_grad
    (weights * dweights).sum().backward()

    def loss(z):
        s = torch.sigmoid(z) if scores == "sigmoid" else torch.softmax(z, 1)
        c = torch.gather(s, 1, experts.long())
        c = c / c.sum(1, keepdim=True) if renormalize else c
        return (2.0 * c * dweights.double()).sum(1)

    z = logits.double()
    for e in range(24):
        step = torch.zeros_like(z)
        step[:, e] = 1e-4
        assert ((loss(z + step) - loss(z - step)) / 2e-4 - leaf.grad[:, e]).abs().max() < 1e-5


# ------------------------------------------------- rows to experts and back
def dispatch_reference(x, experts, e):
    ids = experts.reshape(-1).long()
    ids = torch.where((ids < 0) | (ids >= e), torch.full_like(ids, e), ids)
    order = torch.sort(ids, stable=True).indices
    places = torch.empty_like(order)
    places[order] = torch.arange(len(order), device=order.device)
    offsets = torch.zeros(e + 1, dtype=torch.long, device=order.device)
    offsets[1:] = torch.cumsum(torch.bincount(ids, minlength=e + 1)[:e], 0)
    return x[order // experts.shape[1]], places.reshape(experts.shape).to(I32), offsets.to(I32)


def check_dispatch(x, experts, e):
    ref = dispatch_reference(x, experts, e)
    got = sptg.dispatch_rows(x, experts, e)
    for a, b in zip(got, ref):
        assert a.dtype == b.dtype and torch.equal(a, b)
    return got


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rows,cols,top,e", [(1, 8, 1, 1), (1, 4096, 8, 64), (4, 2048, 8, 64), (3, 7, 2, 5),
                                             (33, 1000, 3, 17), (129, 520, 8, 256), (513, 64, 8, 1024),
                                             (700, 129, 6, 24), (5000, 16, 2, 8), (20011, 8, 7, 100)])
def test_dispatch(rows, cols, top, e, dtype):
    g = gen(rows + cols)
    x = rand(g, rows, cols, dtype=dtype)
    experts = torch.randint(0, e, (rows, top), device="cuda", generator=g, dtype=I32)
    check_dispatch(x, experts, e)
    experts[rows // 2:] = -1  # padding
    experts[0, 0] = e  # and others outside
    check_dispatch(x, experts, e)
    experts[:] = e - 1  # all to the last
    check_dispatch(x, experts, e)
    experts[:] = 1 << 30  # none to any
    check_dispatch(x, experts, e)


def test_dispatch_of_no_experts_no_rows_and_no_columns():
    x = rand(gen(1), 5, 16)
    none = torch.zeros(5, 2, dtype=I32, device="cuda")
    rows, places, offsets = check_dispatch(x, none, 0)
    assert offsets.tolist() == [0]
    rows, places, offsets = sptg.dispatch_rows(x[:0], none[:0], 3)
    assert rows.shape == (0, 16) and places.shape == (0, 2) and offsets.tolist() == [0, 0, 0, 0]
    rows, places, offsets = sptg.dispatch_rows(x[:, :0], none, 3)
    assert rows.shape == (10, 0) and offsets.tolist() == [0, 10, 10, 10] and places[0, 1] == 1


@pytest.mark.parametrize("off,cols", [(0, 96), (8, 96), (3, 96), (0, 97)])
def test_dispatch_and_combine_strided_rows(off, cols):
    g = gen(12)
    wide = rand(g, 30, 300)
    experts = torch.randint(0, 4, (30, 3), device="cuda", generator=g, dtype=I32)
    out = torch.full((90, 200), NAN, dtype=BF16, device="cuda")
    x = wide[:, off:off + cols]
    ref, places, _ = dispatch_reference(x, experts, 4)
    got = sptg.dispatch_rows(x, experts, 4, out=out[:, off:off + cols])[0]
    assert torch.equal(got, ref)
    assert torch.isnan(out[:, :off]).all() and torch.isnan(out[:, off + cols:]).all()
    weights = torch.rand(30, 3, device="cuda", generator=g)
    base = wide[:, off:off + cols].clone()
    into = wide[:, off:off + cols]
    want, S = combine_reference(got, places, weights, base)
    sptg.combine_rows(got, places, weights, base=into, out=into)  # in place
    assert_within(into, want, 5 * UNIT * S)


def combine_reference(y, places, weights, base=None):
    inside = (places >= 0) & (places < y.shape[0])
    rows = torch.zeros(*places.shape, y.shape[1], dtype=torch.float64, device=y.device)
    rows[inside] = y[places[inside].long()].double()
    if weights is not None:
        rows = torch.where(inside[:, :, None], rows * weights.double()[:, :, None], rows)
    ref, S = rows.sum(1), rows.abs().sum(1)
    if base is not None:
        ref, S = ref + base.double(), S + base.double().abs()
    return ref, S


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("weighted,based", [(True, False), (True, True), (False, False)])
@pytest.mark.parametrize("rows,cols,top", [(1, 8, 1), (1, 4096, 8), (4, 2048, 8), (3, 7, 2), (33, 1000, 3),
                                           (129, 520, 9), (700, 129, 6), (300, 2056, 17), (40, 5000, 4)])
def test_combine_and_its_gradients(rows, cols, top, weighted, based, dtype):
    g = gen(rows + cols)
    y = rand(g, rows * top, cols, dtype=dtype)
    places = torch.randperm(rows * top, device="cuda", generator=g).to(I32).reshape(rows, top)
    weights = rand(g, rows, top, dtype=F32) if weighted else None
    base = rand(g, rows, cols, dtype=dtype) if based else None
    ref, S = combine_reference(y, places, weights, base)
    assert_within(sptg.combine_rows(y, places, weights, base=base), ref, (top + 2) * UNIT * S)
    dout = rand(g, rows, cols, dtype=dtype)
    dy, dweights = sptg.combine_rows_grad(dout, y, places, weights)
    flat = places.reshape(-1).long()
    d = dout.double().repeat_interleave(top, 0)
    want = torch.empty_like(y, dtype=torch.float64)
    want[flat] = d if weights is None else d * weights.double().reshape(-1, 1)
    assert_within(dy, want, UNIT * want.abs())
    if weights is None:
        assert dweights is None
    else:
        p = y[flat].double() * d
        assert_within(dweights, p.sum(1).reshape(rows, top),
                      (cols / 128 + 16) * UNIT * p.abs().sum(1).reshape(rows, top))


@pytest.mark.parametrize("cols", [64, 65])
def test_combine_of_places_outside_and_of_infinities(cols):
    g = gen(14)
    y = rand(g, 20, cols)
    places = torch.randperm(24, device="cuda", generator=g).to(I32).reshape(8, 3)  # 20 ... 23 are outside
    places[0, 0], places[1, 1], places[2, 2] = -1, -(1 << 31), (1 << 31) - 1
    weights = rand(g, 8, 3, dtype=F32)
    weights[0, 0] = NAN  # of a place that adds nothing
    ref, S = combine_reference(y, places, weights)
    assert_within(sptg.combine_rows(y, places, weights), ref, 5 * UNIT * S)
    dy = torch.full_like(y, 7.0)
    _, dweights = sptg.combine_rows_grad(rand(g, 8, cols), y, places, weights, dy=dy)
    named = torch.zeros(20, dtype=torch.bool, device="cuda")
    named[places[(places >= 0) & (places < 20)].long()] = True
    assert (dy[~named] == 7.0).all()
    assert not dweights[(places < 0) | (places >= 20)].any() and torch.isfinite(dweights).all()
    y[int(places[5, 0]) if 0 <= int(places[5, 0]) < 20 else 0, 3] = INF
    out = sptg.combine_rows(y, places, weights)
    assert int((~torch.isfinite(out)).sum()) <= 1


@pytest.mark.parametrize("rows,cols", [(40, 64), (40, 65)])
def test_dispatch_and_combine_are_differentiated(rows, cols):
    g = gen(15)
    x = rand(g, rows, cols, dtype=F16).requires_grad_()
    base = rand(g, rows, cols, dtype=F16).requires_grad_()
    weights = torch.rand(rows, 3, device="cuda", generator=g).requires_grad_()
    experts = torch.randint(-1, 6, (rows, 3), device="cuda", generator=g, dtype=I32)
    sorted_rows, places, offsets = sptg.dispatch_rows(x, experts, 6)
    out = sptg.combine_rows(sorted_rows * 2, places, weights, base=base)
    out.sum().backward()  # (an expanded gradient of ones)
    total = weights.detach().double().sum(1, keepdim=True)
    # 2 w is rounded for each place, then the sum of them
    want = (2 * total).expand(rows, cols)
    assert_within(x.grad, want, 2.0 ** -10 * want + 8 * UNIT * want)
    assert torch.equal(base.grad, torch.ones_like(base))
    dw = 2 * x.detach().double().sum(1, keepdim=True).expand(rows, 3)
    assert_within(weights.grad, dw, 20 * UNIT * 2 * x.detach().double().abs().sum(1, keepdim=True))


# ---------------------------------------------------------- the end of a block
def gate_norm_reference(y, x, w2, w1, gate, alpha, eps, dh=None, dv=None):
    """Values and gradients of the formula in 64 bits, each with the magnitudes of its terms."""
    def d(t):
        return None if t is None else t.double()
    y, x, w2, w1, gate, dh, dv = (d(t) for t in (y, x, w2, w1, gate, dh, dv))
    n = y.shape[1]
    g = torch.ones_like(y) if gate is None else gate.expand_as(y)
    p = 1.0 if w1 is None else 1 / torch.sqrt((y * y).sum(1, keepdim=True) / n + eps)
    w = torch.ones_like(y) if w1 is None else w1.expand_as(y)
    yn = y * p
    u = yn * w
    h, H = alpha * x + g * u, (alpha * x).abs() + (g * u).abs()
    q = 1 / torch.sqrt((h * h).sum(1, keepdim=True) / n + eps)
    hn, HN = h * q, H * q
    # the root's relative error is that of the mean of h's squares
    r = (H * H).sum(1, keepdim=True) * q * q / n + 1
    out = {"h": (h, H), "v": (hn * w2, (HN * r * w2).abs())}
    if dh is None and dv is None:
        return out
    dh, dv = (torch.zeros_like(y) if t is None else t for t in (dh, dv))
    a = dv * w2
    dt = dh + q * (a - hn * ((a * hn).sum(1, keepdim=True) / n))
    DT = dh.abs() + q * r * (a.abs() + HN * r * ((a.abs() * HN).sum(1, keepdim=True) / n))
    du, DU = dt * g, DT * g.abs()
    out["residual"] = (alpha * dt, abs(alpha) * DT)
    out["weight"] = ((dv * hn).sum(0), (dv.abs() * HN * r).sum(0))
    if gate is not None:
        dg, DG = dt * u, DT * u.abs()
        form = tuple(gate.shape)
        if form == (n,):
            out["gate"] = (dg.sum(0), DG.sum(0))
        elif form == tuple(y.shape):
            out["gate"] = (dg, DG)
        elif form == (y.shape[0], 1):
            out["gate"] = (dg.sum(1, keepdim=True), DG.sum(1, keepdim=True))
        else:
            out["gate"] = (dg.sum(0, keepdim=True), DG.sum(0, keepdim=True))
    if w1 is None:
        out["y"] = (du, DU)
    else:
        b, B = du * w, DU * w.abs()
        out["block_weight"] = ((du * yn).sum(0), (DU * yn.abs()).sum(0))
        out["y"] = (p * (b - yn * ((b * yn).sum(1, keepdim=True) / n)),
                    p * (B + yn.abs() * ((B * yn.abs()).sum(1, keepdim=True) / n)))
    return out


def gate_of(g, kind, rows, cols, dtype):
    if kind == "none":
        return None
    return rand(g, *{"cols": (cols,), "1cols": (1, cols), "rows": (rows, 1), "full": (rows, cols)}[kind], dtype=dtype)


def check_gate_norm(y, x, w2, w1, gate, alpha=0.75, eps=1e-5, dh=None, dv=None, out_dtype=F32, **kw):
    rows, cols = y.shape
    ref = gate_norm_reference(y, x, w2, w1, gate, alpha, eps, dh, dv)
    k = (cols / 128 + 128) * UNIT
    if dh is not None or dv is not None:
        grads = sptg.gate_add_rms_norm_grad(dh, dv, y, x, w2, w1, gate, alpha, eps, out_dtype=out_dtype)
        for name, got in zip(("y", "residual", "weight", "block_weight", "gate"), grads):
            assert (got is None) == (name not in ref), name
            if got is not None:
                want, mag = ref[name]
                wide = name in ("y", "residual") or (name == "gate" and got.shape == y.shape)
                assert got.dtype == (y.dtype if wide else out_dtype)
                assert_within(got, want, (k if wide else k + (rows / 128 + 64) * UNIT) * mag)
    h, v = sptg.gate_add_rms_norm(y, x, w2, block_weight=w1, gate=gate, alpha=alpha, eps=eps, **kw)
    assert_within(h, ref["h"][0], k * ref["h"][1])
    assert_within(v, ref["v"][0], k * ref["v"][1])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("block", [True, False])
@pytest.mark.parametrize("kind", ["none", "cols", "rows", "full", "1cols"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8), (3, 7), (5, 64), (2, 1000), (1, 4096), (4, 4104), (2, 5001),
                                       (2, 8192), (3, 8200), (2, 16384), (2, 16392), (700, 264)])
def test_gate_norm(rows, cols, kind, block, dtype):
    g = gen(rows * 7 + cols)
    y, x = rand(g, rows, cols, dtype=dtype), rand(g, rows, cols, dtype=dtype, std=2.0)
    w2, w1 = 1 + rand(g, cols, dtype=dtype, std=0.2), rand(g, cols, dtype=dtype) if block else None
    gate = gate_of(g, kind, rows, cols, dtype)
    dh, dv = rand(g, rows, cols, dtype=dtype), rand(g, rows, cols, dtype=dtype)
    check_gate_norm(y, x, w2, w1, gate, dh=dh, dv=dv)
    check_gate_norm(y, x, w2, w1, gate, dh=dh, out_dtype=dtype)
    check_gate_norm(y, x, w2, w1, gate, dv=dv)


@pytest.mark.parametrize("kind", ["rows", "full"])
@pytest.mark.parametrize("off,cols", [(0, 96), (8, 96), (3, 96), (0, 97)])
def test_gate_norm_strided_and_in_place(off, cols, kind):
    g = gen(16)
    rows = 6
    wy, wx, wg, wh = (rand(g, rows, 200) for _ in range(4))
    y, x, dh = wy[:, off:off + cols], wx[:, off:off + cols], wh[:, off:off + cols]
    gate = wg[:, off:off + cols] if kind == "full" else wg[:, 5:6]
    w2, w1 = rand(g, cols), rand(g, cols)
    check_gate_norm(y, x, w2, w1, gate, dh=dh, dv=x)
    for target in (x, y):
        ref = gate_norm_reference(y, x, w2, w1, gate, 1.0, 1e-6)
        keep = wx.clone(), wy.clone()
        h, v = sptg.gate_add_rms_norm(y, x, w2, w1, gate, h=target)
        assert h is target
        assert_within(h, ref["h"][0], 130 * UNIT * ref["h"][1])
        assert_within(v, ref["v"][0], 130 * UNIT * ref["v"][1])
        for now, old in zip((wx, wy), keep):
            assert torch.equal(now[:, :off], old[:, :off]) and torch.equal(now[:, off + cols:], old[:, off + cols:])


def test_gate_norm_of_no_rows_and_no_columns():
    for rows, cols in ((0, 64), (3, 0), (0, 0)):
        y = torch.empty(rows, cols, dtype=F16, device="cuda")
        w = torch.ones(cols, dtype=F16, device="cuda")
        for gate in (None, w, torch.ones(rows, 1, dtype=F16, device="cuda")):
            h, v = sptg.gate_add_rms_norm(y, y, w, w, gate)
            assert h.shape == v.shape == (rows, cols)
            grads = sptg.gate_add_rms_norm_grad(y, y, y, y, w, w, gate, out_dtype=F32)
            for got in grads[2:]:
                assert got is None or not got.any()


def test_gate_norm_of_zeros_infinities_and_nan():
    g = gen(17)
    y, x, w = rand(g, 8, 512), rand(g, 8, 512), rand(g, 512)
    y[1], x[1] = 0, 0
    y[2, 5], x[3, 9], x[4, 0] = NAN, INF, NAN
    y[5] = 3e38  # the sum of squares passes 32 bits: normalised to 0
    h, v = sptg.gate_add_rms_norm(y, x, w, w)
    assert not h[1].any() and not v[1].any()
    assert torch.isnan(h[2]).all() and torch.isnan(v[[2, 4]]).all() and not torch.isfinite(v[3]).all()
    assert torch.equal(h[5], x[5])
    fine = [0, 1, 5, 6, 7]
    assert torch.isfinite(h[fine]).all() and torch.isfinite(v[fine]).all()
    grads = sptg.gate_add_rms_norm_grad(y, x, y, x, w, w)
    assert torch.isfinite(grads[0][[0, 1, 6, 7]]).all() and torch.isfinite(grads[1][[0, 1, 6, 7]]).all()


@pytest.mark.parametrize("kind", ["none", "cols", "rows", "full"])
@pytest.mark.parametrize("block", [True, False])
def test_gate_norm_gradients_against_differences(kind, block):
    """Central differences of the 64-bit formula along a random direction of each input."""
    g = gen(18)
    rows, cols, eps, alpha = 4, 24, 1e-3, 0.5
    y, x, dh, dv = (rand(g, rows, cols) for _ in range(4))
    w2, w1 = rand(g, cols), rand(g, cols) if block else None
    gate = gate_of(g, kind, rows, cols, BF16)
    inputs = {"y": y, "residual": x, "weight": w2, "block_weight": w1, "gate": gate}
    leaves = {k: t.clone().requires_grad_() for k, t in inputs.items() if t is not None}
    h, v = sptg.gate_add_rms_norm(leaves["y"], leaves["residual"], leaves["weight"], leaves.get("block_weight"),
                                  leaves.get("gate"), alpha=alpha, eps=eps)
    torch.autograd.backward((h, v), (dh, dv))

    def loss(t):
        r = gate_norm_reference(t["y"], t["residual"], t["weight"], t.get("block_weight"), t.get("gate"), alpha, eps)
        return float((r["h"][0] * dh.double()).sum() + (r["v"][0] * dv.double()).sum())

    for name, leaf in leaves.items():
        way = torch.randn(leaf.shape, device="cuda", generator=g, dtype=torch.float64)
        base = {k: t.double() for k, t in inputs.items() if t is not None}
        diff = (loss({**base, name: base[name] + 1e-5 * way}) - loss({**base, name: base[name] - 1e-5 * way})) / 2e-5
        terms = leaf.grad.double() * way
        # one rounding to bfloat16 a value, and the differences' own error
        assert abs(float(terms.sum()) - diff) <= 2.0 ** -8 * float(terms.abs().sum()) + 1e-5 * (1 + abs(diff))
