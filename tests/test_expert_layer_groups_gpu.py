"""The router's choice of groups by sums of two scores, against arithmetic of 60 digits.

Sums of two scores without a bias are compared exactly whatever their size: of groups far below the row's largest
logit (softmax), of scores that all lie near zero or near one (sigmoid), and of logits that stand for no score that
32 or 64 bits hold.
"""
import functools
from decimal import Decimal, localcontext

import pytest
import torch

import software_pipelined_tiled_gb300 as sptg
from test_expert_layer_gpu import BF16, F16, F32, I32, INF, UNIT, assert_within, check_route, distance, gen, rand

pytestmark = pytest.mark.gpu
LOWEST = torch.finfo(F32).min


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    torch.cuda.synchronize()
    assert sptg.device_error() == 0


@functools.lru_cache(1 << 16)
def score(l, scores):
    """exp(l), or 1 / (1 + exp(-l)) for l <= 0.  (Logits below -10^5 are 0 beside any other.)"""
    with localcontext() as ctx:
        ctx.prec = 60
        e = Decimal(l).exp() if l > -1e5 else Decimal(0)
        return e if scores == "softmax" else e / (1 + e)


def larger_sum(a, b, scores):
    """Whether the scores of the two logits a have a larger sum than those of b."""
    if a[0] == b[0] or a[1] == b[1] or (a[0] > b[0]) == (a[1] > b[1]):  # (scores rise with their logits)
        return a > b
    ones, terms = 0, []
    for sign, l in ((1, a[0]), (1, a[1]), (-1, b[0]), (-1, b[1])):
        if scores == "sigmoid" and l > 0:  # 1 - 1 / (1 + exp(l)), the 1 added up apart
            ones, sign, l = ones + sign, -sign, -l
        terms.append(sign * score(l, scores))
    with localcontext() as ctx:
        ctx.prec = 60
        off = ones + sum(terms)
        return off > Decimal("1e-50") * max(abs(t) for t in terms)


def exact_choice(logits, top, scores, groups, top_groups):
    """The experts of each row: groups of the largest sums of two scores, of equal ones the first; then by logits."""
    t, e = logits.shape
    out = torch.full((t, top), -1, dtype=I32)
    for r, row in enumerate(logits.double().cpu().tolist()):
        size = e // groups
        two = [sorted(row[g * size:(g + 1) * size] + [-INF], reverse=True)[:2] for g in range(groups)]
        rank = [0] * groups
        for g in range(groups):
            for o in range(g):  # (the first of equal ones goes before)
                rank[o if larger_sum(two[g], two[o], scores) else g] += 1
        live = [x for x in range(e) if rank[x // size] < top_groups and row[x] > -INF]
        live.sort(key=lambda x: (-row[x], x))
        out[r, :len(live[:top])] = torch.tensor(live[:top], dtype=I32)
    return out.cuda()


def check(logits, top, scores, groups, top_groups):
    weights, chosen = sptg.route_experts(logits, top, scores=scores, groups=groups, top_groups=top_groups, group_best=2)
    want = exact_choice(logits, top, scores, groups, top_groups)
    wrong = (chosen != want).any(1).nonzero().flatten().tolist()
    assert not wrong, (wrong, chosen[wrong[0]].tolist(), want[wrong[0]].tolist())
    z = torch.gather(logits.double(), 1, want.clamp(min=0).long()).masked_fill(want < 0, -INF)
    w = torch.softmax(z if scores == "softmax" else torch.nn.functional.logsigmoid(z), 1).nan_to_num(0.0)
    assert_within(weights, w, (64 + distance(logits)) * UNIT * w)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_groups_of_two_whose_scores_32_bits_hold_no_more(scores):
    rows = [[0, 0, -120, -130, -110, -115],    # the third group's sum is the second largest
            [0, 0, -110, -115, -120, -130],
            [0, 0, -110, -115, -110, -114],    # by the smaller of two scores
            [0, 0, -110, -800, -110, -799],    # (of which 64 bits hold nothing either)
            [0, 0, -900, -901, -899, -1000],
            [0, 0, -900, -901, -900, -901],    # equal
            [0, -1, -110, -INF, -110, -200],
            [0, 0, LOWEST, LOWEST, -3e38, LOWEST],
            [0, 0, LOWEST, LOWEST, LOWEST, LOWEST]]
    for offset in (0.0, 5.0) if scores == "softmax" else (0.0, 40.0):
        logits = torch.tensor(rows, dtype=torch.float64) + offset
        check(logits.clamp(min=LOWEST).masked_fill(torch.tensor(rows) == -INF, -INF).float().cuda(), 3, scores, 3, 2)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,groups,top_groups", [(64, 32, 3), (64, 8, 4), (40, 5, 3), (256, 8, 4), (96, 3, 2)])
@pytest.mark.parametrize("std", [1.0, 40.0, 300.0])
def test_groups_of_spread_logits(std, e, groups, top_groups, scores, dtype):
    g = gen(e + groups)
    check(rand(g, 40, e, dtype=dtype, std=std), 4, scores, groups, top_groups)


@pytest.mark.parametrize("e,groups,top_groups", [(1024, 16, 8), (1023, 3, 2), (512, 4, 2)])
def test_groups_of_many_experts(e, groups, top_groups):
    for scores in ("softmax", "sigmoid"):
        check(rand(gen(e), 6, e, dtype=F32, std=150.0), 16, scores, groups, top_groups)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("at", [-69.0, -80.0, -90.0, -95.0, -100.0, -103.0, -108.0, -400.0, 20.0, 36.0, 60.0])
def test_groups_a_few_units_apart(at, scores):
    """Every group's two best logits lie some units of 32 bits around `at`, but the first's, which are 0 (a softmax's
    scores are e^at of those then; a sigmoid's of at > 0 lie e^-at below 1)."""
    g = gen(int(abs(at)))
    unit = 2.0 ** -17 if abs(at) > 64 else 2.0 ** -18
    for size in (2, 8):
        logits = torch.full((80, 8, size), LOWEST if at < 0 else at - 90, device="cuda")
        logits[:, :, :2] = at + unit * torch.randint(-6, 7, (80, 8, 2), device="cuda", generator=g)
        logits[:, 0, :2] = 0.0 if at < 0 else at + 10
        order = torch.rand(80, 8, size, device="cuda", generator=g).argsort(2)
        check(torch.gather(logits, 2, order).reshape(80, 8 * size).contiguous(), 4, scores, 8, 3)


def test_sums_of_scores_of_opposite_logits_are_equal():
    """1 / (1 + exp(-l)) + 1 / (1 + exp(l)) = 1 for every l: the first groups are chosen."""
    g = gen(3)
    half = rand(g, 200, 16, std=6.0).float()
    logits = torch.stack([half, -half], 2).reshape(200, 32)
    _, chosen = sptg.route_experts(logits, 4, scores="sigmoid", groups=16, top_groups=2)
    assert (chosen < 4).all()


@pytest.mark.parametrize("top_groups", [1, 2, 3])
def test_groups_of_biases_whose_sums_pass_32_bits(top_groups):
    """Sums of two keys past 3.4e38, all different (scores are nothing beside them)."""
    g = gen(4)
    logits = rand(g, 20, 32, dtype=F32)
    for sign in (1.0, -1.0):
        for scores in ("softmax", "sigmoid"):
            bias = sign * torch.linspace(2.0e38, 3.3e38, 32, device="cuda")[torch.randperm(32, device="cuda", generator=g)]
            check_route(logits, 4, bias=bias, scores=scores, groups=4, top_groups=top_groups)


def test_rows_of_lowest_values_in_groups():
    """Rows whose scores are all zero in 64 bits too: by the logits that stand for them."""
    g = gen(6)
    logits = rand(g, 6, 64, dtype=F32)
    logits[0] = LOWEST
    logits[1, :60] = LOWEST
    logits[2, 3:] = LOWEST
    logits[3] = LOWEST
    logits[3, 40] = -3e38
    logits[4, ::8] = LOWEST
    logits[5, 8:] = -INF
    for scores in ("softmax", "sigmoid"):
        for top_groups in (1, 4):
            check(logits, 8, scores, 8, top_groups)
