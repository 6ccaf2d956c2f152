"""What the operators around an expert layer cost: cases, inputs, plain forms and exact values.

Four operators, which surround the products grouped by expert in a decoder's feed-forward half:

* ``route``     the router: scores of the experts from logits, the best ones of each row and their weights, and
                the logits' gradient
* ``dispatch``  rows sorted by expert, for the grouped products, and the rows' gradient
* ``combine``   the experts' outputs back in the order of the rows, weighted and added up, and their gradients
* ``norm``      the block's end: norm of its output, gate, scaled residual, norm for the next block, and the gradients

``own`` selects between the plain form (elementary torch operations) and the framework's kernels.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6


def listed():
    return [
        # one token through a router: latency counts
        {"name": "route_token", "op": "route", "rows": 1, "experts": 64, "top": 8, "scores": "softmax", "bias": False,
         "groups": 1, "top_groups": 1, "group_best": 1, "renormalize": True, "scale": 1.0, "dtype": "bf16", "grad": False},
        # a serving batch, experts in groups of an odd size, a bias that balances their loads
        {"name": "route_batch", "op": "route", "rows": 331, "experts": 160, "top": 6, "scores": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 3, "group_best": 2, "renormalize": True, "scale": 2.5, "dtype": "f32", "grad": False},
        # a training batch through many experts, with the gradient
        {"name": "route_train", "op": "route", "rows": 32768, "experts": 256, "top": 8, "scores": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "group_best": 2, "renormalize": True, "scale": 2.5, "dtype": "f32", "grad": True},
        # a few tokens of a decoding step
        {"name": "dispatch_token", "op": "dispatch", "rows": 4, "cols": 2048, "experts": 64, "top": 8, "skew": 1.0,
         "padded": 0.0, "dtype": "bf16", "grad": False},
        # a training batch, with the gradient; the last rows are padding and go to no expert
        {"name": "dispatch_train", "op": "dispatch", "rows": 16384, "cols": 4096, "experts": 128, "top": 8, "skew": 0.5,
         "padded": 0.02, "dtype": "bf16", "grad": True},
        # a few tokens of a decoding step
        {"name": "combine_token", "op": "combine", "rows": 4, "cols": 2048, "experts": 64, "top": 8, "skew": 1.0,
         "base": False, "dtype": "bf16", "grad": False},
        # a small ragged batch with the output of experts that every row goes through, and the gradients
        {"name": "combine_ragged", "op": "combine", "rows": 1531, "cols": 2056, "experts": 24, "top": 6, "skew": 1.5,
         "base": True, "dtype": "f16", "grad": True},
        # a training batch, with the gradients
        {"name": "combine_train", "op": "combine", "rows": 16384, "cols": 4096, "experts": 128, "top": 8, "skew": 0.5,
         "base": False, "dtype": "bf16", "grad": True},
        # one token at the end of a block
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 4096, "block": True, "gate": "cols", "alpha": 1.0,
         "dtype": "bf16", "grad": False},
        # a small batch at an odd row count and a width that is no power of two, a gate for every element, all gradients
        {"name": "norm_ragged", "op": "norm", "rows": 333, "cols": 5000, "block": True, "gate": "full", "alpha": 0.5,
         "dtype": "f16", "grad": True},
        # a long prompt, or many prompts packed together
        {"name": "norm_prompt", "op": "norm", "rows": 16384, "cols": 8192, "block": True, "gate": "rows", "alpha": 1.0,
         "dtype": "bf16", "grad": False},
        # a training batch with all gradients
        {"name": "norm_train", "op": "norm", "rows": 16384, "cols": 4096, "block": True, "gate": "cols", "alpha": 0.75,
         "dtype": "bf16", "grad": True},
    ]


def _log(rng, low, high, step=1):
    """A multiple of `step` between low and high, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return int(min(max(round(v / step) * step, low), high))


def draw(rng):
    op = rng.choice(["route", "dispatch", "combine", "norm"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        experts = _log(rng, 16, 256, 2 * groups)
        experts = max(experts // groups, 2) * groups
        top_groups = rng.randint(min(2, groups), groups)
        return {"op": op, "rows": _log(rng, 1, 32768), "experts": experts,
                "top": rng.randint(1, min(8, experts // groups * top_groups)), "scores": rng.choice(["softmax", "sigmoid"]),
                "bias": rng.random() < 0.5, "groups": groups, "top_groups": top_groups, "group_best": rng.choice([1, 2]),
                "renormalize": rng.random() < 0.6, "scale": rng.choice([1.0, 2.5]), "dtype": rng.choice(["bf16", "f16", "f32"]),
                "grad": rng.random() < 0.5}
    dtype, grad = rng.choice(["bf16", "f16"]), rng.random() < 0.5
    if op == "norm":
        cols = _log(rng, 512, 8192, 8 if rng.random() < 0.75 else 1)
        rows = min(_log(rng, 1, 16384), 16384 * (2048 if grad else 6144) // cols)
        return {"op": op, "rows": rows, "cols": cols, "block": rng.random() < 0.75,
                "gate": rng.choice(["none", "cols", "rows", "full"]), "alpha": rng.choice([1.0, 0.5, 0.22]), "dtype": dtype,
                "grad": grad}
    case = {"op": op, "rows": _log(rng, 1, 16384), "cols": _log(rng, 512, 4096, 8 if rng.random() < 0.75 else 1),
            "experts": _log(rng, 8, 256), "top": rng.randint(1, 8), "skew": rng.choice([0.0, 0.5, 1.0, 1.5])}
    if op == "dispatch":
        case["padded"] = rng.choice([0.0, 0.1])
    else:
        case["base"] = case["top"] < 8 and rng.random() < 0.5
    return {**case, "dtype": dtype, "grad": grad}


def work(case):
    op, t = case["op"], case["rows"]
    if op == "route":
        e, k, b = case["experts"], case["top"], BYTES[case["dtype"]]
        # logits and bias in, weights and experts out; their gradients in and the logits' out
        return {"bytes": t * e * b + (e * 4 if case["bias"] else 0) + t * k * 8 + (t * k * 4 + t * e * b if case["grad"] else 0),
                "flops": 4.0 * t * e * (2 if case["grad"] else 1)}
    c = case["cols"]
    if op == "dispatch":
        k = case["top"]
        # experts and rows in; sorted rows, places and offsets out; the sorted rows' gradient in, the rows' out
        return {"bytes": t * k * 8 + (case["experts"] + 1) * 4 + t * c * 2 * (1 + k) * (2 if case["grad"] else 1),
                "flops": float(t * c * k) if case["grad"] else 0.0}
    if op == "combine":
        k, base = case["top"], 1 if case["base"] else 0
        # places, weights, experts' outputs (and the base) in, rows out; the rows' gradient in, those of the
        # experts' outputs and of the weights out
        return {"bytes": t * k * 8 + t * c * 2 * (k + 1 + base) + (t * k * 4 + t * c * 2 * (1 + k) if case["grad"] else 0),
                "flops": 2.0 * t * c * k * (2.5 if case["grad"] else 1)}
    gate = {"none": 0, "cols": c, "rows": t, "full": t * c}[case["gate"]] * 2
    weights = (2 if case["block"] else 1) * c * 2
    # the block's output, the residual, weights and gate in, the new residual and its norm out; gradients of these
    # two in, of all the inputs out
    return {"bytes": t * c * 8 + weights + gate + (t * c * 8 + weights + gate if case["grad"] else 0),
            "flops": 12.0 * t * c * (3 if case["grad"] else 1)}


def _chosen(case, g, dev):
    """Experts of each row, distinct and in no order, of uneven load; rows of padding have none (-1)."""
    t, e, k = case["rows"], case["experts"], min(case["top"], case["experts"])
    load = case["skew"] * torch.randn(e, device=dev, generator=g)
    noise = -torch.log(-torch.log(torch.rand(t, e, device=dev, generator=g).clamp(1e-9, 1 - 1e-7)))
    chosen = torch.sort(load + noise, dim=1, descending=True).indices[:, :k].to(torch.int32).contiguous()
    padded = int(t * case.get("padded", 0.0))
    if padded:
        chosen[t - padded:] = -1
    return chosen


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(dev).manual_seed(int(seed))
    dtype = TYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=dtype):
        return torch.randn(*shape, device=dev, generator=g).mul_(std).add_(mean).to(dtype)

    s, op, t = dict(case), case["op"], case["rows"]
    if op == "route":
        d = {"logits": normal(t, case["experts"], std=1.5),
             "bias": normal(case["experts"], std=0.05, dtype=torch.float32) if case["bias"] else None}
        if case["grad"]:
            d["dweights"] = normal(t, case["top"], dtype=torch.float32)
    elif op == "norm":
        c = case["cols"]
        d = {"y": normal(t, c, std=0.7), "residual": normal(t, c, std=2.0), "weight": normal(c, std=0.1, mean=1.0),
             "block_weight": normal(c, std=0.1, mean=0.5) if case["block"] else None, "gate": None}
        if case["gate"] != "none":
            d["gate"] = normal(*{"cols": (c,), "rows": (t, 1), "full": (t, c)}[case["gate"]], std=0.3, mean=0.6)
        if case["grad"]:
            d["dh"], d["dv"] = normal(t, c), normal(t, c)
    else:
        c, chosen = case["cols"], _chosen(case, g, dev)
        k = chosen.shape[1]
        if op == "dispatch":
            d = {"x": normal(t, c), "experts": chosen}
            if case["grad"]:
                d["dsorted"] = normal(t * k, c)
        else:
            # what the dispatch of these rows left: where each of them went
            order = torch.sort(chosen.reshape(-1), stable=True).indices
            places = torch.empty_like(order)
            places[order] = torch.arange(t * k, device=dev)
            weights = torch.rand(t, k, device=dev, generator=g) + 0.05
            d = {"y": normal(t * k, c), "places": places.to(torch.int32).reshape(t, k),
                 "weights": weights / weights.sum(1, keepdim=True), "base": normal(t, c) if case["base"] else None}
            if case["grad"]:
                d["dout"] = normal(t, c)
    s["data"] = d
    return s


def _route_scores(s, logits):
    if s["scores"] == "sigmoid":
        return 1 / (1 + torch.exp(-logits))
    p = torch.exp(logits - logits.amax(1, keepdim=True))
    return p / p.sum(1, keepdim=True)


def _plain_route(s):
    d = s["data"]
    # in 64 bits: two experts' scores may lie closer than 32 bits tell apart
    scores = _route_scores(s, d["logits"].double())
    keys = scores if d["bias"] is None else scores + d["bias"].double()
    t, e = keys.shape
    if s["groups"] > 1:
        members = keys.reshape(t, s["groups"], -1)
        best = torch.sort(members, dim=2, descending=True).values[:, :, :s["group_best"]].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        live = torch.zeros(t, s["groups"], dtype=torch.bool, device=keys.device)
        live[torch.arange(t, device=keys.device)[:, None], kept] = True
        keys = torch.where(live[:, :, None], members, torch.full_like(members, -math.inf)).reshape(t, e)
    experts = torch.sort(keys, dim=1, descending=True, stable=True).indices[:, :s["top"]]
    at = (torch.arange(t, device=keys.device)[:, None], experts)
    chosen = scores[at]
    total = chosen.sum(1, keepdim=True)
    out = {"weights": ((chosen / total if s["renormalize"] else chosen) * s["scale"]).float(), "experts": experts.to(torch.int32)}
    if s["grad"]:
        dchosen = d["dweights"].double() * s["scale"]
        if s["renormalize"]:
            dchosen = (dchosen - (dchosen * chosen / total).sum(1, keepdim=True)) / total
        dscores = torch.zeros_like(scores)
        dscores[at] = dchosen
        if s["scores"] == "sigmoid":
            dlogits = dscores * scores * (1 - scores)
        else:
            dlogits = scores * (dscores - (dscores * scores).sum(1, keepdim=True))
        out["dlogits"] = dlogits.to(d["logits"].dtype)
    return out


def _plain_dispatch(s):
    d, e = s["data"], s["experts"]
    t, k = d["experts"].shape
    ids = d["experts"].reshape(-1)
    ids = torch.where((ids >= 0) & (ids < e), ids, torch.full_like(ids, e))  # those of no expert come last
    order = torch.sort(ids, stable=True).indices
    places = torch.empty_like(order)
    places[order] = torch.arange(t * k, device=ids.device)
    counts = (ids[:, None] == torch.arange(e, device=ids.device)).sum(0)
    offsets = torch.zeros(e + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = torch.cumsum(counts, 0)
    out = {"sorted": d["x"][order // k], "places": places.to(torch.int32).reshape(t, k), "offsets": offsets}
    if s["grad"]:
        out["dx"] = _plain_sum(d["dsorted"], out["places"], None, None)
    return out


def _plain_sum(y, places, weights, base):
    out = torch.zeros(places.shape[0], y.shape[1], device=y.device) if base is None else base.float()
    for j in range(places.shape[1]):
        rows = y[places[:, j].long()].float()
        out += rows if weights is None else rows * weights[:, j, None]
    return out.to(y.dtype)


def _plain_combine(s):
    d = s["data"]
    out = {"out": _plain_sum(d["y"], d["places"], d["weights"], d["base"])}
    if s["grad"]:
        dout, dy, dweights = d["dout"].float(), torch.empty_like(d["y"]), torch.empty_like(d["weights"])
        for j in range(d["places"].shape[1]):
            at = d["places"][:, j].long()
            dweights[:, j] = (d["y"][at].float() * dout).sum(1)
            dy[at] = (dout * d["weights"][:, j, None]).to(dy.dtype)
        out["dy"], out["dweights"] = dy, dweights
    return out


def _plain_norm(s):
    d = s["data"]
    dtype = d["y"].dtype
    y, x, w2 = d["y"].float(), d["residual"].float(), d["weight"].float()
    u, r1 = y, None
    if d["block_weight"] is not None:
        w1, r1 = d["block_weight"].float(), torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
        u = y * r1 * w1
    g = 1.0 if d["gate"] is None else d["gate"].float()
    h = s["alpha"] * x + g * u
    r2 = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    out = {"h": h.to(dtype), "v": (h * r2 * w2).to(dtype)}
    if s["grad"]:
        dv = d["dv"].float()
        a = dv * w2
        dh = d["dh"].float() + r2 * (a - h * r2 * r2 * (a * h).mean(1, keepdim=True))
        out["dresidual"] = (s["alpha"] * dh).to(dtype)
        out["dweight"] = (dv * h * r2).sum(0)
        du = dh * g
        if s["gate"] == "cols":
            out["dgate"] = (dh * u).sum(0)
        elif s["gate"] == "rows":
            out["dgate"] = (dh * u).sum(1, keepdim=True)
        elif s["gate"] == "full":
            out["dgate"] = (dh * u).to(dtype)
        if r1 is None:
            out["dy"] = du.to(dtype)
        else:
            b = du * w1
            out["dy"] = (r1 * (b - y * r1 * r1 * (b * y).mean(1, keepdim=True))).to(dtype)
            out["dblock_weight"] = (du * y * r1).sum(0)
    return out


_PLAIN = {"route": _plain_route, "dispatch": _plain_dispatch, "combine": _plain_combine, "norm": _plain_norm}


def run(state):
    s, op, d = state, state["op"], state["data"]
    if not own:
        return _PLAIN[op](s)
    import software_pipelined_tiled_gb300 as sptg
    if op == "route":
        weights, experts = sptg.route_experts(
            d["logits"], s["top"], bias=d["bias"], scores=s["scores"], groups=s["groups"], top_groups=s["top_groups"],
            group_best=s["group_best"], renormalize=s["renormalize"], scale=s["scale"])
        out = {"weights": weights, "experts": experts}
        if s["grad"]:
            out["dlogits"] = sptg.route_experts_dlogits(d["dweights"], d["logits"], experts, scores=s["scores"],
                                                        renormalize=s["renormalize"], scale=s["scale"])
        return out
    if op == "dispatch":
        rows, places, offsets = sptg.dispatch_rows(d["x"], d["experts"], s["experts"])
        out = {"sorted": rows, "places": places, "offsets": offsets}
        if s["grad"]:
            out["dx"] = sptg.dispatch_rows_dx(d["dsorted"], places)
        return out
    if op == "combine":
        out = {"out": sptg.combine_rows(d["y"], d["places"], d["weights"], base=d["base"])}
        if s["grad"]:
            out["dy"], out["dweights"] = sptg.combine_rows_grad(d["dout"], d["y"], d["places"], d["weights"])
        return out
    h, v = sptg.gate_add_rms_norm(d["y"], d["residual"], d["weight"], block_weight=d["block_weight"], gate=d["gate"],
                                  alpha=s["alpha"], eps=EPS)
    out = {"h": h, "v": v}
    if s["grad"]:
        # the broadcast inputs' gradients in 32 bits, as an optimizer adds them up
        grads = sptg.gate_add_rms_norm_grad(d["dh"], d["dv"], d["y"], d["residual"], d["weight"],
                                            block_weight=d["block_weight"], gate=d["gate"], alpha=s["alpha"], eps=EPS,
                                            out_dtype=torch.float32)
        out["dy"], out["dresidual"], out["dweight"] = grads[:3]
        if d["block_weight"] is not None:
            out["dblock_weight"] = grads[3]
        if d["gate"] is not None:
            out["dgate"] = grads[4]
    return out


def _exact_route(case, d):
    z = d["logits"].to(torch.float64)
    t, e = z.shape
    row = torch.arange(t, device=z.device)
    p = torch.sigmoid(z) if case["scores"] == "sigmoid" else torch.softmax(z, dim=1)
    key = p.clone() if d["bias"] is None else p + d["bias"].to(torch.float64)
    if case["groups"] > 1:
        size = e // case["groups"]
        best = torch.stack([key[:, i * size:(i + 1) * size].topk(case["group_best"], dim=1).values.sum(1)
                            for i in range(case["groups"])], 1)
        for _ in range(case["groups"] - case["top_groups"]):  # the worst group leaves, of equal ones the last
            worst = case["groups"] - 1 - best.flip(1).argmin(1)
            best[row, worst] = math.inf
            key.masked_fill_((torch.arange(e, device=z.device) // size)[None, :] == worst[:, None], -math.inf)
    picks = []
    for _ in range(case["top"]):
        pick = key.argmax(1)
        key[row, pick] = -math.inf
        picks.append(pick)
    picks = torch.stack(picks, 1)
    w = torch.gather(p, 1, picks)
    norm = w.sum(1, keepdim=True) if case["renormalize"] else torch.ones_like(w[:, :1])
    out = {"weights": case["scale"] * w / norm, "experts": picks.to(torch.int32)}
    if case["grad"]:
        # of every score by every logit: the chosen ones' derivatives, row by row
        gw = case["scale"] * d["dweights"].to(torch.float64) / norm
        if case["renormalize"]:
            gw = gw - (gw * w).sum(1, keepdim=True) / norm
        if case["scores"] == "sigmoid":
            out["dlogits"] = torch.zeros_like(z).scatter_(1, picks, gw * w * (1 - w))
        else:
            out["dlogits"] = (torch.zeros_like(z).scatter_(1, picks, gw * w) - p * (gw * w).sum(1, keepdim=True))
    return out


def _exact_dispatch(case, d):
    t, k = d["experts"].shape
    e = case["experts"]
    ids = d["experts"].cpu().long().reshape(-1)
    ids[(ids < 0) | (ids >= e)] = e
    count = torch.bincount(ids, minlength=e + 1)
    order = torch.argsort(ids * (t * k) + torch.arange(t * k))  # (all different)
    places = torch.argsort(order)
    dev = d["x"].device
    out = {"sorted": d["x"].to(torch.float64)[order.to(dev) // k], "places": places.reshape(t, k).to(torch.int32),
           "offsets": torch.cat([torch.zeros(1, dtype=torch.int64), count[:e].cumsum(0)]).to(torch.int32)}
    if case["grad"]:
        dx = torch.zeros(d["x"].shape, dtype=torch.float64, device=dev)
        out["dx"] = dx.index_add_(0, order.to(dev) // k, d["dsorted"].to(torch.float64))
    return out


def _exact_combine(case, d):
    t, k = d["places"].shape
    y, w = d["y"].to(torch.float64), d["weights"].to(torch.float64)
    flat = d["places"].long().reshape(-1)
    source = torch.empty_like(flat)
    source[flat] = torch.arange(t * k, device=flat.device)  # the entry that each row of y belongs to
    out = torch.zeros(t, y.shape[1], dtype=torch.float64, device=y.device)
    out.index_add_(0, source // k, y * w.reshape(-1)[source, None])
    if d["base"] is not None:
        out += d["base"].to(torch.float64)
    result = {"out": out}
    if case["grad"]:
        dout = d["dout"].to(torch.float64)[source // k]
        dw = torch.empty(t * k, dtype=torch.float64, device=y.device)
        dw[source] = torch.einsum("rc,rc->r", y, dout)
        result["dweights"] = dw.reshape(t, k)
        del y
        result["dy"] = dout.mul_(w.reshape(-1)[source, None])
    return result


def _exact_norm(case, d):
    def f64(name):
        return None if d[name] is None else d[name].to(torch.float64)

    y, x, w2, w1, gate = f64("y"), f64("residual"), f64("weight"), f64("block_weight"), f64("gate")
    n = y.shape[1]
    a1 = None if w1 is None else ((y ** 2).sum(1, keepdim=True) / n + EPS) ** -0.5
    u = y if w1 is None else y * a1 * w1
    gu = u if gate is None else u * gate
    h = case["alpha"] * x + gu
    a2 = ((h ** 2).sum(1, keepdim=True) / n + EPS) ** -0.5
    unit = h * a2
    out = {"h": h, "v": unit * w2}
    if case["grad"]:
        dunit = f64("dv") * w2
        out["dweight"] = torch.einsum("tc,tc->c", f64("dv"), unit)
        dh = f64("dh") + a2 * (dunit - unit * ((dunit * unit).sum(1, keepdim=True) / n))
        out["dresidual"] = case["alpha"] * dh
        if case["gate"] != "none":
            form = {"cols": "tc,tc->c", "rows": "tc,tc->t", "full": "tc,tc->tc"}[case["gate"]]
            dgate = torch.einsum(form, dh, u)
            out["dgate"] = dgate[:, None] if case["gate"] == "rows" else dgate
        du = dh if gate is None else dh * gate
        if w1 is None:
            out["dy"] = du
        else:
            unit1 = y * a1
            out["dblock_weight"] = torch.einsum("tc,tc->c", du, unit1)
            b = du * w1
            out["dy"] = a1 * (b - unit1 * ((b * unit1).sum(1, keepdim=True) / n))
    return out


def exact(case, seed):
    d = prepare(case, seed)["data"]
    return {"route": _exact_route, "dispatch": _exact_dispatch, "combine": _exact_combine, "norm": _exact_norm}[case["op"]](case, d)
