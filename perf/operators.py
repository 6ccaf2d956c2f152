"""What the operators around the dense products cost: cases, inputs, plain forms and exact values.

Three operators, as a decoder's feed-forward half uses them:

* ``norm``     residual addition and root-mean-square norm with an 8-bit output and a scale for each row
* ``w4``       products of a few rows with 4-bit weights and group scales (rows in 16 bits, or in 8 bits
               with a scale for each row, as ``norm`` writes them)
* ``experts``  products grouped by expert with ragged sizes; ``experts_grad`` their two gradients

``own`` selects between the plain form (elementary torch operations in 32 bits) and the framework's kernels.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
         "s8": torch.int8, "e4m3": torch.float8_e4m3fn}
LARGEST_8BIT = {"s8": 127.0, "e4m3": 448.0}
EPS = 1e-6


def listed():
    return [
        # one token's hidden state on its way into a feed-forward block
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 4096, "dtype": "bf16"},
        # a serving batch at an odd row count and a width that is no power of two
        {"name": "norm_batch", "op": "norm", "rows": 333, "cols": 5000, "dtype": "f16"},
        # a long prompt, or many prompts packed together
        {"name": "norm_prompt", "op": "norm", "rows": 16384, "cols": 8192, "dtype": "bf16"},
        # one token through a square projection: latency counts
        {"name": "w4_token", "op": "w4", "rows": 1, "n": 4096, "k": 4096, "group": 128, "zeros": False,
         "x": "bf16", "dtype": "bf16"},
        # one token through the widest projection of a large model: streaming the weights counts
        {"name": "w4_token_wide", "op": "w4", "rows": 1, "n": 32768, "k": 8192, "group": 64, "zeros": True,
         "x": "f16", "dtype": "f16"},
        # a decoding batch whose rows come in 8 bits from the norm
        {"name": "w4_batch", "op": "w4", "rows": 16, "n": 8192, "k": 8192, "group": 128, "zeros": False,
         "x": "s8", "dtype": "bf16"},
        # a larger batch at ragged sizes, with the smallest groups
        {"name": "w4_ragged", "op": "w4", "rows": 61, "n": 5001, "k": 4128, "group": 32, "zeros": True,
         "x": "bf16", "dtype": "bf16"},
        # one decoding step of a small batch: a few rows, most experts idle
        {"name": "experts_decode", "op": "experts", "rows": 32, "experts": 16, "n": 4096, "k": 2048,
         "skew": 1.0, "dtype": "bf16", "out": "bf16"},
        # a prompt through many experts of uneven load
        {"name": "experts_prompt", "op": "experts", "rows": 8192, "experts": 64, "n": 2048, "k": 4096,
         "skew": 1.0, "dtype": "f16", "out": "f16"},
        # a training batch through a few large experts
        {"name": "experts_train", "op": "experts", "rows": 32768, "experts": 16, "n": 4096, "k": 4096,
         "skew": 0.5, "dtype": "bf16", "out": "bf16"},
        # gradients of a small batch at ragged sizes, the weights' in 32 bits for accumulation
        {"name": "grad_ragged", "op": "experts_grad", "rows": 1531, "experts": 24, "n": 1112, "k": 2056,
         "skew": 1.5, "dtype": "f16", "out": "f32"},
        # gradients of a training batch
        {"name": "grad_train", "op": "experts_grad", "rows": 16384, "experts": 16, "n": 4096, "k": 4096,
         "skew": 0.5, "dtype": "bf16", "out": "bf16"},
    ]


def _log(rng, low, high, step=1):
    """A multiple of `step` between low and high, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return int(min(max(round(v / step) * step, low), high))


def draw(rng):
    op = rng.choice(["norm", "w4", "w4", "experts", "experts_grad"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "norm":
        return {"op": op, "rows": _log(rng, 1, 16384), "cols": _log(rng, 512, 8192, 8), "dtype": dtype}
    if op == "w4":
        group = rng.choice([32, 64, 128])
        return {"op": op, "rows": _log(rng, 1, 64), "n": _log(rng, 1000, 32768), "k": _log(rng, 1024, 8192, group),
                "group": group, "zeros": rng.random() < 0.5, "x": rng.choice([dtype, dtype, "s8", "e4m3"]),
                "dtype": dtype}
    rows = _log(rng, 8, 32768 if op == "experts" else 16384)
    return {"op": op, "rows": rows, "experts": _log(rng, 4, 64), "n": _log(rng, 512, 4096, 8),
            "k": _log(rng, 512, 4096, 8), "skew": rng.choice([0.0, 0.5, 1.0, 1.5]), "dtype": dtype,
            "out": rng.choice([dtype, "f32"])}


def work(case):
    op = case["op"]
    if op == "norm":
        r, c = case["rows"], case["cols"]
        # x and residual in, residual and 8-bit values out, the weight once, a scale for each row
        return {"bytes": r * c * 7 + c * 2 + r * 4, "flops": 8.0 * r * c}
    if op == "w4":
        m, n, k, g = case["rows"], case["n"], case["k"], case["group"]
        x = m * k * 2 if case["x"] in ("bf16", "f16") else m * k + m * 4
        return {"bytes": n * k // 2 + n * (k // g) * (3 if case["zeros"] else 2) + x + m * n * 2,
                "flops": 2.0 * m * n * k}
    t, n, k = case["rows"], case["n"], case["k"]
    # experts without rows need not be read: at most one for each row
    used, wide = min(case["experts"], t), 4 if case["out"] == "f32" else 2
    if op == "experts":
        return {"bytes": t * k * 2 + used * n * k * 2 + t * n * wide, "flops": 2.0 * t * n * k}
    # dY and W in, dX out; dY and X in, dW out (whole: idle experts get zeros)
    return {"bytes": t * n * 2 + t * k * 2 + used * n * k * 2 + t * k * 2 + case["experts"] * n * k * wide,
            "flops": 4.0 * t * n * k}


def _sizes(case, seed):
    """Rows of each expert: a draw from loads whose logarithms are normal with deviation `skew`."""
    r = np.random.RandomState(seed % (1 << 31))
    load = np.exp(case["skew"] * r.randn(case["experts"]))
    return r.multinomial(case["rows"], load / load.sum())


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(dev).manual_seed(int(seed))
    dtype = TYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, device=dev, generator=g, dtype=torch.float32).mul_(std).to(dtype)

    s = dict(case)
    if case["op"] == "norm":
        r, c = case["rows"], case["cols"]
        s["data"] = {"x": normal(r, c), "residual": normal(r, c, std=4.0),
                     "weight": (1 + 0.1 * torch.randn(c, device=dev, generator=g)).to(dtype)}
    elif case["op"] == "w4":
        m, n, k, gr = case["rows"], case["n"], case["k"], case["group"]
        d = {}
        # two codes a byte, the even column's in the low half
        d["packed"] = torch.randint(0, 256, (n, k // 2), device=dev, generator=g, dtype=torch.uint8)
        d["scales"] = (torch.rand(n, k // gr, device=dev, generator=g) * 0.01 + 0.002).to(dtype)
        d["zeros"] = (torch.randint(5, 11, (n, k // gr), device=dev, generator=g, dtype=torch.uint8)
                      if case["zeros"] else None)
        x = torch.randn(m, k, device=dev, generator=g)
        if case["x"] in LARGEST_8BIT:
            top = LARGEST_8BIT[case["x"]]
            d["x_scales"] = x.abs().amax(1) / top
            x = x / d["x_scales"][:, None]
            d["x"] = x.round().to(torch.int8) if case["x"] == "s8" else x.to(torch.float8_e4m3fn)
        else:
            d["x"], d["x_scales"] = x.to(dtype), None
        s["data"] = d
    else:
        t, e, n, k = case["rows"], case["experts"], case["n"], case["k"]
        sizes = _sizes(case, seed)
        off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        d = {"offsets": torch.from_numpy(off).to(dev), "W": normal(e, n, k, std=k ** -0.5), "X": normal(t, k)}
        if case["op"] == "experts_grad":
            d["dY"] = normal(t, n)
        s["data"], s["most"] = d, int(max(1, sizes.max()))  # the plain form pads every expert to the largest
    return s


def _plain_norm(s):
    d = s["data"]
    h = d["x"].float() + d["residual"].float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * d["weight"].float()
    a = y.abs().amax(1, keepdim=True)
    q = torch.where(a > 0, y * (448.0 / a), torch.zeros_like(y))
    return {"h": h.to(d["x"].dtype), "q": q.to(torch.float8_e4m3fn), "scales": a[:, 0] / 448.0}


def _plain_w4(s):
    d, gr = s["data"], s["group"]
    n = s["n"]
    codes = torch.stack([d["packed"] & 15, d["packed"] >> 4], dim=2).reshape(n, -1, gr).float()
    zero = 8.0 if d["zeros"] is None else d["zeros"].float()[:, :, None]
    w = ((codes - zero) * d["scales"].float()[:, :, None]).reshape(n, -1)
    y = d["x"].float() @ w.t()
    if d["x_scales"] is not None:
        y = y * d["x_scales"][:, None]
    return {"y": y.to(d["scales"].dtype)}


def _padded(rows, offsets, most):
    """The rows of each expert, padded with zero rows to `most`: (experts, most, columns)."""
    at = offsets[:-1, None].long() + torch.arange(most, device=rows.device)
    live = at < offsets[1:, None]
    return rows[at.clamp(max=rows.shape[0] - 1)].float() * live[:, :, None]


def _unpadded(padded, offsets, count):
    t = torch.arange(count, device=padded.device)
    e = torch.searchsorted(offsets.long(), t, right=True) - 1
    return padded[e, t - offsets.long()[e]]


def _plain_experts(s):
    d = s["data"]
    y = torch.bmm(_padded(d["X"], d["offsets"], s["most"]), d["W"].float().transpose(1, 2))
    return {"y": _unpadded(y, d["offsets"], s["rows"]).to(TYPES[s["out"]])}


def _plain_experts_grad(s):
    d = s["data"]
    dy = _padded(d["dY"], d["offsets"], s["most"])
    dx = torch.bmm(dy, d["W"].float())
    dw = torch.bmm(dy.transpose(1, 2), _padded(d["X"], d["offsets"], s["most"]))
    return {"dx": _unpadded(dx, d["offsets"], s["rows"]).to(d["X"].dtype), "dw": dw.to(TYPES[s["out"]])}


_PLAIN = {"norm": _plain_norm, "w4": _plain_w4, "experts": _plain_experts, "experts_grad": _plain_experts_grad}


def run(state):
    op, d = state["op"], state["data"]
    if not own:
        return _PLAIN[op](state)
    import software_pipelined_tiled_gb300 as sptg
    if op == "norm":
        h, q, scales = sptg.add_rms_norm(d["x"], d["residual"], d["weight"], eps=EPS, out_dtype=torch.float8_e4m3fn)
        return {"h": h, "q": q, "scales": scales}
    if op == "w4":
        return {"y": sptg.gemm_w4(d["x"], d["packed"], d["scales"], d["zeros"], x_scales=d["x_scales"])}
    if op == "experts":
        return {"y": sptg.grouped_gemm(d["X"], d["W"], d["offsets"], out_dtype=TYPES[state["out"]])}
    return {"dx": sptg.grouped_gemm_dx(d["dY"], d["W"], d["offsets"]),
            "dw": sptg.grouped_gemm_dw(d["dY"], d["X"], d["offsets"], out_dtype=TYPES[state["out"]])}


def _e4m3(y):
    """The e4m3 value nearest to each of y (64 bits, |y| <= 448), ties to even: 3 fraction bits from 2**-6 up, steps of 2**-9 below."""
    exponent = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(exponent - 3)
    return torch.round(y / step) * step


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    d = s["data"]
    if op == "norm":
        h = d["x"].double() + d["residual"].double()
        rms = (h.square().sum(1) / h.shape[1] + EPS).sqrt()
        y = h / rms[:, None] * d["weight"].double()
        scale = y.abs().max(1).values / 448
        return {"h": h, "q": _e4m3(y / scale[:, None]), "scales": scale}
    if op == "w4":
        n, k, gr = case["n"], case["k"], case["group"]
        w = torch.empty(n, k, dtype=torch.float64, device=d["x"].device)
        w[:, 0::2] = d["packed"].bitwise_and(15).double()
        w[:, 1::2] = torch.div(d["packed"], 16, rounding_mode="floor").double()
        w -= 8 if d["zeros"] is None else d["zeros"].double().repeat_interleave(gr, 1)
        w *= d["scales"].double().repeat_interleave(gr, 1)
        y = torch.einsum("mk,nk->mn", d["x"].to(torch.float32).double(), w)
        return {"y": y if d["x_scales"] is None else torch.einsum("mn,m->mn", y, d["x_scales"].double())}
    if (2.0 if op == "experts" else 4.0) * case["rows"] * case["n"] * case["k"] > 6e12:
        return None
    off = d["offsets"].tolist()
    t, n, k = case["rows"], case["n"], case["k"]
    dev = d["X"].device
    if op == "experts":
        y = torch.zeros(t, n, dtype=torch.float64, device=dev)
        for e in range(case["experts"]):
            a, b = off[e], off[e + 1]
            y[a:b] = d["X"][a:b].double() @ d["W"][e].double().T
        return {"y": y}
    dx = torch.zeros(t, k, dtype=torch.float64, device=dev)
    dw = torch.zeros(case["experts"], n, k, dtype=torch.float64, device=dev)
    for e in range(case["experts"]):
        a, b = off[e], off[e + 1]
        dy = d["dY"][a:b].double()
        dx[a:b] = dy @ d["W"][e].double()
        dw[e] = dy.T @ d["X"][a:b].double()
    return {"dx": dx, "dw": dw}
