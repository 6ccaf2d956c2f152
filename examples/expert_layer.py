"""A decoder's feed-forward half on the library's operators, for decoding and for training.

    python examples/expert_layer.py [--rows 64] [--hidden 2048] [--inner 4096] [--experts 16] [--top 2]

One step, as a serving process makes it for the tokens in flight:

1. residual addition and norm into int8 with a scale for each row (``add_rms_norm``);
2. a dense projection with 4-bit weights on those rows (``gemm_w4``);
3. residual addition and norm into 16 bits;
4. a router's logits (``gemm``), the best experts of each row, rows sorted by expert;
5. two products grouped by expert around an activation (``grouped_gemm``).

A training step then takes the gradients of the experts' weights and inputs
(``grouped_gemm_dw``, ``grouped_gemm_dx``).  Weights and inputs are random.  The
script prints the time of a step and how far it is from a plain float32 version
on the same data.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import software_pipelined_tiled_gb300 as sptg  # noqa: E402

EPS, GROUP = 1e-6, 128


def make_layer(hidden: int, inner: int, experts: int, dtype=torch.bfloat16, seed: int = 0) -> dict:
    """Random weights of one layer on the current GPU."""
    g = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape, std):
        return (torch.randn(*shape, device="cuda", generator=g) * std).to(dtype)

    return {
        "norm1": 1 + normal(hidden, std=0.1), "norm2": 1 + normal(hidden, std=0.1),
        # 4-bit codes, two to a byte, with a scale and a zero point for each 128 columns
        "codes": torch.randint(0, 256, (hidden, hidden // 2), device="cuda", generator=g,
                               dtype=torch.uint8),
        "scales": (torch.rand(hidden, hidden // GROUP, device="cuda", generator=g) * 0.004
                   + 0.001).to(dtype),
        "zeros": torch.randint(6, 10, (hidden, hidden // GROUP), device="cuda", generator=g,
                               dtype=torch.uint8),
        "router": normal(experts, hidden, std=hidden ** -0.5),
        "up": normal(experts, inner, hidden, std=hidden ** -0.5),
        "down": normal(experts, hidden, inner, std=inner ** -0.5),
    }


def route(logits, top: int):
    """Rows sorted by expert: (row of each sorted row, its weight, offsets of the experts)."""
    weights, chosen = torch.topk(torch.softmax(logits.float(), dim=1), top, dim=1)
    weights = weights / weights.sum(1, keepdim=True)
    expert, order = torch.sort(chosen.reshape(-1), stable=True)
    counts = torch.zeros(logits.shape[1], dtype=torch.int64, device=logits.device)
    counts.index_add_(0, expert, torch.ones_like(expert))
    offsets = torch.zeros(logits.shape[1] + 1, dtype=torch.int32, device=logits.device)
    torch.cumsum(counts, 0, out=offsets[1:])
    return order // top, weights.reshape(-1)[order], offsets


def forward(layer: dict, x, residual, top: int) -> dict:
    """One step of the layer; keeps what the gradients need."""
    h, q, s = sptg.add_rms_norm(x, residual, layer["norm1"], eps=EPS, out_dtype=torch.int8)
    a = sptg.gemm_w4(q, layer["codes"], layer["scales"], layer["zeros"], x_scales=s)
    h, y, _ = sptg.add_rms_norm(a, h, layer["norm2"], eps=EPS)
    rows, weight, offsets = route(sptg.gemm(y, layer["router"]), top)
    sorted_rows = y[rows]
    u = sptg.grouped_gemm(sorted_rows, layer["up"], offsets)
    act = torch.nn.functional.silu(u)
    d = sptg.grouped_gemm(act, layer["down"], offsets)
    out = torch.zeros(y.shape, dtype=torch.float32, device=y.device)
    out.index_add_(0, rows, d.float() * weight[:, None])
    return {"out": out.to(y.dtype), "residual": h, "y": y, "rows": rows, "weight": weight,
            "offsets": offsets, "sorted_rows": sorted_rows, "u": u, "act": act}


def expert_gradients(layer: dict, kept: dict, dout) -> dict:
    """Gradients of the experts' weights (float32) and of the rows that went into them."""
    offsets = kept["offsets"]
    dd = (dout[kept["rows"]].float() * kept["weight"][:, None]).to(dout.dtype)
    dact = sptg.grouped_gemm_dx(dd, layer["down"], offsets)
    sig = torch.sigmoid(kept["u"].float())
    du = (dact.float() * sig * (1 + kept["u"].float() * (1 - sig))).to(dout.dtype)
    return {"down": sptg.grouped_gemm_dw(dd, kept["act"], offsets, out_dtype=torch.float32),
            "up": sptg.grouped_gemm_dw(du, kept["sorted_rows"], offsets, out_dtype=torch.float32),
            "rows": sptg.grouped_gemm_dx(du, layer["up"], offsets)}


def plain_forward(layer: dict, x, residual, kept: dict):
    """The same step in float32, with the routing that `kept` chose."""
    def norm(t, w):
        return t * torch.rsqrt((t * t).mean(1, keepdim=True) + EPS) * w.float()

    n = layer["codes"].shape[0]
    codes = torch.stack([layer["codes"] & 15, layer["codes"] >> 4], 2).reshape(n, -1).float()
    w4 = ((codes - layer["zeros"].float().repeat_interleave(GROUP, 1))
          * layer["scales"].float().repeat_interleave(GROUP, 1))
    h = x.float() + residual.float()
    h = h + norm(h, layer["norm1"]) @ w4.t()
    y = norm(h, layer["norm2"])
    out = torch.zeros_like(y)
    offsets = kept["offsets"].tolist()
    for e in range(len(offsets) - 1):
        r = kept["rows"][offsets[e]:offsets[e + 1]]
        u = y[r] @ layer["up"][e].float().t()
        d = torch.nn.functional.silu(u) @ layer["down"][e].float().t()
        out.index_add_(0, r, d * kept["weight"][offsets[e]:offsets[e + 1], None])
    return out


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--rows", type=int, default=64)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inner", type=int, default=4096)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--top", type=int, default=2)
    a = ap.parse_args(argv)
    layer = make_layer(a.hidden, a.inner, a.experts)
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(a.rows, a.hidden, device="cuda", generator=g).bfloat16()
    residual = torch.randn(a.rows, a.hidden, device="cuda", generator=g).bfloat16()
    kept = forward(layer, x, residual, a.top)
    grads = expert_gradients(layer, kept, kept["out"])
    ref = plain_forward(layer, x, residual, kept)
    off = float((kept["out"].float() - ref).norm() / ref.norm())

    def ms(f, n=20):
        f()
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        start.record()
        for _ in range(n):
            f()
        end.record()
        torch.cuda.synchronize()
        return start.elapsed_time(end) / n

    t = {"step_ms": ms(lambda: forward(layer, x, residual, a.top)),
         "gradients_ms": ms(lambda: expert_gradients(layer, kept, kept["out"]))}
    assert sptg.device_error() == 0
    print(f"{a.rows} rows, hidden {a.hidden}, {a.experts} experts of {a.inner}, top {a.top}: "
          f"step {t['step_ms']:.3f} ms, gradients {t['gradients_ms']:.3f} ms, "
          f"distance from float32 {off:.4f}")
    return {"distance": off, "grads": grads, "kept": kept, "layer": layer, **t}


if __name__ == "__main__":
    main()
