"""Plain float64 references of the router and of the experts' e4m3 products,
written from their definitions with numpy and torch on the CPU."""
from __future__ import annotations

import math

import numpy as np
import torch

LOWEST = {torch.float32: -3.4028234663852886e38, torch.bfloat16: -3.3895313892515355e38}


def masked_logits(logits: torch.Tensor):
    """(float64 logits with +inf clamped, eligible) of one tensor [..., E]."""
    low = LOWEST[logits.dtype]
    l = logits.double().numpy().copy()
    ok = l > low  # false for NaN, -inf and the lowest value
    l = np.where(ok, np.minimum(l, -low), 0.0)
    return l, ok


def scores(logits: torch.Tensor, score: str):
    l, ok = masked_logits(logits)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-l))
        return np.where(ok, s, 0.0), ok
    m = np.where(ok, l, -np.inf).max(-1, keepdims=True)
    e = np.where(ok, np.exp(np.where(ok, l - np.where(np.isfinite(m), m, 0.0), -np.inf)), 0.0)
    total = e.sum(-1, keepdims=True)
    return np.where(total > 0, e / np.where(total > 0, total, 1.0), 0.0), ok


def route(logits: torch.Tensor, bias, K, score, G=1, topk_groups=1, group_top=1, renorm=True, scale=1.0):
    """(topk_idx [tokens, K], topk_w [tokens, K] float64) by plain loops."""
    E = logits.shape[-1]
    flat = logits.reshape(-1, E)
    s, ok = scores(flat, score)
    key = s + (0.0 if bias is None else bias.double().numpy())
    if score == "softmax" and bias is None and group_top == 1:
        key = masked_logits(flat)[0]  # same order, free of equal roundings
    with np.errstate(invalid="ignore"):
        ok = ok & (key > -np.inf)
    idx = np.full((flat.shape[0], K), -1, dtype=np.int64)
    w = np.zeros((flat.shape[0], K))
    per = E // G
    for t in range(flat.shape[0]):
        live = [e for e in range(E) if ok[t, e]]
        if topk_groups < G:
            best = []
            for g in range(G):
                ks = sorted((key[t, e] for e in live if e // per == g), reverse=True)[:group_top]
                if ks:
                    best.append((-sum(ks), g))
            kept = {g for _, g in sorted(best)[:topk_groups]}
            live = [e for e in live if e // per in kept]
        live.sort(key=lambda e: (-key[t, e], e))
        for k, e in enumerate(live[:K]):
            idx[t, k] = e
            w[t, k] = s[t, e]
        total = w[t].sum()
        if renorm:
            w[t] = w[t] / total if total > 0 else 0.0
    return idx, w * scale


def weights_of(l64: torch.Tensor, ok: torch.Tensor, idx: torch.Tensor, score, renorm, scale) -> torch.Tensor:
    """Differentiable float64 weights of the given slots (idx -1: weight 0)."""
    if score == "softmax":
        s = torch.softmax(torch.where(ok, l64, torch.full_like(l64, -math.inf)), -1)
    else:
        s = torch.sigmoid(l64)
    s = torch.where(ok, s, torch.zeros_like(s))
    w = torch.gather(s, -1, idx.clamp(min=0)) * (idx >= 0)
    if renorm:
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
    return w * scale


def route_backward(logits: torch.Tensor, idx: torch.Tensor, g: torch.Tensor, score, renorm, scale) -> torch.Tensor:
    l, ok = masked_logits(logits)
    l64 = torch.from_numpy(l).requires_grad_(True)
    ok = torch.from_numpy(ok)
    live = ok.any(-1, keepdim=True)
    w = weights_of(l64, ok | ~live, torch.where(live, idx, torch.full_like(idx, -1)), score, renorm, scale)
    (w * g.double()).sum().backward()
    return torch.where(ok, l64.grad, torch.zeros_like(l64.grad))


# ------------------------------------------------------------------ e4m3
def fp8(t: torch.Tensor) -> torch.Tensor:
    return t.view(torch.float8_e4m3fn).double()


def cast_blocks(x: torch.Tensor):
    """bf16 / fp32 [..., n] -> (e4m3 bytes, fp32 scales) with fp32 arithmetic, bit for bit."""
    n = x.shape[-1]
    q = torch.empty(x.shape, dtype=torch.uint8)
    scales = []
    for b in range(0, n, 128):
        v = x[..., b:b + 128].float()
        amax = torch.nan_to_num(v.abs(), nan=0.0, posinf=math.inf).amax(-1, keepdim=True)
        s = torch.clamp(amax, min=2.0 ** -100) / 448.0
        q[..., b:b + 128] = (v / s).to(torch.float8_e4m3fn).view(torch.uint8)
        scales.append(s)
    return q, torch.cat(scales, -1)


def expand(scales: torch.Tensor, n: int, dim: int) -> torch.Tensor:
    return scales.double().repeat_interleave(128, dim).narrow(dim, 0, n)


def product(a, a_scales, w, w_scales):
    """(a @ w^T, its sum of magnitudes) of one expert in float64 ([m, n] each)."""
    k = a.shape[-1]
    av = fp8(a) * expand(a_scales, k, -1)
    wv = fp8(w) * expand(expand(w_scales, w.shape[-2], -2), k, -1)
    return av @ wv.T, av.abs() @ wv.abs().T


def sum_error(k: int) -> float:
    """Bound of fp32 summation relative to the sum of magnitudes: 128 terms of a
    block in any order, the block products' scalings and their sum."""
    return (128 + -(-k // 128) + 4) * 2.0 ** -24
