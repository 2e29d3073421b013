"""Measured cases of the MoE layer's operators around the low-latency dispatch: the router
(``ep_route`` and its gradient), the dispatch that casts rows to e4m3 (``ep_ll_dispatch_fp8``)
and the experts' block-scaled e4m3 products (``ep_ll_gemm_swiglu_fp8``, ``ep_ll_gemm_fp8``).

``run`` computes each operator in its plain form (elementary torch operations in fp32, rounded
once at the end) where ``own`` is false, and through the library's entry points where it is true.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 128          # columns that share one scale
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100  # keeps the scale of an all-zero block a normal number
FP8 = torch.float8_e4m3fn


def _ceil(a: int, b: int) -> int:
    return -(-a // b)


# --------------------------------------------------------------------------- cases
def listed() -> list:
    return [
        # one decode step of 16 ranks, one token each: the smallest call, latency only
        dict(name="route_sigmoid_groups_token", op="route", R=16, T=1, E=256, K=8, dtype="fp32", score="sigmoid",
             bias=True, G=8, topk_groups=4, group_top=2, renorm=True, scale=2.5),
        # prefill workload: balance bias and groups, fp32 scores
        dict(name="route_sigmoid_groups_prefill", op="route", R=8, T=4096, E=256, K=8, dtype="fp32",
             score="sigmoid", bias=True, G=8, topk_groups=4, group_top=2, renorm=True, scale=2.5),
        # the largest workload of the dispatch benchmark, bf16 logits
        dict(name="route_softmax_large", op="route", R=32, T=16384, E=256, K=8, dtype="bf16", score="softmax",
             bias=False, G=1, topk_groups=1, group_top=1, renorm=True, scale=1.0),
        # training step, gradient dense over all experts (weights are plain softmax probabilities)
        dict(name="route_backward_softmax_skewed", op="route_backward", R=16, T=8192, E=256, K=8, dtype="fp32",
             score="softmax", renorm=False, scale=1.0),
        # training step of a small batch, sigmoid scores renormalised over the kept experts, bf16
        dict(name="route_backward_sigmoid_small", op="route_backward", R=16, T=128, E=256, K=8, dtype="bf16",
             score="sigmoid", renorm=True, scale=2.5),
        # low-latency workload: 2048 tokens to 256 experts
        dict(name="dispatch_fp8_low_latency", op="dispatch", R=16, T=128, H=7168, E=256, K=8, cap=128),
        # prefill workload: 32768 tokens to 256 experts
        dict(name="dispatch_fp8_prefill", op="dispatch", R=8, T=4096, H=7168, E=256, K=8, cap=1280),
        # one token decodes: eight experts of 32 have one row, the rest none; bound by their weights
        dict(name="swiglu_fp8_one_token", op="swiglu", E=32, tokens=1, K=8, cap=16, zipf=False, hidden=7168,
             ffn=2048),
        # low-latency workload, all 256 experts with about 64 rows each; bound by 7.5 GB of weights
        dict(name="swiglu_fp8_low_latency", op="swiglu", E=256, tokens=2048, K=8, cap=128, zipf=False, hidden=7168,
             ffn=2048),
        # 4096 tokens to 32 local experts, about 1024 rows each; bound by the tensor cores
        dict(name="swiglu_fp8_prefill", op="swiglu", E=32, tokens=4096, K=8, cap=1280, zipf=False, hidden=7168,
             ffn=2048),
        # down product of one rank's 16 experts in the low-latency workload: about 64 rows each
        dict(name="gemm_fp8_low_latency", op="gemm", E=16, tokens=128, K=8, cap=128, zipf=False, hidden=2048,
             out=7168),
        # down product with Zipf popularity: row counts from a few to thousands
        dict(name="gemm_fp8_skewed", op="gemm", E=32, tokens=4096, K=8, cap=4096, zipf=True, hidden=2048, out=7168),
    ]


def _log_int(rng, lo: int, hi: int) -> int:
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_ranks(rng, most_tokens: int):
    R = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16, 24, 32])
    return R, _log_int(rng, 1, max(1, most_tokens // R))


def draw(rng) -> dict:
    op = rng.choice(["route", "route_backward", "dispatch", "swiglu", "gemm"])
    if op in ("route", "route_backward"):
        R, T = _draw_ranks(rng, 262144)
        G = rng.choice([1, 2, 4, 8]) if op == "route" else 1
        E = R * G * _log_int(rng, 2, 16)
        score = rng.choice(["softmax", "sigmoid"])
        topk_groups = rng.randint(1, G)
        K = rng.randint(1, min(16, E // G * topk_groups))
        c = dict(op=op, R=R, T=T, E=E, K=K, dtype=rng.choice(["fp32", "bf16"]), score=score,
                 renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]))
        while R * c["T"] * E > 32 * 16384 * 256:  # no dearer than the largest listed one
            c["T"] = max(1, c["T"] // 2)
        if op == "route":
            c |= dict(bias=score == "sigmoid" and rng.random() < 0.7, G=G, topk_groups=topk_groups,
                      group_top=rng.choice([1, 2]) if score == "sigmoid" else 1)
        return c
    if op == "dispatch":
        R, T = _draw_ranks(rng, 32768)
        H = 16 * _log_int(rng, 8, 448)
        E = R * rng.randint(1, 256 // R)
        K = rng.randint(1, min(8, E))
        mean = R * T * K / E
        return dict(op=op, R=R, T=T, H=H, E=E, K=K, cap=8 * _ceil(int(mean + 6 * math.sqrt(mean) + 8), 8))
    E = _log_int(rng, 1, 64)
    K = rng.randint(1, min(8, E))
    tokens = _log_int(rng, 1, 4096)
    zipf = rng.random() < 0.3
    hidden = 16 * _log_int(rng, 16, 448)
    n = 16 * _log_int(rng, 8, 448)
    mean = tokens * K / E
    cap = 8 * _ceil(tokens if zipf else int(mean + 6 * math.sqrt(mean) + 8), 8)
    while E * cap * hidden * n > 64 * 2048 * 4096 * 2048:
        n = max(16, n // 2 // 16 * 16)
    if op == "swiglu":
        return dict(op=op, E=E, tokens=tokens, K=K, cap=cap, zipf=zipf, hidden=hidden, ffn=max(16, n // 32 * 16))
    return dict(op=op, E=E, tokens=tokens, K=K, cap=cap, zipf=zipf, hidden=hidden, out=n)


# --------------------------------------------------------------------------- inputs
def _dtype(name: str):
    return {"fp32": torch.float32, "bf16": torch.bfloat16}[name]


def _pick(g, tokens: int, E: int, K: int, zipf: bool) -> torch.Tensor:
    """K distinct experts for every token, in random order ([tokens, K] int64)."""
    keys = torch.rand(tokens, E, generator=g, device="cuda")
    if zipf:
        keys = -torch.log(-torch.log(keys.clamp(1e-12, 1 - 1e-7)))
        keys = keys - 1.2 * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    return torch.sort(keys, dim=1, descending=True).indices[:, :K].contiguous()


def _logits(g, c) -> torch.Tensor:
    # multiples of 2^-10: two scores are equal or clearly apart, whatever rounding an exp has
    x = torch.randn(c["R"], c["T"], c["E"], generator=g, device="cuda") * 1.5
    return (torch.round(x * 1024) / 1024).to(_dtype(c["dtype"]))


def _fp8_normal(g, *shape) -> torch.Tensor:
    """e4m3 bytes of normal values that use the type's range, as a cast by block maxima leaves them."""
    out = torch.empty(shape, dtype=torch.uint8, device="cuda")
    for part in out.split(max(1, (1 << 28) // max(1, math.prod(shape[1:])))):
        v = torch.randn(part.shape, generator=g, device="cuda") * 120.0
        part.copy_(v.clamp_(-E4M3_MAX, E4M3_MAX).to(FP8).view(torch.uint8))
    return out


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=c, status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if c["op"] in ("route", "route_backward"):
        R, T, E, K = c["R"], c["T"], c["E"], c["K"]
        s["logits"] = _logits(g, c)
        if c["op"] == "route":
            s["bias"] = torch.randn(E, generator=g, device="cuda") * 0.05 if c["bias"] else None
            s["topk_idx"] = torch.empty(R, T, K, dtype=torch.int64, device="cuda")
            s["topk_w"] = torch.empty(R, T, K, device="cuda")
        else:
            s["topk_idx"] = _pick(g, R * T, E, K, False).view(R, T, K)
            s["grad_topk_w"] = torch.randn(R, T, K, generator=g, device="cuda")
            s["grad_logits"] = torch.empty_like(s["logits"])
        return s
    if c["op"] == "dispatch":
        R, T, H, E, K, cap = c["R"], c["T"], c["H"], c["E"], c["K"], c["cap"]
        idx = _pick(g, R * T, E, K, False)
        flat = idx.reshape(-1)
        order = torch.sort(flat, stable=True).indices
        start = torch.cumsum(torch.bincount(flat, minlength=E), 0) - torch.bincount(flat, minlength=E)
        pos = torch.empty_like(flat)
        pos[order] = torch.arange(flat.numel(), device="cuda") - start[flat[order]]
        pos = torch.where(pos < cap, pos, -1)  # beyond the capacity: dropped by the layout
        # activations with a spread over tokens, as after a residual stream's norm
        x = torch.randn(R * T, H, generator=g, device="cuda")
        x *= torch.exp(torch.randn(R * T, 1, generator=g, device="cuda"))
        s["x"] = x.to(torch.bfloat16).view(R, T, H)
        s["topk_idx"] = idx.view(R, T, K)
        s["slot_pos"] = pos.to(torch.int32).view(R, T, K)
        s["recv_x"] = torch.zeros(E, cap, H, dtype=torch.uint8, device="cuda")
        s["recv_x_scales"] = torch.zeros(E, cap, _ceil(H, BLOCK), device="cuda")
        s["recv_src_info"] = torch.zeros(E, cap, 2, dtype=torch.int32, device="cuda")
        return s
    E, cap, H = c["E"], c["cap"], c["hidden"]
    idx = _pick(g, c["tokens"], E, c["K"], c["zipf"])
    s["count"] = torch.bincount(idx.reshape(-1), minlength=E).clamp(max=cap).to(torch.int32)
    s["a"] = _fp8_normal(g, E, cap, H)
    s["a_scales"] = torch.exp(torch.randn(E, cap, _ceil(H, BLOCK), generator=g, device="cuda") * 0.5) / 120
    if c["op"] == "swiglu":
        F = c["ffn"]
        s["w"] = _fp8_normal(g, E, 2, F, H)
        s["w_scales"] = torch.exp(
            torch.randn(E, 2, _ceil(F, BLOCK), _ceil(H, BLOCK), generator=g, device="cuda") * 0.3) / 120 / math.sqrt(H)
        s["y"] = torch.zeros(E, cap, F, dtype=torch.uint8, device="cuda")
        s["y_scales"] = torch.zeros(E, cap, _ceil(F, BLOCK), device="cuda")
    else:
        N = c["out"]
        s["w"] = _fp8_normal(g, E, N, H)
        s["w_scales"] = torch.exp(
            torch.randn(E, _ceil(N, BLOCK), _ceil(H, BLOCK), generator=g, device="cuda") * 0.3) / 120 / math.sqrt(H)
        s["y"] = torch.zeros(E, cap, N, dtype=torch.bfloat16, device="cuda")
    return s


# --------------------------------------------------------------------------- one pass
def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _plain_scores(c, logits):
    """(scores, eligible) in fp32: an infinite or lowest-value logit, or a NaN, masks its expert."""
    lim = torch.finfo(logits.dtype)
    eligible = logits > lim.min
    l = torch.where(eligible, logits.clamp(max=lim.max).float(), -math.inf)
    if c["score"] == "softmax":
        m = l.amax(-1, keepdim=True)
        e = torch.where(eligible, torch.exp(l - m), 0.0)
        s = e / e.sum(-1, keepdim=True)
        return torch.where(eligible, s, 0.0), eligible
    return torch.where(eligible, 1.0 / (1.0 + torch.exp(-l)), 0.0), eligible


def _plain_route(s):
    c = s["case"]
    R, T, E, K, G = c["R"], c["T"], c["E"], c["K"], c["G"]
    scores, eligible = _plain_scores(c, s["logits"])
    keys = scores if s["bias"] is None else scores + s["bias"]
    keys = torch.where(eligible, keys, -math.inf)
    if G > 1:
        best = torch.sort(keys.view(R, T, G, E // G), dim=-1, descending=True).values[..., :c["group_top"]]
        group = torch.where(best[..., 0] > -math.inf, torch.where(best > -math.inf, best, 0.0).sum(-1), -math.inf)
        order = torch.sort(group, dim=-1, descending=True, stable=True).indices[..., :c["topk_groups"]]
        keep = torch.zeros(R, T, G, dtype=torch.bool, device=keys.device).scatter_(-1, order, True)
        keys = torch.where(keep.unsqueeze(-1), keys.view(R, T, G, E // G), -math.inf).view(R, T, E)
    top = torch.sort(keys, dim=-1, descending=True, stable=True)
    idx, found = top.indices[..., :K], top.values[..., :K] > -math.inf
    w = torch.where(found, scores.gather(-1, idx), 0.0)
    if c["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return dict(topk_idx=torch.where(found, idx, -1), topk_w=w * c["scale"])


def _plain_route_backward(s):
    c = s["case"]
    idx, g = s["topk_idx"], s["grad_topk_w"]
    scores, _ = _plain_scores(c, s["logits"])
    valid = idx >= 0
    at = idx.clamp(min=0)
    kept = torch.where(valid, scores.gather(-1, at), 0.0)
    g = torch.where(valid, g, 0.0) * c["scale"]
    if c["renorm"]:
        total = kept.sum(-1, keepdim=True)
        v = kept / total
        g = torch.where(valid, (g - (g * v).sum(-1, keepdim=True)) / total, 0.0)
    ds = torch.zeros_like(scores).scatter_add_(-1, at, g)
    if c["score"] == "softmax":
        d = scores * (ds - (kept * g).sum(-1, keepdim=True))
    else:
        d = scores * (1.0 - scores) * ds
    return dict(grad_logits=d.to(s["logits"].dtype))


def _plain_cast(x):
    """fp32 [..., n] -> (e4m3 [..., n], scales [..., ceil(n / 128)])."""
    n = x.shape[-1]
    pad = torch.nn.functional.pad(x, (0, -n % BLOCK)).unflatten(-1, (-1, BLOCK))
    scale = pad.abs().amax(-1).clamp(min=AMAX_FLOOR) / E4M3_MAX
    return (pad / scale.unsqueeze(-1)).flatten(-2)[..., :n].to(FP8), scale


def _plain_dispatch(s):
    c = s["case"]
    R, T, H, K = c["R"], c["T"], c["H"], c["K"]
    q, scale = _plain_cast(s["x"].view(R * T, H).float())
    slot = (s["slot_pos"].view(-1) >= 0).nonzero().squeeze(-1)
    e, row = s["topk_idx"].view(-1)[slot], s["slot_pos"].view(-1)[slot].long()
    token = slot // K
    s["recv_x"][e, row] = q.view(torch.uint8)[token]
    s["recv_x_scales"][e, row] = scale[token]
    s["recv_src_info"][e, row] = torch.stack([token // T, token % T], -1).to(torch.int32)
    return dict(recv_x=s["recv_x"].view(FP8), recv_x_scales=s["recv_x_scales"], recv_src_info=s["recv_src_info"])


def _plain_weights(w, scales):
    """e4m3 bytes [..., N, K] with one scale per 128x128 block -> fp32."""
    N, K = w.shape[-2:]
    full = scales.repeat_interleave(BLOCK, -2)[..., :N, :].repeat_interleave(BLOCK, -1)[..., :K]
    return w.view(FP8).float().mul_(full)


def _plain_rows(s):
    K = s["a"].shape[-1]
    return s["a"].view(FP8).float().mul_(s["a_scales"].repeat_interleave(BLOCK, -1)[..., :K])


def _plain_valid(s):
    return (torch.arange(s["case"]["cap"], device="cuda") < s["count"].unsqueeze(-1)).unsqueeze(-1)


def _plain_gemm(s):
    y = torch.bmm(_plain_rows(s), _plain_weights(s["w"], s["w_scales"]).transpose(1, 2))
    return dict(y=torch.where(_plain_valid(s), y, 0.0).to(torch.bfloat16))


def _plain_swiglu(s):
    c = s["case"]
    w = _plain_weights(s["w"], s["w_scales"]).view(c["E"], 2 * c["ffn"], c["hidden"])
    gate, up = torch.bmm(_plain_rows(s), w.transpose(1, 2)).chunk(2, -1)
    q, scale = _plain_cast(gate / (1.0 + torch.exp(-gate)) * up)
    valid = _plain_valid(s)
    return dict(y=torch.where(valid, q.view(torch.uint8), 0).view(FP8), y_scales=torch.where(valid, scale, 0.0))


_plain = dict(route=_plain_route, route_backward=_plain_route_backward, dispatch=_plain_dispatch, gemm=_plain_gemm,
              swiglu=_plain_swiglu)


def _shape(ep, c):
    return ep.EpShape.make(c["R"], c["T"], c["K"], c["E"], c.get("H", 8), 1)


def _own_route(s):
    from combine_get_dispatch_notify_gb300 import ep
    c = s["case"]
    cfg = ep.EpRoute.make(c["score"], c["G"], c["topk_groups"], c["group_top"], c["renorm"], c["scale"])
    ep.ep_route(_shape(ep, c), cfg, s["logits"], s["bias"], s["topk_idx"], s["topk_w"], s["status"])
    return dict(topk_idx=s["topk_idx"], topk_w=s["topk_w"])


def _own_route_backward(s):
    from combine_get_dispatch_notify_gb300 import ep
    c = s["case"]
    cfg = ep.EpRoute.make(c["score"], renormalize=c["renorm"], scale=c["scale"])
    ep.ep_route_backward(_shape(ep, c), cfg, s["logits"], s["topk_idx"], s["grad_topk_w"], s["grad_logits"],
                         s["status"])
    return dict(grad_logits=s["grad_logits"])


def _own_dispatch(s):
    from combine_get_dispatch_notify_gb300 import ep
    c = s["case"]
    ep.ep_ll_dispatch_fp8(_shape(ep, c), s["x"], s["topk_idx"], s["slot_pos"], c["cap"], s["recv_x"],
                          s["recv_x_scales"], s["recv_src_info"], s["status"])
    return dict(recv_x=s["recv_x"].view(FP8), recv_x_scales=s["recv_x_scales"], recv_src_info=s["recv_src_info"])


def _own_gemm(s):
    from combine_get_dispatch_notify_gb300 import ep
    ep.ep_ll_gemm_fp8(s["a"], s["a_scales"], s["w"], s["w_scales"], s["count"], s["y"], s["status"])
    return dict(y=s["y"])


def _own_swiglu(s):
    from combine_get_dispatch_notify_gb300 import ep
    ep.ep_ll_gemm_swiglu_fp8(s["a"], s["a_scales"], s["w"], s["w_scales"], s["count"], s["y"], s["y_scales"],
                             s["status"])
    return dict(y=s["y"].view(FP8), y_scales=s["y_scales"])


_own = dict(route=_own_route, route_backward=_own_route_backward, dispatch=_own_dispatch, gemm=_own_gemm,
            swiglu=_own_swiglu)


# --------------------------------------------------------------------------- what a pass cannot do without
def work(case) -> dict:
    c = case
    if c["op"] in ("route", "route_backward"):
        tokens, E, K = c["R"] * c["T"], c["E"], c["K"]
        b = 4 if c["dtype"] == "fp32" else 2
        if c["op"] == "route":
            return dict(bytes=tokens * (E * b + 12 * K) + (4 * E if c["bias"] else 0), flops=tokens * E * 8)
        dense = c["score"] == "softmax" and not c["renorm"]
        return dict(bytes=tokens * ((2 * E if dense else E + K) * b + 12 * K), flops=tokens * (E if dense else K) * 8)
    if c["op"] == "dispatch":
        tokens, H, K = c["R"] * c["T"], c["H"], c["K"]
        return dict(bytes=tokens * (2 * H + 12 * K) + tokens * K * (H + 4 * _ceil(H, BLOCK) + 8),
                    flops=tokens * H * 3)
    E, H, rows = c["E"], c["hidden"], c["tokens"] * c["K"]
    # experts that have a row: all but those that every token passes by
    active = _active(E, c["K"], c["tokens"], c["zipf"])
    if c["op"] == "swiglu":
        N, out = 2 * c["ffn"], c["ffn"] + 4 * _ceil(c["ffn"], BLOCK)
        blocks = 2 * _ceil(c["ffn"], BLOCK)
    else:
        N, out, blocks = c["out"], 2 * c["out"], _ceil(c["out"], BLOCK)
    return dict(bytes=active * (N * H + 4 * blocks * _ceil(H, BLOCK)) + rows * (H + 4 * _ceil(H, BLOCK) + out) + 4 * E,
                flops=2 * rows * N * H)


def _active(E: int, K: int, tokens: int, zipf: bool) -> float:
    share = [1.0 / E] * E
    if zipf:
        total = sum((e + 1) ** -1.2 for e in range(E))
        share = [(e + 1) ** -1.2 / total for e in range(E)]
    return sum(1.0 - (1.0 - min(1.0, K * p)) ** tokens for p in share)


# --------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    c = dict(case)
    s = prepare(case, seed)
    return dict(route=_exact_route, route_backward=_exact_route_backward, dispatch=_exact_dispatch, gemm=_exact_gemm,
                swiglu=_exact_swiglu)[c["op"]](c, s)


def _exact_route(c, s):
    R, T, E, K, G = c["R"], c["T"], c["E"], c["K"], c["G"]
    out_idx = torch.empty(R * T, K, dtype=torch.int64, device="cuda")
    out_w = torch.empty(R * T, K, dtype=torch.float64, device="cuda")
    for lo in range(0, R * T, 65536):
        l = s["logits"].view(R * T, E)[lo:lo + 65536].double()
        p = torch.softmax(l, -1) if c["score"] == "softmax" else torch.sigmoid(l)
        key = p.clone() if s["bias"] is None else p + s["bias"].double()
        if G > 1:
            per = key.view(-1, G, E // G)
            group = torch.topk(per, min(c["group_top"], E // G), dim=-1).values.sum(-1)
            rank = (group.unsqueeze(1) > group.unsqueeze(2)).sum(-1)  # groups above each one
            tie = (group.unsqueeze(1) == group.unsqueeze(2)).tril(-1).sum(-1)
            per[(rank + tie) >= c["topk_groups"]] = -math.inf
        idx = torch.argsort(key, dim=-1, descending=True, stable=True)[:, :K]
        w = torch.gather(p, 1, idx)
        if c["renorm"]:
            w = w / w.sum(-1, keepdim=True)
        out_idx[lo:lo + 65536], out_w[lo:lo + 65536] = idx, w * c["scale"]
    return dict(topk_idx=None, topk_w=out_w.view(R, T, K))


def _exact_route_backward(c, s):
    E, K = c["E"], c["K"]
    rows = c["R"] * c["T"]
    out = torch.empty(rows, E, dtype=torch.float64, device="cuda")
    for lo in range(0, rows, 65536):
        l = s["logits"].view(rows, E)[lo:lo + 65536].double().requires_grad_(True)
        p = torch.softmax(l, -1) if c["score"] == "softmax" else torch.sigmoid(l)
        w = torch.gather(p, 1, s["topk_idx"].view(rows, K)[lo:lo + 65536])
        if c["renorm"]:
            w = w / w.sum(-1, keepdim=True)
        (w * c["scale"] * s["grad_topk_w"].view(rows, K)[lo:lo + 65536].double()).sum().backward()
        out[lo:lo + 65536] = l.grad
    return dict(grad_logits=out.view(c["R"], c["T"], E))


def _exact_cast(x):
    """float64 [m, n] -> (values on the e4m3 grid, scales), by the grid's spacing at each value."""
    m, n = x.shape
    blocks = _ceil(n, BLOCK)
    scale = torch.empty(m, blocks, dtype=torch.float64, device=x.device)
    q = torch.empty_like(x)
    for b in range(blocks):
        v = x[:, b * BLOCK:(b + 1) * BLOCK]
        scale[:, b] = v.abs().amax(1).clamp(min=AMAX_FLOOR) / E4M3_MAX
        v = v / scale[:, b:b + 1]
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        q[:, b * BLOCK:(b + 1) * BLOCK] = torch.round(v / step) * step
    return q, scale


def _exact_dispatch(c, s):
    R, T, H, E, K, cap = c["R"], c["T"], c["H"], c["E"], c["K"], c["cap"]
    if E * cap * H > 6e9:
        return None
    q, scale = _exact_cast(s["x"].view(R * T, H).double())
    rq = torch.zeros(E * cap, H, dtype=torch.float64, device="cuda")
    rs = torch.zeros(E * cap, scale.shape[1], dtype=torch.float64, device="cuda")
    pos = s["slot_pos"].view(R * T, K)
    for k in range(K):
        ok = pos[:, k] >= 0
        to = (s["topk_idx"].view(R * T, K)[:, k] * cap + pos[:, k])[ok]
        rq[to], rs[to] = q[ok], scale[ok]
    return dict(recv_x=rq.view(E, cap, H), recv_x_scales=rs.view(E, cap, -1), recv_src_info=None)


def _exact_products(c, s):
    """For every expert with rows: (expert, rows, product of its rows and weights in float64 [rows, N])."""
    H = c["hidden"]
    col = torch.arange(H, device="cuda") // BLOCK
    for e, m in enumerate(s["count"].tolist()):
        if m == 0:
            continue
        a = s["a"][e, :m].view(FP8).double() * s["a_scales"][e, :m].double()[:, col]
        parts = s["w"][e].view(-1, s["w"].shape[-2], H)
        scales = s["w_scales"][e].view(parts.shape[0], -1, s["w_scales"].shape[-1])
        row = torch.arange(parts.shape[1], device="cuda") // BLOCK
        yield e, m, [a @ (w.view(FP8).double() * v.double()[row][:, col]).T for w, v in zip(parts, scales)]


def _exact_gemm(c, s):
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    for e, m, (p,) in _exact_products(c, s):
        y[e, :m] = p
    return dict(y=y)


def _exact_swiglu(c, s):
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    ys = torch.zeros(s["y_scales"].shape, dtype=torch.float64, device="cuda")
    for e, m, (gate, up) in _exact_products(c, s):
        y[e, :m], ys[e, :m] = _exact_cast(gate * torch.sigmoid(gate) * up)
    return dict(y=y, y_scales=ys)
