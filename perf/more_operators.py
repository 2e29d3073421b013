"""Measured cases of what trains an expert layer in bf16 and serves it in int8, on the per-expert
packed (low-latency) layout: the gated feed-forward block of the experts and its backward pass
(``ep_ll_gemm_swiglu_bf16``, ``ep_ll_gemm_bf16``, ``ep_ll_gemm_dswiglu_bf16``,
``ep_ll_gemm_dgrad_bf16``, ``ep_ll_gemm_wgrad_bf16``), the gradient of the weighted combine
(``ep_ll_combine_backward``), the dispatch that casts rows to int8 (``ep_ll_dispatch_int8``) and
the block's int8 products with a scale for each token and channel (``ep_ll_gemm_swiglu_int8``,
``ep_ll_gemm_int8``).

``run`` computes each operator in its plain form (elementary torch operations in fp32, each of its
outputs rounded once) where ``own`` is false, and through the library's entry points where it is true.
"""
from __future__ import annotations

import math

import torch

own = False

INT8_MAX = 127.0
AMAX_FLOOR = 2.0 ** -100  # keeps the scale of an all-zero row a normal number


def _ceil(a: int, b: int) -> int:
    return -(-a // b)


# --------------------------------------------------------------------------- cases
def listed() -> list:
    return [
        # one token decodes with bf16 weights: eight of 32 experts have one row; bound by their weights
        dict(name="ffn_one_token", op="ffn", E=32, tokens=1, K=8, cap=16, zipf=False, hidden=7168, ffn=2048,
             train=False),
        # training step's forward pass, about 1024 rows to each of 32 experts, both projections kept for the gradient
        dict(name="ffn_train", op="ffn", E=32, tokens=4096, K=8, cap=1280, zipf=False, hidden=7168, ffn=2048,
             train=True),
        # backward pass of a small layer with odd sizes and Zipf popularity: from no row to hundreds
        dict(name="ffn_backward_small", op="ffn_backward", E=24, tokens=300, K=3, cap=304, zipf=True, hidden=1160,
             ffn=520, part="all"),
        # backward pass of the training step above
        dict(name="ffn_backward_train", op="ffn_backward", E=32, tokens=4096, K=8, cap=1280, zipf=False, hidden=7168,
             ffn=2048, part="all"),
        # a schedule that puts the weights' gradients off until the rows' ones are sent: only they, in fp32, from the
        # projections' gradients that were kept
        dict(name="ffn_backward_weights", op="ffn_backward", E=32, tokens=2048, K=8, cap=640, zipf=False, hidden=7168,
             ffn=2048, part="weights"),
        # gradient of the combine: low-latency workload, 2048 tokens of 256 experts
        dict(name="combine_backward_low_latency", op="combine_backward", R=16, T=128, H=7168, E=256, K=8, cap=128),
        # training step of 32768 tokens
        dict(name="combine_backward_prefill", op="combine_backward", R=8, T=4096, H=7168, E=256, K=8, cap=1280),
        # the same two workloads' tokens on their way to int8 experts
        dict(name="dispatch_int8_low_latency", op="dispatch_int8", R=16, T=128, H=7168, E=256, K=8, cap=128),
        dict(name="dispatch_int8_prefill", op="dispatch_int8", R=8, T=4096, H=7168, E=256, K=8, cap=1280),
        # one token decodes with int8 weights
        dict(name="ffn_int8_one_token", op="ffn_int8", E=32, tokens=1, K=8, cap=16, zipf=False, hidden=7168, ffn=2048),
        # 64 experts with about 64 rows each; bound by 2.8 GB of weights
        dict(name="ffn_int8_low_latency", op="ffn_int8", E=64, tokens=512, K=8, cap=128, zipf=False, hidden=7168,
             ffn=2048),
        # 4096 tokens to 32 experts, about 1024 rows each; bound by the tensor cores
        dict(name="ffn_int8_prefill", op="ffn_int8", E=32, tokens=4096, K=8, cap=1280, zipf=False, hidden=7168,
             ffn=2048),
    ]


def _log_int(rng, lo: int, hi: int) -> int:
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng) -> dict:
    op = rng.choice(["ffn", "ffn_backward", "combine_backward", "dispatch_int8", "ffn_int8"])
    if op in ("combine_backward", "dispatch_int8"):
        R = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16, 24, 32])
        T = _log_int(rng, 1, max(1, 32768 // R))
        H = 8 * _log_int(rng, 8, 896) if op == "combine_backward" else 16 * _log_int(rng, 4, 448)
        E = R * rng.randint(1, 256 // R)
        K = rng.randint(1, min(8, E))
        mean = R * T * K / E
        return dict(op=op, R=R, T=T, H=H, E=E, K=K, cap=8 * _ceil(int(mean + 6 * math.sqrt(mean) + 8), 8))
    E = _log_int(rng, 1, 64)
    K = rng.randint(1, min(8, E))
    tokens = _log_int(rng, 1, 4096)
    zipf = rng.random() < 0.3
    unit = 16 if op == "ffn_int8" else 8
    hidden = unit * _log_int(rng, 128 // unit, 7168 // unit)
    ffn = unit * _log_int(rng, 64 // unit, 2048 // unit)
    mean = tokens * K / E
    cap = 8 * _ceil(tokens if zipf else int(mean + 6 * math.sqrt(mean) + 8), 8)
    while E * cap * hidden * ffn > 40960 * 7168 * 2048:  # no dearer than the largest listed one
        ffn = max(unit, ffn // 2 // unit * unit)
        if ffn == unit:
            break
    c = dict(op=op, E=E, tokens=tokens, K=K, cap=cap, zipf=zipf, hidden=hidden, ffn=ffn)
    if op == "ffn":
        c["train"] = rng.random() < 0.5
    elif op == "ffn_backward":
        c["part"] = rng.choice(["all", "weights"])
    return c


# --------------------------------------------------------------------------- inputs
def _pick(g, tokens: int, E: int, K: int, zipf: bool) -> torch.Tensor:
    """K distinct experts for every token, in random order ([tokens, K] int64)."""
    keys = torch.rand(tokens, E, generator=g, device="cuda")
    if zipf:
        keys = -torch.log(-torch.log(keys.clamp(1e-12, 1 - 1e-7)))
        keys = keys - 1.2 * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    return torch.sort(keys, dim=1, descending=True).indices[:, :K].contiguous()


def _normal(g, scale: float, *shape) -> torch.Tensor:
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for part in out.split(max(1, (1 << 28) // max(1, math.prod(shape[1:])))):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * scale)
    return out


def _int8_normal(g, *shape) -> torch.Tensor:
    """int8 of normal values that use the type's range, as a cast by a row's maximum leaves them."""
    out = torch.empty(shape, dtype=torch.int8, device="cuda")
    for part in out.split(max(1, (1 << 28) // max(1, math.prod(shape[1:])))):
        part.copy_((torch.randn(part.shape, generator=g, device="cuda") * 32.0).round_().clamp_(-INT8_MAX, INT8_MAX))
    return out


def _slots(g, c):
    """(topk_idx, slot_pos): every slot's expert and its row there, -1 beyond the capacity."""
    R, T, E, K, cap = c["R"], c["T"], c["E"], c["K"], c["cap"]
    idx = _pick(g, R * T, E, K, False)
    flat = idx.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    count = torch.bincount(flat, minlength=E)
    start = torch.cumsum(count, 0) - count
    pos = torch.empty_like(flat)
    pos[order] = torch.arange(flat.numel(), device="cuda") - start[flat[order]]
    pos = torch.where(pos < cap, pos, -1)
    return idx.view(R, T, K), pos.to(torch.int32).view(R, T, K)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=c, status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    zeros = lambda dt, *shape: torch.zeros(shape, dtype=dt, device="cuda")  # noqa: E731
    bf16, fp32 = torch.bfloat16, torch.float32
    if c["op"] in ("combine_backward", "dispatch_int8"):
        R, T, H, E, K, cap = c["R"], c["T"], c["H"], c["E"], c["K"], c["cap"]
        s["topk_idx"], s["slot_pos"] = _slots(g, c)
        if c["op"] == "dispatch_int8":
            # activations with a spread over tokens, as after a residual stream's norm
            x = torch.randn(R * T, H, generator=g, device="cuda")
            x *= torch.exp(torch.randn(R * T, 1, generator=g, device="cuda"))
            s["x"] = x.to(bf16).view(R, T, H)
            s["recv_x"], s["recv_x_scales"] = zeros(torch.int8, E, cap, H), zeros(fp32, E, cap)
            s["recv_src_info"] = zeros(torch.int32, E, cap, 2)
        else:
            s["grad"] = _normal(g, 1e-3, R * T, H).view(R, T, H)
            s["y"] = _normal(g, 1.0, E, cap, H)
            w = torch.rand(R, T, K, generator=g, device="cuda") + 0.05
            s["topk_w"] = w / w.sum(-1, keepdim=True)
            s["grad_y"], s["grad_topk_w"] = zeros(bf16, E, cap, H), zeros(fp32, R, T, K)
        return s
    E, cap, H, F = c["E"], c["cap"], c["hidden"], c["ffn"]
    idx = _pick(g, c["tokens"], E, c["K"], c["zipf"])
    s["count"] = torch.bincount(idx.reshape(-1), minlength=E).clamp(max=cap).to(torch.int32)
    if c["op"] == "ffn_int8":
        s["a"], s["w13"], s["w2"] = _int8_normal(g, E, cap, H), _int8_normal(g, E, 2, F, H), _int8_normal(g, E, H, F)
        near = lambda *shape: torch.exp(torch.randn(shape, generator=g, device="cuda") * 0.3) / 32  # noqa: E731
        s["a_scales"], s["w13_scales"] = near(E, cap), near(E, 2, F) / math.sqrt(H)
        s["w2_scales"] = near(E, H) / math.sqrt(F)
        s["inner"], s["inner_scales"] = zeros(torch.int8, E, cap, F), zeros(fp32, E, cap)
        s["workspace"] = torch.empty(E * cap * F * 4, dtype=torch.uint8, device="cuda")
        s["y"] = zeros(bf16, E, cap, H)
        return s
    # the rows behind an expert's count are what an earlier step left there
    s["a"] = _normal(g, 1.0, E, cap, H)
    s["w13"], s["w2"] = _normal(g, H ** -0.5, E, 2, F, H), _normal(g, F ** -0.5, E, H, F)
    if c["op"] == "ffn":
        s["inner"], s["y"] = zeros(bf16, E, cap, F), zeros(bf16, E, cap, H)
        s["gate_up"] = zeros(bf16, E, cap, 2, F) if c["train"] else None
        return s
    s["gate_up"] = _normal(g, 1.0, E, cap, 2, F)
    s["inner"] = torch.empty(E, cap, F, dtype=bf16, device="cuda")
    for e in range(E):  # as the forward pass leaves it
        gate, up = s["gate_up"][e].float().unbind(1)
        s["inner"][e] = gate / (1.0 + torch.exp(-gate)) * up
    s["grad_y"] = _normal(g, 1e-3, E, cap, H)
    if c["part"] == "weights":
        gt = fp32
        s["grad_gate_up"] = _normal(g, 1e-3, E, cap, 2, F)
    else:
        gt = bf16
        s["grad_gate_up"], s["grad_a"] = zeros(bf16, E, cap, 2, F), zeros(bf16, E, cap, H)
    s["grad_w13"], s["grad_w2"] = zeros(gt, E, 2, F, H), zeros(gt, E, H, F)
    return s


# --------------------------------------------------------------------------- one pass
def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _plain_valid(s):
    return (torch.arange(s["case"]["cap"], device="cuda") < s["count"].unsqueeze(-1)).unsqueeze(-1)


def _plain_ffn(s):
    c = s["case"]
    E, cap, H, F = c["E"], c["cap"], c["hidden"], c["ffn"]
    valid = _plain_valid(s)
    a = torch.where(valid, s["a"].float(), 0.0)
    p = torch.bmm(a, s["w13"].float().view(E, 2 * F, H).transpose(1, 2))
    gate, up = p[..., :F], p[..., F:]
    inner = (gate / (1.0 + torch.exp(-gate)) * up).to(torch.bfloat16)
    y = torch.bmm(inner.float(), s["w2"].float().transpose(1, 2)).to(torch.bfloat16)
    out = dict(y=y, inner=inner)
    if c["train"]:
        out["gate_up"] = p.to(torch.bfloat16).view(E, cap, 2, F)
    return out


def _plain_ffn_backward(s):
    c = s["case"]
    E, cap, H, F = c["E"], c["cap"], c["hidden"], c["ffn"]
    valid = _plain_valid(s)
    live = lambda t: torch.where(valid, t.float(), 0.0)  # noqa: E731
    gy = live(s["grad_y"])
    out = {}
    if c["part"] == "weights":
        g = live(s["grad_gate_up"].view(E, cap, 2 * F))
    else:
        gh = torch.bmm(gy, s["w2"].float())
        gate, up = live(s["gate_up"].view(E, cap, 2 * F)).split(F, -1)
        sig = 1.0 / (1.0 + torch.exp(-gate))
        gate_grad = gh * up * sig * (1.0 + gate * (1.0 - sig))
        ggu = torch.cat([gate_grad, gh * gate * sig], -1).to(torch.bfloat16)
        g = ggu.float()
        out["grad_gate_up"] = ggu.view(E, cap, 2, F)
        out["grad_a"] = torch.bmm(g, s["w13"].float().view(E, 2 * F, H)).to(torch.bfloat16)
    gt = s["grad_w2"].dtype
    out["grad_w13"] = torch.bmm(g.transpose(1, 2), live(s["a"])).to(gt).view(E, 2, F, H)
    out["grad_w2"] = torch.bmm(gy.transpose(1, 2), live(s["inner"])).to(gt)
    return out


def _plain_combine_backward(s):
    c = s["case"]
    R, T, H, K = c["R"], c["T"], c["H"], c["K"]
    pos = s["slot_pos"].view(-1)
    slot = (pos >= 0).nonzero().squeeze(-1)
    e, row, token = s["topk_idx"].view(-1)[slot], pos[slot].long(), slot // K
    w, grad = s["topk_w"].view(-1), s["grad"].view(R * T, H)
    grad_w = torch.zeros(R * T * K, device="cuda")
    for part in slot.split(1 << 16):
        lo = int(part.numel())
        i = slice(0, lo)
        e_, row_, t_ = e[i], row[i], token[i]
        e, row, token = e[lo:], row[lo:], token[lo:]
        g = grad[t_].float()
        grad_w[part] = (g * s["y"][e_, row_].float()).sum(-1)
        s["grad_y"][e_, row_] = (g * w[part].unsqueeze(-1)).to(torch.bfloat16)
    return dict(grad_y=s["grad_y"], grad_topk_w=grad_w.view(R, T, K))


def _plain_cast(x):
    """fp32 [..., n] -> (whole numbers in [-127, 127], one scale for each row)."""
    scale = x.abs().amax(-1).clamp(min=AMAX_FLOOR) / INT8_MAX
    return torch.round(x / scale.unsqueeze(-1)), scale


def _plain_dispatch_int8(s):
    c = s["case"]
    R, T, H, K = c["R"], c["T"], c["H"], c["K"]
    q, scale = _plain_cast(s["x"].view(R * T, H).float())
    pos = s["slot_pos"].view(-1)
    slot = (pos >= 0).nonzero().squeeze(-1)
    e, row, token = s["topk_idx"].view(-1)[slot], pos[slot].long(), slot // K
    s["recv_x"][e, row] = q.to(torch.int8)[token]
    s["recv_x_scales"][e, row] = scale[token]
    s["recv_src_info"][e, row] = torch.stack([token // T, token % T], -1).to(torch.int32)
    # whole numbers: cast and quotient are fp32's own on both sides
    return dict(recv_x=s["recv_x"], recv_x_scales=s["recv_x_scales"], recv_src_info=s["recv_src_info"])


def _plain_ffn_int8(s):
    c = s["case"]
    E, H, F = c["E"], c["hidden"], c["ffn"]
    valid = _plain_valid(s)
    p = torch.bmm(s["a"].float(), s["w13"].float().view(E, 2 * F, H).transpose(1, 2))
    p = p * s["a_scales"].unsqueeze(-1) * s["w13_scales"].view(E, 1, 2 * F)
    gate, up = torch.where(valid, p, 0.0).split(F, -1)
    q, scale = _plain_cast(gate / (1.0 + torch.exp(-gate)) * up)
    y = torch.bmm(q, s["w2"].float().transpose(1, 2)) * scale.unsqueeze(-1) * s["w2_scales"].unsqueeze(1)
    return dict(y=torch.where(valid, y, 0.0).to(torch.bfloat16),
                inner_scales=torch.where(valid.squeeze(-1), scale, 0.0))


_plain = dict(ffn=_plain_ffn, ffn_backward=_plain_ffn_backward, combine_backward=_plain_combine_backward,
              dispatch_int8=_plain_dispatch_int8, ffn_int8=_plain_ffn_int8)


def _own_ffn(s):
    from combine_get_dispatch_notify_gb300 import ep
    ep.ep_ll_gemm_swiglu_bf16(s["a"], s["w13"], s["count"], s["inner"], s["gate_up"], s["status"])
    ep.ep_ll_gemm_bf16(s["inner"], s["w2"], s["count"], s["y"], s["status"])
    out = dict(y=s["y"], inner=s["inner"])
    if s["gate_up"] is not None:
        out["gate_up"] = s["gate_up"]
    return out


def _own_ffn_backward(s):
    from combine_get_dispatch_notify_gb300 import ep
    c = s["case"]
    E, cap, H, F = c["E"], c["cap"], c["hidden"], c["ffn"]
    count, st = s["count"], s["status"]
    ggu = s["grad_gate_up"].view(E, cap, 2 * F)
    out = {}
    if c["part"] == "all":
        ep.ep_ll_gemm_dswiglu_bf16(s["grad_y"], s["w2"], s["gate_up"], count, s["grad_gate_up"], st)
        ep.ep_ll_gemm_dgrad_bf16(ggu, s["w13"].view(E, 2 * F, H), count, s["grad_a"], st)
        out = dict(grad_gate_up=s["grad_gate_up"], grad_a=s["grad_a"])
    ep.ep_ll_gemm_wgrad_bf16(ggu, s["a"], count, s["grad_w13"].view(E, 2 * F, H), st)
    ep.ep_ll_gemm_wgrad_bf16(s["grad_y"], s["inner"], count, s["grad_w2"], st)
    return dict(out, grad_w13=s["grad_w13"], grad_w2=s["grad_w2"])


def _shape(ep, c):
    return ep.EpShape.make(c["R"], c["T"], c["K"], c["E"], c["H"], 1)


def _own_combine_backward(s):
    from combine_get_dispatch_notify_gb300 import ep
    c = s["case"]
    ep.ep_ll_combine_backward(_shape(ep, c), s["grad"], s["y"], c["cap"], s["topk_idx"], s["topk_w"], s["slot_pos"],
                              s["grad_y"], s["grad_topk_w"], s["status"])
    return dict(grad_y=s["grad_y"], grad_topk_w=s["grad_topk_w"])


def _own_dispatch_int8(s):
    from combine_get_dispatch_notify_gb300 import ep
    c = s["case"]
    ep.ep_ll_dispatch_int8(_shape(ep, c), s["x"], s["topk_idx"], s["slot_pos"], c["cap"], s["recv_x"],
                           s["recv_x_scales"], s["recv_src_info"], s["status"])
    return dict(recv_x=s["recv_x"], recv_x_scales=s["recv_x_scales"], recv_src_info=s["recv_src_info"])


def _own_ffn_int8(s):
    from combine_get_dispatch_notify_gb300 import ep
    ep.ep_ll_gemm_swiglu_int8(s["a"], s["a_scales"], s["w13"], s["w13_scales"], s["count"], s["inner"],
                              s["inner_scales"], s["workspace"], s["status"])
    ep.ep_ll_gemm_int8(s["inner"], s["inner_scales"], s["w2"], s["w2_scales"], s["count"], s["y"], s["status"])
    return dict(y=s["y"], inner_scales=s["inner_scales"])


_own = dict(ffn=_own_ffn, ffn_backward=_own_ffn_backward, combine_backward=_own_combine_backward,
            dispatch_int8=_own_dispatch_int8, ffn_int8=_own_ffn_int8)


# --------------------------------------------------------------------------- what a pass cannot do without
def work(case) -> dict:
    c = case
    if c["op"] in ("combine_backward", "dispatch_int8"):
        tokens, H, K = c["R"] * c["T"], c["H"], c["K"]
        if c["op"] == "dispatch_int8":
            return dict(bytes=tokens * (2 * H + 12 * K) + tokens * K * (H + 12), flops=tokens * H * 3)
        return dict(bytes=tokens * (2 * H + 20 * K) + tokens * K * 4 * H, flops=tokens * K * H * 3)
    E, H, F, rows = c["E"], c["hidden"], c["ffn"], c["tokens"] * c["K"]
    active = _active(E, c["K"], c["tokens"], c["zipf"])  # experts that have a row
    flops = 2 * rows * 3 * F * H
    if c["op"] == "ffn_int8":
        return dict(bytes=active * (3 * F * H + 4 * (2 * F + H)) + rows * (H + 4 + 2 * H) + 4 * E, flops=flops)
    if c["op"] == "ffn":
        kept = 6 * F if c["train"] else 0
        return dict(bytes=active * 6 * F * H + rows * (4 * H + kept) + 4 * E, flops=flops)
    if c["part"] == "weights":  # a, grad_y, grad_gate_up and inner in, every expert's weight gradients out
        return dict(bytes=rows * (4 * H + 6 * F) + E * 12 * F * H + 4 * E, flops=flops)
    # both weights, a, grad_y, gate_up and inner in; grad_gate_up, grad_a and every expert's weight gradients out
    return dict(bytes=active * 6 * F * H + rows * (6 * H + 10 * F) + E * 6 * F * H + 4 * E, flops=2 * flops)


def _active(E: int, K: int, tokens: int, zipf: bool) -> float:
    share = [1.0 / E] * E
    if zipf:
        total = sum((e + 1) ** -1.2 for e in range(E))
        share = [(e + 1) ** -1.2 / total for e in range(E)]
    return sum(1.0 - (1.0 - min(1.0, K * p)) ** tokens for p in share)


# --------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    c = dict(case)
    if c["op"] in ("ffn", "ffn_backward", "ffn_int8") and c["tokens"] * c["K"] * c["hidden"] * c["ffn"] > 6e11:
        return None
    return dict(ffn=_exact_ffn, ffn_backward=_exact_ffn_backward, combine_backward=_exact_combine_backward,
                dispatch_int8=_exact_dispatch_int8, ffn_int8=_exact_ffn_int8)[c["op"]](c, prepare(case, seed))


def _exact_rows(s):
    """(expert, rows) of every expert that has some."""
    return [(e, m) for e, m in enumerate(s["count"].tolist()) if m > 0]


def _f64(*shape):
    return torch.zeros(shape, dtype=torch.float64, device="cuda")


def _exact_ffn(c, s):
    E, cap, H, F = c["E"], c["cap"], c["hidden"], c["ffn"]
    y, inner, gate_up = _f64(E, cap, H), _f64(E, cap, F), _f64(E, cap, 2, F)
    for e, m in _exact_rows(s):
        x = s["a"][e, :m].double()
        for i in range(2):
            gate_up[e, :m, i] = x @ s["w13"][e, i].double().T
        inner[e, :m] = gate_up[e, :m, 0] * torch.sigmoid(gate_up[e, :m, 0]) * gate_up[e, :m, 1]
        # the second product's rows are the first one's output, held in bf16
        y[e, :m] = inner[e, :m].to(torch.bfloat16).double() @ s["w2"][e].double().T
    return dict(y=y, inner=inner, gate_up=gate_up) if c["train"] else dict(y=y, inner=inner)


def _exact_ffn_backward(c, s):
    E, cap, H, F = c["E"], c["cap"], c["hidden"], c["ffn"]
    out = dict(grad_w13=_f64(E, 2, F, H), grad_w2=_f64(E, H, F))
    if c["part"] == "all":
        out |= dict(grad_gate_up=_f64(E, cap, 2, F), grad_a=_f64(E, cap, H))
    for e, m in _exact_rows(s):
        gy, x = s["grad_y"][e, :m].double(), s["a"][e, :m].double()
        held = s["grad_gate_up"][e, :m].double()
        if c["part"] == "all":
            gu = s["gate_up"][e, :m].double().requires_grad_(True)
            with torch.enable_grad():
                h = torch.nn.functional.silu(gu[:, 0]) * gu[:, 1]
                (h * (gy @ s["w2"][e].double())).sum().backward()
            out["grad_gate_up"][e, :m] = gu.grad
            held = gu.grad.to(torch.bfloat16).double()
            for i in range(2):
                out["grad_a"][e, :m] += held[:, i] @ s["w13"][e, i].double()
        for i in range(2):
            out["grad_w13"][e, i] = held[:, i].T @ x
        out["grad_w2"][e] = gy.T @ s["inner"][e, :m].double()
    return out


def _exact_combine_backward(c, s):
    R, T, H, E, K, cap = c["R"], c["T"], c["H"], c["E"], c["K"], c["cap"]
    if E * cap * H > 4e9:
        return None
    gy, gw = _f64(E * cap, H), _f64(R * T, K)
    idx, pos = s["topk_idx"].view(R * T, K), s["slot_pos"].view(R * T, K)
    g = s["grad"].view(R * T, H).double()
    for k in range(K):
        ok = pos[:, k] >= 0
        at = (idx[:, k] * cap + pos[:, k])[ok]
        gw[ok, k] = torch.einsum("th,th->t", g[ok], s["y"].view(E * cap, H)[at].double())
        gy[at] = g[ok] * s["topk_w"].view(R * T, K)[ok, k].double().unsqueeze(-1)
    return dict(grad_y=gy.view(E, cap, H), grad_topk_w=gw.view(R, T, K))


def _exact_dispatch_int8(c, s):
    R, T, H, E, K, cap = c["R"], c["T"], c["H"], c["E"], c["K"], c["cap"]
    scale = s["x"].view(R * T, H).double().abs().amax(-1).clamp(min=AMAX_FLOOR) / INT8_MAX
    out = _f64(E * cap)
    for k in range(K):
        pos = s["slot_pos"].view(R * T, K)[:, k]
        ok = pos >= 0
        out[(s["topk_idx"].view(R * T, K)[:, k] * cap + pos)[ok]] = scale[ok]
    # the quotients of 64 bits round to another whole number beside a tie
    return dict(recv_x=None, recv_x_scales=out.view(E, cap), recv_src_info=None)


def _exact_ffn_int8(c, s):
    E, cap, H, F = c["E"], c["cap"], c["hidden"], c["ffn"]
    y, scales = _f64(E, cap, H), _f64(E, cap)
    for e, m in _exact_rows(s):
        x = s["a"][e, :m].double()
        gate, up = ((x @ s["w13"][e, i].double().T) * s["a_scales"][e, :m, None].double() * s["w13_scales"][e, i].double()
                    for i in range(2))
        h = torch.nn.functional.silu(gate) * up
        scales[e, :m] = h.abs().amax(-1).clamp(min=AMAX_FLOOR) / INT8_MAX
        q = torch.round(h / scales[e, :m, None])
        y[e, :m] = (q @ s["w2"][e].double().T) * scales[e, :m, None] * s["w2_scales"][e].double()
    return dict(y=y, inner_scales=scales)
