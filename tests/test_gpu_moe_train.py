"""MoETrainLayer: forward and backward of a whole expert layer, each stage checked on what the one
before it left (routing and layout exactly, the rest in float64 with the bounds of experts_ref), and
all of it against float64 gradients of the layer's definition; MoELayer with int8 experts likewise."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import experts_ref as ref
import moe_ref
import oracle
from combine_get_dispatch_notify_gb300 import ep
from combine_get_dispatch_notify_gb300.workloads import Workload, gen_x

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.lib()


LAYERS = {  # R, T, H, E, K, ffn, capacity (None: no drop), groups
    "tiny": (2, 32, 256, 16, 2, 128, None, 1),
    "one_token": (1, 1, 512, 8, 3, 256, None, 1),
    "grouped": (4, 50, 384, 64, 6, 160, None, 8),
    "many_ranks": (24, 5, 256, 48, 4, 128, None, 1),       # the layout step counts
    "long_expert": (2, 300, 256, 4, 2, 144, None, 1),      # rows beyond one tile
    "capacity_drop": (2, 64, 256, 4, 2, 128, 20, 1),
    "no_tokens": (2, 0, 256, 4, 2, 128, 8, 1),
}


def make(name, seed=1):
    R, T, H, E, K, F, cap, G = LAYERS[name]
    g = torch.Generator().manual_seed(seed)
    w13 = (torch.randn(E, 2, F, H, generator=g) / H ** 0.5).to(BF16)
    w2 = (torch.randn(E, H, F, generator=g) / F ** 0.5).to(BF16)
    logits = torch.round(torch.randn(R, T, E, generator=g) * 64) / 64
    bias = torch.round(torch.randn(E, generator=g) * 8) / 32
    grad = torch.randn(R, T, H, generator=g).to(BF16)
    x = gen_x(Workload("m", R=R, T=T, H=H, E=E, K=K, C=1, seed=seed))
    cap = max(1, R * T) if cap is None else cap
    shape = ep.EpShape.make(R, T, K, E, H, 1)
    route = ep.EpRoute.make("sigmoid", G, max(1, G // 2), 2 if G > 1 else 1, True, 2.5)
    return shape, route, F, cap, x, logits, bias, w13, w2, grad


def step(layer, x, logits, bias, w13, w2, grad, dtype=torch.float32):
    """One forward and backward on the current stream: (out, grad_x, grad_logits, grad_w13, grad_w2)."""
    gl = torch.full_like(logits, 7.0)
    g13, g2 = torch.full_like(w13, 7.0, dtype=dtype), torch.full_like(w2, 7.0, dtype=dtype)
    out = layer.run(x, logits, bias, w13, w2)
    gx = layer.backward(grad, logits, w13, w2, gl, g13, g2)
    return out, gx, gl, g13, g2


@pytest.mark.parametrize("name", sorted(LAYERS))
def test_layer_stage_by_stage(name):
    shape, route, F, cap, x, logits, bias, w13, w2, grad = make(name)
    R, T, K, E, H = shape.num_ranks, shape.num_tokens, shape.num_topk, shape.num_experts, shape.hidden
    layer = ep.MoETrainLayer(shape, route, F, cap)
    got = step(layer, *(t.cuda() for t in (x, logits, bias, w13, w2, grad)))
    rc = ep.ep_sync_status(layer.status)
    out, gx, gl, g13, g2 = (t.cpu() for t in got)
    if T == 0:
        assert rc == ep.EP_OK and out.numel() == 0 and not g13.any() and not g2.any()
        return
    idx = layer.topk_idx.cpu()
    wt = layer.topk_w.cpu().view(-1, K)
    ridx, rwt = moe_ref.route(logits, bias, K, "sigmoid", route.num_groups, route.topk_groups, route.group_top, True, 2.5)
    assert np.array_equal(idx.view(-1, K).numpy(), ridx)
    np.testing.assert_allclose(wt.double().numpy(), rwt, rtol=1e-5)
    lay = oracle.ll_layout(oracle.load(), R, T, K, E, cap, idx.numpy())
    assert rc == (ep.EP_ERR_CAPACITY if lay["dropped"] else ep.EP_OK)
    slot = layer.slot_pos.cpu()
    assert np.array_equal(slot.numpy(), lay["slot_pos"])
    rows, gu, inner, y = (t.cpu() for t in (layer.rows, layer.gate_up, layer.inner, layer.y))
    gy, gwt, ggu, grows = (t.cpu() for t in (layer.grad_y, layer.grad_topk_w, layer.grad_gate_up, layer.grad_rows))
    flat, gflat = x.view(-1, H), grad.view(-1, H)
    want = torch.zeros(R * T, H, dtype=torch.float64)
    mag, wantx, magx = torch.zeros_like(want), torch.zeros_like(want), torch.zeros_like(want)
    for t in range(R * T):
        for k in range(K):
            e, p = int(idx.view(-1, K)[t, k]), int(slot.view(-1, K)[t, k])
            if e < 0 or p < 0:
                assert float(gwt.view(-1, K)[t, k]) == 0
                continue
            assert torch.equal(rows[e, p], flat[t])
            term = float(wt[t, k]) * y[e, p].double()
            want[t] += term
            mag[t] += term.abs()
            wantx[t] += grows[e, p].double()
            magx[t] += grows[e, p].double().abs()
            assert torch.equal(gy[e, p], (gflat[t].float() * wt[t, k]).to(BF16))
            dot = gflat[t].double() * y[e, p].double()
            assert abs(float(gwt.view(-1, K)[t, k]) - float(dot.sum())) <= float(dot.abs().sum()) * ref.sum_error(H)
    ref.close_bf16("out", out.view(-1, H), want, mag * ref.sum_error(K))
    ref.close_bf16("grad_x", gx.view(-1, H), wantx, magx * ref.sum_error(K))
    for e in range(E):
        m = min(int(layer.count[e]), cap)
        h, dh, (g, u), (dg, du) = ref.gated(rows[e, :m], w13[e])
        ref.close_bf16("gate", gu[e, :m, 0], g, dg)
        ref.close_bf16("up", gu[e, :m, 1], u, du)
        ref.close_bf16("inner", inner[e, :m], h, dh)
        ref.close_bf16("y", y[e, :m], *ref.product(inner[e, :m], w2[e]))
        gh, dgh = ref.product(gy[e, :m], w2[e].T)
        parts, bounds = ref.gated_gradient(gh, dgh, gu[e, :m, 0], gu[e, :m, 1])
        for i in range(2):
            ref.close_bf16("grad_gate_up", ggu[e, :m, i], parts[i], bounds[i])
            ref.close_fp32("grad_w13", g13[e, i], *ref.product(ggu[e, :m, i].T, rows[e, :m].T))
        ref.close_bf16("grad_rows", grows[e, :m], *ref.product(ggu[e, :m].flatten(1), w13[e].flatten(0, 1).T))
        ref.close_fp32("grad_w2", g2[e], *ref.product(gy[e, :m].T, inner[e, :m].T))
    want_gl = moe_ref.route_backward(logits, idx, gwt, "sigmoid", True, 2.5)
    scale = gwt.double().abs().amax() * 2.5
    assert ((gl.double() - want_gl).abs() <= 1e-5 * (want_gl.abs() + 1e-2 * scale)).all()


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_gradients_of_the_whole_layer(dtype):
    """Against float64 autograd through routing weights, experts and combine.  bf16 roundings on the
    way (gate and up, h, y, both gradients between, the result): a handful of 2^-8 steps of the
    gradient's size bound its distance."""
    shape, route, F, cap, x, logits, bias, w13, w2, grad = make("tiny")
    K, E, H = shape.num_topk, shape.num_experts, shape.hidden
    layer = ep.MoETrainLayer(shape, route, F, cap)
    got = [t.cpu() for t in step(layer, *(t.cuda() for t in (x, logits, bias, w13, w2, grad)), dtype=dtype)]
    assert got[3].dtype == dtype
    idx = layer.topk_idx.cpu()
    leaves = [t.double().requires_grad_(True) for t in (x, logits, w13, w2)]
    dx, dl, d13, d2 = leaves
    wt = moe_ref.weights_of(dl, torch.ones(1, dtype=torch.bool), idx, "sigmoid", True, 2.5)
    flat = dx.view(-1, H)
    out = 0
    for k in range(K):
        e = idx.view(-1, K)[:, k]
        g = torch.einsum("th,tfh->tf", flat, d13[e, 0])
        u = torch.einsum("th,tfh->tf", flat, d13[e, 1])
        out = out + torch.einsum("tf,thf->th", ref.silu(g) * u, d2[e]) * wt.view(-1, K)[:, k:k + 1]
    (out * grad.double().view(-1, H)).sum().backward()
    for name, t, want in zip(("out", "x", "logits", "w13", "w2"), got, [out.detach().view_as(x)] + [t.grad for t in leaves]):
        err = float((t.double() - want).norm() / want.norm())
        assert err <= 6 * ref.HALF, (name, err)


def test_layer_repeats_and_takes_new_inputs():
    args = make("grouped")
    other = make("grouped", seed=2)
    shape, route, F, cap = args[:4]
    layer, fresh = ep.MoETrainLayer(shape, route, F, cap), ep.MoETrainLayer(shape, route, F, cap)
    run = lambda l, a: [t.cpu() for t in step(l, *(v.cuda() for v in a[4:]))]  # noqa: E731
    first, second = run(layer, args), run(layer, other)
    for a, b in zip(second, run(fresh, other)):
        assert torch.equal(a, b)
    for a, b in zip(first, run(layer, args)):
        assert torch.equal(a, b)
    assert ep.ep_sync_status(layer.status) == ep.EP_OK


def test_training_step_in_a_cuda_graph():
    args = make("long_expert")
    shape, route, F, cap = args[:4]
    on = [t.cuda() for t in args[4:]]
    layer = ep.MoETrainLayer(shape, route, F, cap)
    want = [t.cpu() for t in step(layer, *on)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(layer, *on)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(layer, *on)
    for t in got:
        t.zero_()
    graph.replay()
    graph.replay()
    assert ep.ep_sync_status(layer.status) == ep.EP_OK
    for a, b in zip(got, want):
        assert torch.equal(a.cpu(), b)


@pytest.mark.parametrize("name", sorted(LAYERS))
def test_int8_layer_stage_by_stage(name):
    shape, route, F, cap, x, logits, bias, w13, w2, _ = make(name)
    R, T, K, E, H = shape.num_ranks, shape.num_tokens, shape.num_topk, shape.num_experts, shape.hidden
    q13, s13 = ep.cast_weight_channels(w13)
    q2, s2 = ep.cast_weight_channels(w2)
    layer = ep.MoELayer(shape, route, F, cap, weights="int8")
    out = layer.run(*(t.cuda() for t in (x, logits, bias, q13, s13, q2, s2))).cpu()
    rc = ep.ep_sync_status(layer.status)
    if T == 0:
        assert rc == ep.EP_OK and out.numel() == 0
        return
    idx, wt = layer.topk_idx.cpu(), layer.topk_w.cpu().view(-1, K)
    lay = oracle.ll_layout(oracle.load(), R, T, K, E, cap, idx.numpy())
    assert rc == (ep.EP_ERR_CAPACITY if lay["dropped"] else ep.EP_OK)
    slot = layer.slot_pos.cpu()
    assert np.array_equal(slot.numpy(), lay["slot_pos"])
    q, s = ref.cast_rows(x.view(-1, H))
    rows, scales, inner, inner_scales, y = (t.cpu() for t in (layer.rows, layer.row_scales, layer.inner, layer.inner_scales,
                                                              layer.y))
    want = torch.zeros(R * T, H, dtype=torch.float64)
    mag = torch.zeros_like(want)
    for t in range(R * T):
        for k in range(K):
            e, p = int(idx.view(-1, K)[t, k]), int(slot.view(-1, K)[t, k])
            if e < 0 or p < 0:
                continue
            assert torch.equal(rows[e, p], q[t]) and float(scales[e, p]) == float(s[t])
            term = float(wt[t, k]) * y[e, p].double()
            want[t] += term
            mag[t] += term.abs()
    ref.close_bf16("out", out.view(-1, H), want, mag * ref.sum_error(K))
    for e in range(E):
        m = min(int(layer.count[e]), cap)
        if m == 0:
            continue
        g, u = ((rows[e, :m].double() @ q13[e, i].double().T) * scales[e, :m].double().unsqueeze(-1) * s13[e, i].double()
                for i in range(2))
        h = ref.silu(g) * u
        dh = h.abs() * 2.0 ** -19 + (g.abs() + 1) * u.abs() * 2.0 ** -21
        step_ = inner_scales[e, :m].double().unsqueeze(-1)
        assert ((inner[e, :m].double() * step_ - h).abs() <= step_ * (0.5 + 2.0 ** -15) + dh).all(), e
        p2 = (inner[e, :m].double() @ q2[e].double().T) * step_ * s2[e].double()
        ref.close_bf16("y", y[e, :m], p2, p2.abs() * 2.0 ** -22)
