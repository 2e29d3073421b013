"""MoELayer: the router, the low-latency layout, the casting dispatch, the experts'
products and the weighted combine together, each stage checked on what the one
before it left (routing, layout and dispatch exactly; the products with the bounds of
test_gpu_ll_fp8; the combine in float64 from the layer's own expert outputs)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import moe_ref
import oracle
from combine_get_dispatch_notify_gb300 import ep
from combine_get_dispatch_notify_gb300.workloads import Workload, gen_x
from test_gpu_ll_fp8 import silu

pytestmark = pytest.mark.gpu


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
    w13, s13 = ep.cast_weight_blocks(torch.randn(E, 2, F, H, generator=g) / H ** 0.5)
    w2, s2 = ep.cast_weight_blocks(torch.randn(E, H, F, generator=g) / F ** 0.5)
    logits = torch.round(torch.randn(R, T, E, generator=g) * 64) / 64
    bias = torch.round(torch.randn(E, generator=g) * 8) / 32
    x = gen_x(Workload("m", R=R, T=T, H=H, E=E, K=K, C=1, seed=seed))
    cap = max(1, R * T) if cap is None else cap
    shape = ep.EpShape.make(R, T, K, E, H, 1)
    route = ep.EpRoute.make("sigmoid", G, max(1, G // 2), 2 if G > 1 else 1, True, 2.5)
    return shape, route, F, cap, x, logits, bias, (w13, s13, w2, s2)


@pytest.mark.parametrize("name", sorted(LAYERS))
def test_layer_stage_by_stage(name):
    shape, route, F, cap, x, logits, bias, weights = make(name)
    R, T, K, E, H = shape.num_ranks, shape.num_tokens, shape.num_topk, shape.num_experts, shape.hidden
    layer = ep.MoELayer(shape, route, F, cap)
    out = layer.run(x.cuda(), logits.cuda(), bias.cuda(), *(t.cuda() for t in weights)).cpu()
    rc = ep.ep_sync_status(layer.status)
    if T == 0:
        assert rc == ep.EP_OK and out.numel() == 0
        return
    idx, wt = moe_ref.route(logits, bias, K, "sigmoid", route.num_groups, route.topk_groups, route.group_top, True, 2.5)
    got_idx, got_w = layer.topk_idx.cpu(), layer.topk_w.cpu()
    assert np.array_equal(got_idx.view(-1, K).numpy(), idx)
    np.testing.assert_allclose(got_w.view(-1, K).double().numpy(), wt, rtol=1e-5)
    ref = oracle.ll_layout(oracle.load(), R, T, K, E, cap, got_idx.numpy())
    assert rc == (ep.EP_ERR_CAPACITY if ref["dropped"] else ep.EP_OK)
    slot = layer.slot_pos.cpu()
    assert np.array_equal(slot.numpy(), ref["slot_pos"])
    q, s = moe_ref.cast_blocks(x.view(R * T, H))
    rows, scales, y = layer.rows.cpu(), layer.row_scales.cpu(), layer.y.cpu()
    inner, inner_scales = layer.inner.cpu(), layer.inner_scales.cpu()
    w13, s13, w2, s2 = weights
    c = moe_ref.sum_error(max(H, F))
    want = torch.zeros(R * T, H, dtype=torch.float64)
    mag = torch.zeros_like(want)
    for t in range(R * T):
        for k in range(K):
            e, p = int(got_idx.view(-1, K)[t, k]), int(slot.view(-1, K)[t, k])
            if e < 0 or p < 0:
                continue
            assert torch.equal(rows[e, p], q[t]) and torch.equal(scales[e, p], s[t])
            term = float(got_w.view(-1, K)[t, k]) * y[e, p].double()
            want[t] += term
            mag[t] += term.abs()
    for e in range(E):
        m = min(int(layer.count[e]), cap)
        if m == 0:
            continue
        gate, gm = moe_ref.product(rows[e, :m], scales[e, :m], w13[e, 0], s13[e, 0])
        up, um = moe_ref.product(rows[e, :m], scales[e, :m], w13[e, 1], s13[e, 1])
        h = silu(gate) * up
        dh = 1.1 * gm * c * (up.abs() + um * c) + silu(gate).abs() * um * c + h.abs() * 2.0 ** -20
        back = moe_ref.fp8(inner[e, :m]) * moe_ref.expand(inner_scales[e, :m], F, -1)
        # half an e4m3 step: 2^-4 of a normal value, 2^-10 of the scale below; and the scale's own error
        tol = h.abs() / 16 + moe_ref.expand(inner_scales[e, :m], F, -1) * 2.0 ** -10 + 4 * dh.amax(-1, True)
        assert ((back - h).abs() <= tol).all(), e
        p2, mag2 = moe_ref.product(inner[e, :m], inner_scales[e, :m], w2[e], s2[e])
        assert ((y[e, :m].double() - p2).abs() <= p2.abs() * 2.0 ** -8 + mag2 * c).all(), e
    err = (out.view(R * T, H).double() - want).abs()
    assert (err <= want.abs() * 2.0 ** -8 + mag * (K + 2) * 2.0 ** -24).all()


def test_layer_runs_repeat_and_take_new_inputs():
    """The same buffers serve call after call: new inputs leave nothing of the old ones, and the old
    inputs give their bits again."""
    shape, route, F, cap, x, logits, bias, weights = make("grouped")
    x2, logits2 = make("grouped", seed=2)[4:6]
    weights = [t.cuda() for t in weights]
    layer, fresh = ep.MoELayer(shape, route, F, cap), ep.MoELayer(shape, route, F, cap)
    run = lambda l, a, b: l.run(a.cuda(), b.cuda(), bias.cuda(), *weights).clone()  # noqa: E731
    first = run(layer, x, logits)
    second = run(layer, x2, logits2)
    assert torch.equal(second, run(fresh, x2, logits2))
    assert torch.equal(first, run(layer, x, logits))
    assert ep.ep_sync_status(layer.status) == ep.EP_OK


def test_layer_in_a_cuda_graph():
    shape, route, F, cap, x, logits, bias, weights = make("long_expert")
    args = [t.cuda() for t in (x, logits, bias, *weights)]
    layer = ep.MoELayer(shape, route, F, cap)
    want = layer.run(*args).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.run(*args)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.run(*args)
    layer.combined_x.zero_()
    graph.replay()
    graph.replay()
    assert ep.ep_sync_status(layer.status) == ep.EP_OK
    assert torch.equal(layer.combined_x, want)


def test_weight_cast_covers_ragged_blocks():
    w = torch.randn(2, 130, 272, generator=torch.Generator().manual_seed(3)) * 3
    q, s = ep.cast_weight_blocks(w)
    assert q.shape == (2, 130, 272) and s.shape == (2, 2, 3) and q.is_contiguous() and s.is_contiguous()
    back = moe_ref.fp8(q) * moe_ref.expand(moe_ref.expand(s, 130, -2), 272, -1)
    sc = moe_ref.expand(moe_ref.expand(s, 130, -2), 272, -1)
    assert ((back - w).abs() <= w.abs() / 16 + sc * 2.0 ** -10).all()


def test_binding_refuses_strided_tensors():
    sh = ep.EpShape.make(1, 4, 2, 8, 256, 1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    wide = torch.zeros(1, 4, 16, device="cuda")[..., ::2]
    idx, w = torch.zeros(1, 4, 2, dtype=torch.int64, device="cuda"), torch.zeros(1, 4, 2, device="cuda")
    with pytest.raises(ValueError):
        ep.ep_route(sh, ep.EpRoute.make(), wide, None, idx, w, status)
    a = torch.zeros(2, 8, 512, dtype=torch.uint8, device="cuda")[..., ::2]
    with pytest.raises(ValueError):
        ep.ep_ll_gemm_fp8(a, torch.zeros(2, 8, 2, device="cuda"), torch.zeros(2, 128, 256, dtype=torch.uint8, device="cuda"),
                          torch.zeros(2, 1, 2, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"),
                          torch.zeros(2, 8, 128, dtype=torch.bfloat16, device="cuda"), status)
    # an address off the 16-byte grid is refused by the library
    flat = torch.zeros(33, device="cuda")
    with pytest.raises(ep.EpError):
        ep.ep_route(sh, ep.EpRoute.make(), flat[1:].view(1, 4, 8), None, idx, w, status)
