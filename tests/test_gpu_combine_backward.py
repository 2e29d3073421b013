"""Gradient of the weighted combine against float64, bit for bit where it is one product."""
from __future__ import annotations

import pytest
import torch

import experts_ref as ref
import oracle
from combine_get_dispatch_notify_gb300 import ep
from combine_get_dispatch_notify_gb300.workloads import Workload, gen_routing
from test_gpu_ll_int8 import BF16, ROUTES, placed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.lib()


MORE = {
    "eight_columns": (2, 21, 8, 6, 2, None),
    "a_warps_longest_row": (1, 17, 1024, 8, 3, None),
    "past_a_warps_row": (1, 17, 1032, 8, 3, None),
    "nine_slots": (1, 50, 200, 12, 9, None),
}


def run(shape, cap, g, y, idx, wt, slot, gy, gw, stream=None):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.ep_ll_combine_backward(shape, g, y, cap, idx, wt, slot, gy, gw, status, stream)
    return ep.ep_sync_status(status, stream)


@pytest.mark.parametrize("name", sorted(ROUTES) + sorted(MORE))
def test_against_float64(name):
    ROUTES.update({k: v for k, v in MORE.items() if k == name})
    try:
        shape, cap, idx, wt, slot, _ = placed(name)
    finally:
        for k in MORE:
            ROUTES.pop(k, None)
    R, T, K, E, H = shape.num_ranks, shape.num_tokens, shape.num_topk, shape.num_experts, shape.hidden
    gen = torch.Generator().manual_seed(2)
    g, y = torch.randn(R, T, H, generator=gen).to(BF16), torch.randn(E, cap, H, generator=gen).to(BF16)
    if R * T > 2:
        idx, slot = idx.clone(), slot.clone()
        idx[0, 0, 0], slot[-1, T - 1, K - 1] = -1, -1
    gy = torch.full((E, cap, H), 7.0, dtype=BF16, device="cuda")
    gw = torch.full((R, T, K), 7.0, device="cuda")
    assert run(shape, cap, g.cuda(), y.cuda(), idx.cuda(), wt.cuda(), slot.cuda(), gy, gw) == ep.EP_OK
    want_gy = torch.full((E, cap, H), 7.0, dtype=BF16)
    want_gw, bound = torch.zeros(R * T, K, dtype=torch.float64), torch.zeros(R * T, K, dtype=torch.float64)
    for t in range(R * T):
        v = g.view(-1, H)[t]
        for k in range(K):
            e, r = int(idx.view(-1, K)[t, k]), int(slot.view(-1, K)[t, k])
            if e < 0 or r < 0:
                continue
            want_gy[e, r] = (v.float() * wt.view(-1, K)[t, k]).to(BF16)
            terms = v.double() * y[e, r].double()
            want_gw[t, k], bound[t, k] = terms.sum(), terms.abs().sum() * ref.sum_error(H)
    assert torch.equal(gy.cpu(), want_gy)
    ref.close_fp32("grad_topk_w", gw.view(-1, K).cpu(), want_gw, bound)


def test_matches_differences_of_the_combine():
    """<grad, d> against the combine itself at shifted weights and outputs (the combine is linear in
    each, so a difference quotient is exact but for its own bf16 result)."""
    shape, cap, idx, wt, slot, _ = placed("short_rows")
    R, T, K, E, H = shape.num_ranks, shape.num_tokens, shape.num_topk, shape.num_experts, shape.hidden
    gen = torch.Generator().manual_seed(3)
    g, y = torch.randn(R, T, H, generator=gen).to(BF16), torch.randn(E, cap, H, generator=gen).to(BF16)
    gy, gw = torch.zeros(E, cap, H, dtype=BF16, device="cuda"), torch.zeros(R, T, K, device="cuda")
    assert run(shape, cap, g.cuda(), y.cuda(), idx.cuda(), wt.cuda(), slot.cuda(), gy, gw) == ep.EP_OK
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def combined(yy, ww):
        out = torch.zeros(R, T, H, dtype=BF16, device="cuda")
        ep.ep_ll_combine(shape, yy.cuda(), cap, idx.cuda(), ww.cuda(), slot.cuda(), out, status)
        return out.cpu().double()

    d = torch.randn(E, cap, H, generator=gen).to(BF16)
    out = combined(d, wt)  # the change along d
    assert abs((gy.cpu().double() * d.double()).sum() - (out * g.double()).sum()) <= \
        2 * ref.HALF * (out.abs() * g.double().abs()).sum() + ref.HALF * (gy.cpu().double() * d.double()).abs().sum()
    dw = torch.randn(R, T, K, generator=gen)
    out = combined(y, dw)
    assert abs((gw.cpu().double() * dw.double()).sum() - (out * g.double()).sum()) <= \
        2 * ref.HALF * (out.abs() * g.double().abs()).sum()


def test_slots_past_their_range_are_reported_and_skipped():
    shape = ep.EpShape.make(1, 3, 2, 4, 16, 1)
    one = torch.ones(1, 3, 16, dtype=BF16, device="cuda")
    y = torch.ones(4, 2, 16, dtype=BF16, device="cuda")
    idx = torch.tensor([[[4, 1], [-1, 2], [3, 0]]]).cuda()
    slot = torch.tensor([[[0, 2], [0, 1], [-1, 0]]], dtype=torch.int32).cuda()
    gy, gw = torch.full((4, 2, 16), 7.0, dtype=BF16, device="cuda"), torch.full((1, 3, 2), 7.0, device="cuda")
    w = torch.full((1, 3, 2), 2.0, device="cuda")
    assert run(shape, 2, one, y, idx, w, slot, gy, gw) == ep.EP_ERR_INCONSISTENT
    assert gw.tolist() == [[[0, 0], [0, 16], [0, 16]]]
    want = torch.full((4, 2, 16), 7.0)
    want[2, 1], want[0, 0] = 2.0, 2.0
    assert torch.equal(gy.cpu().float(), want)


def test_repeats_on_streams_and_in_a_graph():
    shape, cap, idx, wt, slot, _ = placed("model_rows")
    R, T, K, E, H = shape.num_ranks, shape.num_tokens, shape.num_topk, shape.num_experts, shape.hidden
    gen = torch.Generator().manual_seed(4)
    g, y = torch.randn(R, T, H, generator=gen).to(BF16).cuda(), torch.randn(E, cap, H, generator=gen).to(BF16).cuda()
    idx, wt, slot = idx.cuda(), wt.cuda(), slot.cuda()
    make = lambda: (torch.zeros(E, cap, H, dtype=BF16, device="cuda"), torch.zeros(R, T, K, device="cuda"))  # noqa: E731
    a, b, c = make(), make(), make()
    assert run(shape, cap, g, y, idx, wt, slot, *a) == ep.EP_OK
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert run(shape, cap, g, y, idx, wt, slot, *b, stream=side) == ep.EP_OK
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.ep_ll_combine_backward(shape, g, y, cap, idx, wt, slot, *c, status)
    graph.replay()
    graph.replay()
    assert ep.ep_sync_status(status) == ep.EP_OK
    for other in (b, c):
        assert torch.equal(a[0], other[0]) and torch.equal(a[1], other[1])


@pytest.mark.parametrize("K", [4, 9])
def test_an_expert_picked_twice_by_a_token(K):
    """Slots of one token may name the same expert: they have rows, gradients and weights of their own."""
    R, T, H, E = 2, 60, 136, 6
    wl = Workload("m", R=R, T=T, H=H, E=E, K=K, C=1, seed=5, routing="replace")
    idx, wt = gen_routing(wl)
    assert any(len(set(r)) < K for r in idx.view(-1, K).tolist())
    cap = R * T * K
    slot = torch.from_numpy(oracle.ll_layout(oracle.load(), R, T, K, E, cap, idx.numpy())["slot_pos"])
    shape = ep.EpShape.make(R, T, K, E, H, 1)
    gen = torch.Generator().manual_seed(6)
    g, y = torch.randn(R, T, H, generator=gen).to(BF16), torch.randn(E, cap, H, generator=gen).to(BF16)
    gy, gw = torch.zeros(E, cap, H, dtype=BF16, device="cuda"), torch.zeros(R, T, K, device="cuda")
    assert run(shape, cap, g.cuda(), y.cuda(), idx.cuda(), wt.cuda(), slot.cuda(), gy, gw) == ep.EP_OK
    at = idx.view(-1, K), slot.view(-1, K).long()
    assert torch.equal(gy.cpu()[at], (g.view(-1, 1, H).float() * wt.view(-1, K, 1)).to(BF16))
    terms = g.view(-1, 1, H).double() * y[at].double()
    ref.close_fp32("grad_topk_w", gw.view(-1, K).cpu(), terms.sum(-1), terms.abs().sum(-1) * ref.sum_error(H))
