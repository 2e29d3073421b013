"""Experts' int8 products against whole-number sums, the gated product's cast by rows, and the
dispatch that casts to int8, bit for bit."""
from __future__ import annotations

import pytest
import torch

import experts_ref as ref
import oracle
from combine_get_dispatch_notify_gb300 import ep
from combine_get_dispatch_notify_gb300.workloads import Workload, gen_routing, gen_x

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.lib()


# n, k, capacity, rows of each expert
SHAPES = {
    "smallest": (16, 16, 3, [1, 0, 3]),
    "one_row": (128, 64, 1, [1, 0, 1, 1]),
    "odd": (48, 144, 20, [17, 16, 15, 0, 20]),
    "past_a_block": (80, 272, 70, [31, 32, 33, 63, 64, 65, 1]),
    "past_a_tile": (272, 112, 130, [127, 128, 129, 2]),
    "two_tiles": (144, 80, 300, [255, 256, 257, 300, 31, 33]),
    "rows_ten_tiles": (528, 336, 700, [700, 513, 0, 511]),
    "wide": (2064, 64, 40, [33, 40]),
    "deep": (64, 4112, 40, [33, 40]),
    "counts_past_the_capacity": (64, 64, 10, [11, 1 << 30, -1, -(1 << 31), 10]),
    "all_empty": (48, 48, 16, [0, 0, 0]),
    "many_experts": (32, 48, 9, [i % 10 for i in range(300)]),
    "many_tiles_of_all_sizes": (272, 80, 300, [255, 256, 257, 300, 31, 33, 129, 0] * 20),
    "many_longer_experts": (32, 48, 140, [i * 7 % 141 for i in range(300)]),
    "more_tiles_than_sms": (1040, 64, 520, [520] * 24),
}


def rows_of(name):
    n, k, cap, counts = SHAPES[name]
    return n, k, cap, counts, [min(max(c, 0), cap) for c in counts]


def whole(seed, *shape):
    return torch.randint(-127, 128, shape, generator=torch.Generator().manual_seed(seed), dtype=torch.int8)


def near(seed, *shape, scale=1.0):
    return torch.exp(torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * 0.5) * scale


def dev(counts):
    return torch.tensor(counts, dtype=torch.int32, device="cuda")


def sums(a, w):
    """Whole-number sums in float64 (exact) and the bound of fp32 sums beyond 2^24."""
    a, w = a.double(), w.double()
    mags = a.abs() @ w.abs().T
    return a @ w.T, torch.where(mags > 2.0 ** 24, mags * ref.sum_error(a.shape[-1]), torch.zeros_like(mags))


def product(a, s, w, ws):
    p, d = sums(a, w)
    scale = s.double().unsqueeze(-1) * ws.double()
    return p * scale, d * scale + (p * scale).abs() * 2.0 ** -22  # the scales' product, and the sum's by it


def poisoned_scales(s, rows):
    s = s.clone()
    for e, m in enumerate(rows):
        s[e, m:] = float("nan")
    return s.cuda()


def run_plain(a, s, w, ws, counts, y):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.ep_ll_gemm_int8(a, s, w, ws, dev(counts), y, status)
    assert ep.ep_sync_status(status) == ep.EP_OK
    return y.cpu()


def run_gated(a, s, w, ws, counts):
    E, cap, k = a.shape
    n = w.shape[2]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, ys = torch.full((E, cap, n), 99, dtype=torch.int8, device="cuda"), torch.full((E, cap), 7.0, device="cuda")
    work = torch.full((ep.ep_ll_gemm_swiglu_int8_workspace_bytes(ep.EpGemmShape(E, cap, n, k)),), 255, dtype=torch.uint8,
                      device="cuda")
    ep.ep_ll_gemm_swiglu_int8(a, s, w, ws, dev(counts), y, ys, work, status)
    assert ep.ep_sync_status(status) == ep.EP_OK
    return y.cpu(), ys.cpu()


@pytest.mark.parametrize("name", sorted(SHAPES))
def test_product(name):
    n, k, cap, counts, rows = rows_of(name)
    E = len(rows)
    a, w = whole(1, E, cap, k), whole(2, E, n, k)
    s, ws = near(3, E, cap, scale=1 / 64), near(4, E, n, scale=1 / 64)
    y = run_plain(a.cuda(), poisoned_scales(s, rows), w.cuda(), ws.cuda(), counts,
                  torch.full((E, cap, n), 7.0, dtype=BF16, device="cuda"))
    for e, m in enumerate(rows):
        assert (y[e, m:] == 7.0).all(), e
        ref.close_bf16(f"y[{e}]", y[e, :m], *product(a[e, :m], s[e, :m], w[e], ws[e]))


@pytest.mark.parametrize("name", sorted(SHAPES))
def test_gated_product(name):
    n, k, cap, counts, rows = rows_of(name)
    E = len(rows)
    a, w = whole(5, E, cap, k), whole(6, E, 2, n, k)
    s, ws = near(7, E, cap, scale=1 / 64), near(8, E, 2, n, scale=k ** -0.5 / 64)
    y, ys = run_gated(a.cuda(), poisoned_scales(s, rows), w.cuda(), ws.cuda(), counts)
    for e, m in enumerate(rows):
        assert (y[e, m:] == 99).all() and (ys[e, m:] == 7.0).all(), e
        if m == 0:
            continue
        (g, dg), (u, du) = (product(a[e, :m], s[e, :m], w[e, i], ws[e, i]) for i in range(2))
        h = ref.silu(g) * u
        dh = 1.1 * dg * (u.abs() + du) + ref.silu(g).abs() * du + h.abs() * 2.0 ** -20
        amax, damax = h.abs().amax(-1), dh.amax(-1)
        ref.close_fp32(f"scale[{e}]", ys[e, :m], amax / 127, damax / 127 + amax / 127 * 2.0 ** -23)
        step = ys[e, :m].double().unsqueeze(-1)
        # half a step, its own error in the quotient, and h's
        assert ((y[e, :m].double() * step - h).abs() <= step * (0.5 + 2.0 ** -15) + dh).all(), e
        assert int(y[e, :m].abs().max()) <= 127


@pytest.mark.parametrize("k", [1024, 2048, 7168])
def test_largest_sums(k):
    """All operands at the type's ends: exact up to 2^24, fp32's roundings beyond (and -128, which a
    cast never makes, is a number like any other)."""
    a, w = torch.full((1, 5, k), 127, dtype=torch.int8), torch.full((1, 16, k), 127, dtype=torch.int8)
    a[0, 1], a[0, 2, ::2], a[0, 3] = -128, -127, whole(9, k)
    w[0, 3], w[0, 4, 1::2] = -128, -127
    one = torch.ones(1, 5, device="cuda"), torch.ones(1, 16, device="cuda")
    y = run_plain(a.cuda(), one[0], w.cuda(), one[1], [5], torch.zeros(1, 5, 16, dtype=BF16, device="cuda"))[0]
    p, d = sums(a[0], w[0])
    ref.close_bf16("y", y, p, d)
    if k == 1024:
        assert torch.equal(y, p.float().to(BF16))


def test_sums_of_small_numbers_are_exact():
    """Scales of 1 and values in [-3, 3]: sums that bf16 holds come out as they are."""
    E, cap, n, k = 2, 37, 48, 4096
    g = torch.Generator().manual_seed(10)
    a = torch.randint(-1, 2, (E, cap, k), generator=g, dtype=torch.int8)
    w = torch.randint(-3, 4, (E, n, k), generator=g, dtype=torch.int8)
    y = run_plain(a.cuda(), torch.ones(E, cap, device="cuda"), w.cuda(), torch.ones(E, n, device="cuda"), [cap, 5],
                  torch.zeros(E, cap, n, dtype=BF16, device="cuda"))
    for e, m in enumerate((cap, 5)):
        assert torch.equal(y[e, :m], (a[e, :m].double() @ w[e].double().T).float().to(BF16))


def test_rows_without_a_number():
    """Scales that are infinite or NaN make their rows NaN, here and through the gated product's cast."""
    E, cap, n, k = 1, 6, 32, 48
    a, w = whole(11, E, cap, k), whole(12, E, 2, n, k)
    a[0, 4] = 0
    s, ws = near(13, E, cap), near(14, E, 2, n, scale=1e-3)
    s[0, 1], s[0, 3] = float("nan"), float("inf")
    y, ys = run_gated(a.cuda(), s.cuda(), w.cuda(), ws.cuda(), [cap])
    assert torch.isfinite(ys[0, [0, 2, 4, 5]]).all() and not torch.isfinite(ys[0, [1, 3]]).any()
    assert (y[0, [1, 3, 4]] == 0).all() and float(ys[0, 4]) > 0
    w2 = whole(15, E, 16, n)
    out = run_plain(y.cuda(), ys.cuda(), w2.cuda(), torch.ones(1, 16, device="cuda"), [cap],
                    torch.zeros(1, cap, 16, dtype=BF16, device="cuda"))[0]
    assert torch.isnan(out[[1, 3]]).all() and torch.isfinite(out[[0, 2, 4, 5]]).all() and (out[4] == 0).all()


def test_repeats_streams_and_graph():
    n, k, cap, counts, rows = rows_of("two_tiles")
    E = len(rows)
    a, s = whole(20, E, cap, k).cuda(), near(21, E, cap, scale=1 / 64).cuda()
    w, ws = whole(22, E, 2, n, k).cuda(), near(23, E, 2, n, scale=1 / 640).cuda()
    w2, ws2 = whole(24, E, k, n).cuda(), near(25, E, k, scale=1 / 64).cuda()
    count = dev(counts)
    shape = ep.EpGemmShape(E, cap, n, k)

    def make():
        return dict(y=torch.zeros(E, cap, n, dtype=torch.int8, device="cuda"), ys=torch.zeros(E, cap, device="cuda"),
                    z=torch.zeros(E, cap, k, dtype=BF16, device="cuda"), status=torch.zeros(1, dtype=torch.int32, device="cuda"),
                    work=torch.zeros(ep.ep_ll_gemm_swiglu_int8_workspace_bytes(shape), dtype=torch.uint8, device="cuda"))

    def calls(b, stream=None):
        ep.ep_ll_gemm_swiglu_int8(a, s, w, ws, count, b["y"], b["ys"], b["work"], b["status"], stream)
        ep.ep_ll_gemm_int8(b["y"], b["ys"], w2, ws2, count, b["z"], b["status"], stream)

    one, two, three = make(), make(), make()
    calls(one)
    torch.cuda.synchronize()
    want = [one[i].cpu() for i in ("y", "ys", "z")]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        calls(two, s1)
        calls(three, s2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(one)
    for i in ("y", "ys", "z"):
        one[i].zero_()
    graph.replay()
    graph.replay()
    for b in (one, two, three):
        assert ep.ep_sync_status(b["status"]) == ep.EP_OK
        for i, t in zip(("y", "ys", "z"), want):
            assert torch.equal(b[i].cpu(), t)


def test_offsets_past_32_bits():
    E, cap, n, k = 3, 8192, 32, 1 << 17
    a = torch.zeros(E, cap, k, dtype=torch.int8, device="cuda")
    assert a.numel() > 1 << 31
    w = torch.zeros(E, n, k, dtype=torch.int8, device="cuda")
    pick = torch.arange(0, k, k // 16).cuda()
    rows, weights = whole(30, 5, 16), whole(31, n, 16)
    a[2, cap - 5:][:, pick] = rows.cuda()
    w[2][:, pick] = weights.cuda()
    y = run_plain(a, torch.ones(E, cap, device="cuda"), w, torch.ones(E, n, device="cuda"), [0, 0, cap],
                  torch.zeros(E, cap, n, dtype=BF16, device="cuda"))
    assert torch.equal(y[2, cap - 5:], (rows.double() @ weights.double().T).float().to(BF16)) and not y[2, :cap - 5].any()


# ------------------------------------------------------------------ dispatch
ROUTES = {  # R, T, H, E, K, capacity (None: all fit)
    "one_token": (1, 1, 16, 1, 1, None),
    "short_rows": (2, 37, 48, 16, 3, None),
    "a_warps_row": (4, 33, 2048, 16, 4, None),
    "past_a_warp": (4, 33, 2064, 16, 4, None),
    "model_rows": (4, 20, 7168, 32, 8, None),
    "a_teams_row": (2, 9, 8192, 8, 2, None),
    "past_a_team": (2, 9, 8208, 8, 2, None),
    "long_rows": (1, 3, 20480, 4, 2, None),
    "drops": (2, 64, 64, 4, 2, 20),
    "many_slots": (8, 11, 272, 64, 32, None),
    "more_tokens_than_teams": (8, 900, 32, 16, 2, None),
}


def placed(name, seed=1):
    R, T, H, E, K, cap = ROUTES[name]
    wl = Workload("m", R=R, T=T, H=H, E=E, K=K, C=1, seed=seed)
    idx, wt = gen_routing(wl)
    cap = R * T if cap is None else cap
    slot = torch.from_numpy(oracle.ll_layout(oracle.load(), R, T, K, E, cap, idx.numpy())["slot_pos"])
    return ep.EpShape.make(R, T, K, E, H, 1), cap, idx, wt, slot, gen_x(wl)


@pytest.mark.parametrize("name", sorted(ROUTES))
def test_casting_dispatch(name):
    shape, cap, idx, _, slot, x = placed(name)
    R, T, K, E, H = shape.num_ranks, shape.num_tokens, shape.num_topk, shape.num_experts, shape.hidden
    x = x.clone()
    flat = x.view(-1, H)
    flat[0] = 0
    if R * T > 8:
        flat[1, H // 2], flat[2, 0], flat[3, H - 1] = float("nan"), float("inf"), -float("inf")
        flat[4] *= 1e-38
        flat[5] = (torch.arange(H) % 255 - 127).to(BF16)  # whole numbers: quotients on the grid and beside ties
        flat[6] = (torch.arange(H) % 127 + 0.5).to(BF16)
        flat[6, 0] = 127
    if not bool(((idx >= 0) & (slot < 0)).any()) and R * T > 8:
        idx, slot = idx.clone(), slot.clone()
        idx[0, 1 % T, 0], slot[-1, T - 1, K - 1] = -1, -1  # slots that a mask left out
    q = torch.full((E, cap, H), 99, dtype=torch.int8, device="cuda")
    s = torch.full((E, cap), 7.0, device="cuda")
    info = torch.full((E, cap, 2), -5, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.ep_ll_dispatch_int8(shape, x.cuda(), idx.cuda(), slot.cuda(), cap, q, s, info, status)
    assert ep.ep_sync_status(status) == ep.EP_OK
    wq, wscale = ref.cast_rows(flat)
    want_q = torch.full((E, cap, H), 99, dtype=torch.int8)
    want_s, want_info = torch.full((E, cap), 7.0), torch.full((E, cap, 2), -5, dtype=torch.int32)
    for t in range(R * T):
        for k in range(K):
            e, r = int(idx.view(-1, K)[t, k]), int(slot.view(-1, K)[t, k])
            if e < 0 or r < 0:
                continue
            want_q[e, r], want_s[e, r], want_info[e, r] = wq[t], wscale[t], torch.tensor([t // T, t % T])
    assert torch.equal(q.cpu(), want_q)
    assert torch.equal(torch.nan_to_num(s.cpu(), nan=-1.0), torch.nan_to_num(want_s, nan=-1.0))
    assert torch.equal(info.cpu(), want_info)
    q.fill_(99)
    ep.ep_ll_dispatch_int8(shape, x.cuda(), idx.cuda(), slot.cuda(), cap, q, s, None, status)  # without source info
    assert torch.equal(q.cpu(), want_q)


def test_dispatch_skips_ids_and_positions_out_of_range():
    shape = ep.EpShape.make(1, 4, 2, 4, 16, 1)
    idx = torch.tensor([[[4, 1], [-7, 2], [1 << 40, 3], [0, 0]]])
    slot = torch.tensor([[[0, 2], [0, 9], [1, -2], [0, 1]]], dtype=torch.int32)
    q = torch.full((4, 2, 16), 99, dtype=torch.int8, device="cuda")
    s = torch.full((4, 2), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.ep_ll_dispatch_int8(shape, torch.ones(1, 4, 16, dtype=BF16, device="cuda"), idx.cuda(), slot.cuda(), 2, q, s, None,
                           status)
    assert ep.ep_sync_status(status) == ep.EP_OK
    assert (q[0] == 127).all() and (q[1:] == 99).all() and (s[1:] == 7.0).all()
