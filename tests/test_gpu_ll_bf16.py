"""Experts' bf16 products and their gradients against float64, at the sizes and row counts where
tiles, blocks and experts end; rows behind an expert's count hold NaN and have to be ignored and
left alone."""
from __future__ import annotations

import pytest
import torch

import experts_ref as ref
from combine_get_dispatch_notify_gb300 import ep

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
POISON = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.lib()


# n, k, capacity, rows of each expert (None: capacity)
SHAPES = {
    "smallest": (8, 8, 3, [1, 0, 3]),
    "one_row": (128, 64, 1, [1, 0, 1, 1]),
    "odd": (40, 24, 20, [17, 16, 15, 0, 20]),
    "past_a_block": (72, 136, 70, [63, 64, 65, 1]),
    "past_a_tile": (264, 200, 130, [127, 128, 129, 2]),
    "two_tiles": (136, 72, 300, [255, 256, 257, 300, 31, 33]),
    "rows_ten_tiles": (520, 328, 700, [700, 513, 0, 511]),
    "wide": (2056, 64, 40, [33, 40]),
    "deep": (64, 4104, 40, [33, 40]),
    "counts_past_the_capacity": (64, 64, 10, [11, 1 << 30, -1, -(1 << 31), 10]),
    "all_empty": (48, 40, 16, [0, 0, 0]),
    "many_experts": (24, 40, 9, [i % 10 for i in range(300)]),
    "many_tiles_of_all_sizes": (264, 72, 300, [255, 256, 257, 300, 31, 33, 129, 0] * 20),
    "many_longer_experts": (24, 40, 140, [i * 7 % 141 for i in range(300)]),
    "more_tiles_than_sms": (1032, 64, 520, [520] * 24),
}


def rows_of(name):
    n, k, cap, counts = SHAPES[name]
    return n, k, cap, counts, [min(max(c, 0), cap) for c in counts]


def normal(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(BF16)


def poisoned(t, rows):
    """NaN and infinities behind each expert's rows."""
    t = t.clone()
    for e, m in enumerate(rows):
        t[e, m:] = POISON
        t[e, m::2] = float("inf")
    return t.cuda()


def call(fn, *args):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fn(*args, status)
    assert ep.ep_sync_status(status) == ep.EP_OK


def fresh(*shape, dtype=BF16):
    return torch.full(shape, 7.0, dtype=dtype, device="cuda")


def untouched(t, rows):
    for e, m in enumerate(rows):
        assert (t[e, m:] == 7.0).all(), f"expert {e}: rows behind its {m} were written"


def dev(counts):
    return torch.tensor(counts, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("name", sorted(SHAPES))
def test_product(name):
    n, k, cap, counts, rows = rows_of(name)
    E = len(rows)
    a, w = normal(1, E, cap, k), normal(2, E, n, k, scale=k ** -0.5)
    y = fresh(E, cap, n)
    call(ep.ep_ll_gemm_bf16, poisoned(a, rows), w.cuda(), dev(counts), y)
    y = y.cpu()
    untouched(y, rows)
    for e, m in enumerate(rows):
        ref.close_bf16(f"y[{e}]", y[e, :m], *ref.product(a[e, :m], w[e]))


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("name", sorted(SHAPES))
def test_gated_product(name, keep):
    n, k, cap, counts, rows = rows_of(name)
    E = len(rows)
    a, w = normal(3, E, cap, k), normal(4, E, 2, n, k, scale=k ** -0.5)
    y, gu = fresh(E, cap, n), fresh(E, cap, 2, n) if keep else None
    call(ep.ep_ll_gemm_swiglu_bf16, poisoned(a, rows), w.cuda(), dev(counts), y, gu)
    y = y.cpu()
    untouched(y, rows)
    if keep:
        gu = gu.cpu()
        untouched(gu, rows)
    for e, m in enumerate(rows):
        h, dh, (g, u), (dg, du) = ref.gated(a[e, :m], w[e])
        ref.close_bf16(f"y[{e}]", y[e, :m], h, dh)
        if keep:
            ref.close_bf16(f"gate[{e}]", gu[e, :m, 0], g, dg)
            ref.close_bf16(f"up[{e}]", gu[e, :m, 1], u, du)


@pytest.mark.parametrize("name", sorted(SHAPES))
def test_rows_gradient(name):
    k, n, cap, counts, rows = rows_of(name)
    E = len(rows)
    gy, w = normal(5, E, cap, n), normal(6, E, n, k, scale=n ** -0.5)
    ga = fresh(E, cap, k)
    call(ep.ep_ll_gemm_dgrad_bf16, poisoned(gy, rows), w.cuda(), dev(counts), ga)
    ga = ga.cpu()
    untouched(ga, rows)
    for e, m in enumerate(rows):
        ref.close_bf16(f"grad_a[{e}]", ga[e, :m], *ref.product(gy[e, :m], w[e].T))


@pytest.mark.parametrize("name", sorted(SHAPES))
def test_activation_gradient(name):
    k, n, cap, counts, rows = rows_of(name)
    E = len(rows)
    gy, w = normal(7, E, cap, n), normal(8, E, n, k, scale=n ** -0.5)
    gu = normal(9, E, cap, 2, k, scale=3.0)
    out = fresh(E, cap, 2, k)
    call(ep.ep_ll_gemm_dswiglu_bf16, poisoned(gy, rows), w.cuda(), poisoned(gu, rows), dev(counts), out)
    out = out.cpu()
    untouched(out, rows)
    for e, m in enumerate(rows):
        gh, dgh = ref.product(gy[e, :m], w[e].T)
        want, bound = ref.gated_gradient(gh, dgh, gu[e, :m, 0], gu[e, :m, 1])
        for i, part in enumerate(("gate", "up")):
            ref.close_bf16(f"grad_{part}[{e}]", out[e, :m, i], want[i], bound[i])


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("name", sorted(SHAPES))
def test_weights_gradient(name, dtype):
    n, k, cap, counts, rows = rows_of(name)
    E = len(rows)
    gy, a = normal(10, E, cap, n), normal(11, E, cap, k)
    gw = fresh(E, n, k, dtype=dtype)
    call(ep.ep_ll_gemm_wgrad_bf16, poisoned(gy, rows), poisoned(a, rows), dev(counts), gw)
    gw = gw.cpu()
    close = ref.close_bf16 if dtype == BF16 else ref.close_fp32
    for e, m in enumerate(rows):
        close(f"grad_w[{e}]", gw[e], *ref.product(gy[e, :m].T, a[e, :m].T))
        if m == 0:
            assert (gw[e] == 0).all()


def test_weights_gradient_without_a_capacity():
    gw = fresh(2, 16, 24, dtype=torch.float32)
    none = torch.empty(2, 0, 16, dtype=BF16, device="cuda"), torch.empty(2, 0, 24, dtype=BF16, device="cuda")
    call(ep.ep_ll_gemm_wgrad_bf16, *none, dev([0, 5]), gw)
    assert (gw == 0).all()


def test_activation_at_its_ends():
    """Gates from -100 to 100, infinities among the weights: silu and its slope without overflow."""
    gates = torch.tensor([-100.0, -90.0, -88.0, -30.0, -1.28125, -0.0, 0.0, 1e-30, 1.0, 30.0, 88.0, 100.0, -3e38, 1e38, 2.0, 3.0])
    k, n = 16, 8
    a = torch.eye(k).to(BF16).unsqueeze(0)
    w = torch.zeros(1, 2, n, k, dtype=BF16)
    w[0, 0, 0] = gates.to(BF16)
    w[0, 1, 0] = 1.5
    y, gu = fresh(1, k, n), fresh(1, k, 2, n)
    call(ep.ep_ll_gemm_swiglu_bf16, a.cuda(), w.cuda(), dev([k]), y, gu)
    g = w[0, 0, 0].double()
    ref.close_bf16("silu", y[0, :, 0].cpu(), ref.silu(g) * 1.5, (ref.silu(g) * 1.5).abs() * 2.0 ** -20 + 2.0 ** -126)
    assert torch.equal(gu[0, :, 0, 0].cpu(), w[0, 0, 0])
    # the gradient from the same gates, gh = 1
    wd = torch.zeros(1, 8, n, dtype=BF16)
    wd[0, 0, 0] = 1.0
    gy = torch.zeros(1, k, 8, dtype=BF16)
    gy[..., 0] = 1.0
    out = fresh(1, k, 2, n)
    call(ep.ep_ll_gemm_dswiglu_bf16, gy.cuda(), wd.cuda(), gu, dev([k]), out)
    want, bound = ref.gated_gradient(torch.ones(k, dtype=torch.float64), torch.zeros(k, dtype=torch.float64), g,
                                     torch.full((k,), 1.5, dtype=torch.float64))
    for i in range(2):
        ref.close_bf16("slope", out[0, :, i, 0].cpu(), want[i], bound[i] + 2.0 ** -126)


def test_values_that_are_not_finite_stay_in_their_rows_and_columns():
    E, cap, n, k = 1, 40, 72, 80
    a, w = normal(12, E, cap, k), normal(13, E, n, k)
    a[0, 5, 7] = float("nan")
    w[0, 9, 3] = float("inf")
    y = fresh(E, cap, n)
    call(ep.ep_ll_gemm_bf16, a.cuda(), w.cuda(), dev([cap]), y)
    y = y.cpu()[0]
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[5], want[:, 9] = True, True
    assert torch.equal(bad, want)


def block_loss(x, w13, w2, r):
    g, u = x @ w13[0].T, x @ w13[1].T
    return ((ref.silu(g) * u) @ w2.T * r).sum()


def block(x, w13, w2, gy, gt=torch.float32):
    """Forward and backward of one expert's block through the calls: (y, grad_x, grad_w13, grad_w2)."""
    m, H = x.shape
    F = w13.shape[1]
    on = lambda t: t.to(BF16).unsqueeze(0).cuda()  # noqa: E731
    x, w13, w2, gy, count = on(x), on(w13), on(w2), on(gy), dev([m])
    inner, gu, y, ggu, gx = fresh(1, m, F), fresh(1, m, 2, F), fresh(1, m, H), fresh(1, m, 2, F), fresh(1, m, H)
    gw13, gw2 = fresh(1, 2 * F, H, dtype=gt), fresh(1, H, F, dtype=gt)
    call(ep.ep_ll_gemm_swiglu_bf16, x, w13, count, inner, gu)
    call(ep.ep_ll_gemm_bf16, inner, w2, count, y)
    call(ep.ep_ll_gemm_dswiglu_bf16, gy, w2, gu, count, ggu)
    call(ep.ep_ll_gemm_dgrad_bf16, ggu.view(1, m, 2 * F), w13.view(1, 2 * F, H), count, gx)
    call(ep.ep_ll_gemm_wgrad_bf16, ggu.view(1, m, 2 * F), x, count, gw13)
    call(ep.ep_ll_gemm_wgrad_bf16, gy, inner, count, gw2)
    return y[0].cpu(), gx[0].cpu(), gw13[0].view(2, F, H).cpu(), gw2[0].cpu()


@pytest.mark.parametrize("m,H,F", [(1, 8, 8), (37, 72, 40), (130, 136, 264)])
def test_block_gradient_against_differences(m, H, F):
    """Central differences of the loss sum(y r) along random directions.  Each gradient element is
    held to bf16 steps of itself and of what it was made from, so along a direction v the two differ
    by at most that distance times |v|; the differences are exact to 1e-5."""
    x, r = normal(20, m, H).double(), normal(21, m, H).double()
    w13, w2 = normal(22, 2, F, H, scale=H ** -0.5).double(), normal(23, H, F, scale=F ** -0.5).double()
    leaves = [t.clone().requires_grad_(True) for t in (x, w13, w2)]
    block_loss(*leaves, r).backward()
    _, *got = block(x, w13, w2, r)
    eps = 1e-4
    for i, (grad, exact) in enumerate(zip(got, [t.grad for t in leaves])):
        v = torch.randn(exact.shape, generator=torch.Generator().manual_seed(30 + i), dtype=torch.float64)
        args = lambda s: [t + (s * v if j == i else 0) for j, t in enumerate((x, w13, w2))]  # noqa: E731
        slope = (block_loss(*args(eps), r) - block_loss(*args(-eps), r)) / (2 * eps)
        exact_slope = (exact * v).sum()
        assert abs(slope - exact_slope) <= 1e-5 * (exact * v).abs().sum()
        # bf16 roundings on the way (gate and up, h or both their gradients, the result), each of random sign and at
        # most 2^-8 of an element: four of them bound the whole gradient's distance
        spread = (grad.double() - exact).norm() / exact.norm()
        assert spread <= 4 * ref.HALF, spread
        assert abs((grad.double() * v).sum() - slope) <= 4 * ref.HALF * exact.norm() * v.norm()


def run_all(stream=None):
    """(every call once on one stream, their outputs, the status word)."""
    n, k, cap, counts, rows = rows_of("two_tiles")
    E = len(rows)
    a, w = normal(40, E, cap, k).cuda(), normal(41, E, 2, n, k).cuda()
    gy, count, status = normal(42, E, cap, n).cuda(), dev(counts), torch.zeros(1, dtype=torch.int32, device="cuda")
    y, gu, y2, ga = fresh(E, cap, n), fresh(E, cap, 2, n), fresh(E, cap, n), fresh(E, cap, k)
    wd = normal(43, E, k, n).cuda()
    gyd, ggu = normal(44, E, cap, k).cuda(), fresh(E, cap, 2, n)
    gw = fresh(E, n, k, dtype=torch.float32)
    torch.cuda.synchronize()

    def calls():
        ep.ep_ll_gemm_swiglu_bf16(a, w, count, y, gu, status, stream)
        ep.ep_ll_gemm_bf16(a, w0, count, y2, status, stream)
        ep.ep_ll_gemm_dgrad_bf16(gy, w0, count, ga, status, stream)
        ep.ep_ll_gemm_dswiglu_bf16(gyd, wd, gu, count, ggu, status, stream)
        ep.ep_ll_gemm_wgrad_bf16(gy, a, count, gw, status, stream)

    w0 = w[:, 0].contiguous()
    torch.cuda.synchronize()
    return calls, [y, gu, y2, ga, ggu, gw], status


def test_two_runs_give_the_same_bits():
    outs = []
    for _ in range(2):
        calls, out, status = run_all()
        for _ in range(3):
            calls()
        assert ep.ep_sync_status(status) == ep.EP_OK
        outs.append([t.cpu() for t in out])
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_streams_and_graphs():
    """Two sets of calls on two streams at once, and one of them captured and replayed, give the bits
    of calls one after another."""
    calls, out, status = run_all()
    calls()
    assert ep.ep_sync_status(status) == ep.EP_OK
    want = [t.cpu() for t in out]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    (c1, o1, st1), (c2, o2, st2) = run_all(s1), run_all(s2)
    for _ in range(3):
        c1()
        c2()
    torch.cuda.synchronize()
    for o, st in ((o1, st1), (o2, st2)):
        assert ep.ep_sync_status(st) == ep.EP_OK
        for a, b in zip(o, want):
            assert torch.equal(a.cpu(), b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for t in out:
        t.fill_(7.0)
    graph.replay()
    graph.replay()
    assert ep.ep_sync_status(status) == ep.EP_OK
    for a, b in zip(out, want):
        assert torch.equal(a.cpu(), b)


def test_offsets_past_32_bits():
    """An expert whose rows and weights begin beyond 2^32 bytes and 2^31 elements."""
    E, cap, n, k = 3, 4096, 64, 1 << 18
    a = torch.zeros(E, cap, k, dtype=BF16, device="cuda")
    assert a.numel() > 1 << 31
    w = torch.zeros(E, n, k, dtype=BF16, device="cuda")
    pick = torch.arange(0, k, k // 16)
    rows = normal(50, 5, 16).cuda()
    weights = normal(51, n, 16).cuda()
    a[2, :5][:, pick.cuda()] = rows
    w[2][:, pick.cuda()] = weights
    y = fresh(E, cap, n)
    call(ep.ep_ll_gemm_bf16, a, w, dev([0, 0, 5]), y)
    want, bound = ref.product(rows.cpu(), weights.cpu())
    ref.close_bf16("y", y[2, :5].cpu(), want, bound)
    gw = torch.empty(E, n, k, dtype=BF16, device="cuda")
    gy = torch.zeros(E, cap, n, dtype=BF16, device="cuda")
    gy[2, :5] = normal(52, 5, n).cuda()
    call(ep.ep_ll_gemm_wgrad_bf16, gy, a, dev([0, 0, 5]), gw)
    want, bound = ref.product(gy[2, :5].cpu().T, rows.cpu().T)
    ref.close_bf16("grad_w", gw[2][:, pick.cuda()].cpu(), want, bound)
    assert int((gw[2] != 0).sum()) <= n * 16 and not gw[:2].any()


def test_binding_refuses_strided_and_mistyped_tensors():
    a, w, y = fresh(2, 8, 16), fresh(2, 24, 16), fresh(2, 8, 24)
    status, count = torch.zeros(1, dtype=torch.int32, device="cuda"), dev([1, 1])
    for bad in (fresh(2, 8, 32)[..., ::2], a.float(), a[:, :7], a.cpu()):
        with pytest.raises(ValueError):
            ep.ep_ll_gemm_bf16(bad, w, count, y, status)
    with pytest.raises(ValueError):
        ep.ep_ll_gemm_bf16(a, w, count.long(), y, status)
    with pytest.raises(ep.EpError):  # n is no multiple of 8
        ep.ep_ll_gemm_bf16(a, fresh(2, 20, 16), count, fresh(2, 8, 20), status)
    with pytest.raises(ep.EpError):  # off the 16-byte grid
        ep.ep_ll_gemm_bf16(fresh(2 * 8 * 16 + 1)[1:].view(2, 8, 16), w, count, y, status)
