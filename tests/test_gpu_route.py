"""ep_route and ep_route_backward against float64 references.

Tolerances, fixed before the first run: |logits| <= 40, so l - max (or -l) has
a rounding of at most 80 * 2^-24 that exp turns into a relative error, expf and
the divisions add a few ulp and the sums at most log2(E) + 32 roundings more:
80 + 13 + 32 + 8 < 168 roundings of 2^-24 = 1e-5 relative.  Gradients are sums
of two such terms of size scale * max|g|.  bf16 gradients add 2^-8 relative."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import moe_ref
from combine_get_dispatch_notify_gb300 import ep

pytestmark = pytest.mark.gpu

RTOL = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.lib()


def logits_of(R, T, E, dtype, seed, special=None):
    g = torch.Generator().manual_seed(seed)
    l = torch.round(torch.randn(R, T, E, generator=g) * 2 * 64) / 64  # ties on purpose
    flat = l.view(-1, E)
    if special is not None and flat.shape[0]:
        for t in range(flat.shape[0]):
            special(flat, t, g)
    l = l.to(dtype)
    return l


def run_route(logits, bias, K, status=None, **kw):
    R, T, E = logits.shape
    sh = ep.EpShape.make(R, T, K, E, 8, 1)
    cfg = ep.EpRoute.make(kw["score"], kw.get("G", 1), kw.get("topk_groups", 1), kw.get("group_top", 1),
                          kw.get("renorm", True), kw.get("scale", 1.0))
    idx = torch.full((R, T, K), -7, dtype=torch.int64, device="cuda")
    w = torch.full((R, T, K), -7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda") if status is None else status
    ep.ep_route(sh, cfg, logits.cuda(), None if bias is None else bias.cuda(), idx, w, status)
    return idx.cpu(), w.cpu(), ep.ep_sync_status(status)


def check_route(logits, bias, K, want_status=ep.EP_OK, **kw):
    idx, w, rc = run_route(logits, bias, K, **kw)
    assert rc == want_status
    ridx, rw = moe_ref.route(logits, bias, K, **kw)
    assert np.array_equal(idx.view(-1, K).numpy(), ridx)
    np.testing.assert_allclose(w.view(-1, K).double().numpy(), rw, rtol=RTOL, atol=1e-37)


SHAPES = [  # R, T, E, K
    (1, 1, 1, 1), (1, 1, 8, 3), (2, 5, 16, 2), (3, 7, 33, 5), (16, 1, 256, 8), (4, 33, 256, 8), (1, 17, 160, 6),
    (1, 9, 384, 8), (2, 3, 512, 32), (1, 4, 513, 7), (1, 3, 1000, 16), (1, 2, 8192, 8), (8, 0, 64, 4),
    (1, 6, 24, 24), (1, 70, 72, 1),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_route_plain_selection(shape, score, dtype):
    R, T, E, K = shape
    check_route(logits_of(R, T, E, dtype, 1), None, K, score=score, renorm=E % 2 == 0, scale=1.5)


GROUPS = [  # R, T, E, K, G, topk_groups, group_top
    (16, 1, 256, 8, 8, 4, 2), (2, 19, 256, 8, 8, 4, 1), (1, 11, 64, 8, 8, 1, 2), (1, 13, 160, 6, 8, 3, 1),
    (3, 5, 72, 4, 4, 2, 2), (1, 5, 96, 3, 32, 5, 2), (1, 3, 1024, 8, 16, 4, 2), (1, 4, 640, 9, 5, 2, 2),
    (1, 5, 32, 2, 32, 7, 1), (1, 5, 256, 8, 8, 8, 2), (1, 3, 30, 4, 3, 2, 2),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True], ids=["plain", "bias"])
@pytest.mark.parametrize("case", GROUPS, ids=str)
def test_route_groups_and_bias(case, biased, score, dtype):
    R, T, E, K, G, tg, gt = case
    # bias steps of 1/32 and logits steps of 1/64: keys differ by far more than a rounding, or are
    # equal scores of equal logits under equal biases
    bias = torch.round(torch.randn(E, generator=torch.Generator().manual_seed(3)) * 8) / 32 if biased else None
    check_route(logits_of(R, T, E, dtype, 2), bias, K, score=score, G=G, topk_groups=tg, group_top=gt, scale=2.5)


def _mask_some(value):
    def f(flat, t, g):
        n = flat.shape[1]
        keep = t % (n + 1)  # 0 .. n experts stay
        flat[t, torch.randperm(n, generator=g)[keep:]] = value
    return f


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("mask", ["-inf", "lowest"])
def test_route_masked_experts_and_empty_rows(mask, score, dtype):
    value = -float("inf") if mask == "-inf" else torch.finfo(dtype).min
    l = logits_of(2, 40, 16, dtype, 4, _mask_some(value))
    for kw in (dict(), dict(G=4, topk_groups=2, group_top=2), dict(renorm=False, G=4, topk_groups=2)):
        check_route(l, None, 4, score=score, **kw)
        check_route(l, torch.linspace(-0.5, 0.5, 16), 4, score=score, **kw)
    idx, w, _ = run_route(l, None, 4, score=score)
    empty = idx.view(-1, 4)[0]  # row 0 keeps no expert
    assert (empty == -1).all() and (w.view(-1, 4)[0] == 0).all()


def test_route_infinite_logits_and_bias():
    l = logits_of(1, 12, 16, torch.float32, 5)
    l[0, 0, 3] = float("inf")
    l[0, 1, 3] = l[0, 1, 9] = float("inf")
    l[0, 2, :] = float("inf")
    check_route(l, None, 4, score="softmax")
    check_route(l, None, 4, score="sigmoid", renorm=False)
    bias = torch.zeros(16)
    bias[2], bias[7] = -float("inf"), float("inf")
    check_route(l, bias, 4, score="sigmoid")


def test_route_nan_is_masked_and_reported():
    l = logits_of(2, 6, 16, torch.float32, 6)
    l[1, 2, 5] = float("nan")
    check_route(l, None, 4, want_status=ep.EP_ERR_INPUT, score="softmax")
    check_route(l, None, 4, want_status=ep.EP_ERR_INPUT, score="sigmoid", G=4, topk_groups=2, group_top=2)
    l[1, 2] = float("nan")
    idx, w, rc = run_route(l, None, 4, score="softmax")
    assert rc == ep.EP_ERR_INPUT and (idx[1, 2] == -1).all() and (w[1, 2] == 0).all()
    bias = torch.zeros(16)
    bias[3] = float("nan")
    check_route(logits_of(1, 4, 16, torch.float32, 6), bias, 4, want_status=ep.EP_ERR_INPUT, score="sigmoid")


def test_route_scores_that_vanish():
    """Sigmoid scores that underflow: weights 0, not NaN; softmax scores far below the row's
    largest, kept only by the bias, still renormalise."""
    l = torch.full((1, 2, 8), -200.0)
    idx, w, rc = run_route(l, None, 3, score="sigmoid")
    assert rc == ep.EP_OK and torch.isfinite(w).all() and (w == 0).all()
    assert torch.equal(idx, torch.tensor([0, 1, 2]).expand(1, 2, 3))
    l = torch.zeros(1, 1, 8)
    l[0, 0, 0] = 300.0
    l[0, 0, 4:] = torch.tensor([1.0, 2.0, 3.0, 4.0])
    bias = torch.tensor([-9.0] * 4 + [9.0, 8.0, 7.0, 6.0])
    idx, w, _ = run_route(l, bias, 4, score="softmax")
    assert idx.flatten().tolist() == [4, 5, 6, 7]
    np.testing.assert_allclose(w.flatten().double(), torch.softmax(torch.tensor([1., 2, 3, 4]).double(), 0), rtol=RTOL)


def test_route_on_another_stream_and_repeated_calls_agree():
    l = logits_of(2, 300, 64, torch.float32, 7).cuda()
    sh, cfg = ep.EpShape.make(2, 300, 4, 64, 8, 1), ep.EpRoute.make("sigmoid", 8, 3, 2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = []
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side, side):
        idx = torch.empty(2, 300, 4, dtype=torch.int64, device="cuda")
        w = torch.empty(2, 300, 4, device="cuda")
        torch.cuda.synchronize()
        ep.ep_route(sh, cfg, l, None, idx, w, status, stream=stream)
        torch.cuda.synchronize()
        outs.append((idx, w))
    for idx, w in outs[1:]:
        assert torch.equal(idx, outs[0][0]) and torch.equal(w, outs[0][1])


# ------------------------------------------------------------------ backward
def run_backward(logits, idx, g, score, renorm, scale):
    R, T, E = logits.shape
    K = idx.shape[-1]
    sh = ep.EpShape.make(R, T, K, E, 8, 1)
    cfg = ep.EpRoute.make(score, renormalize=renorm, scale=scale)
    d = torch.full_like(logits, 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.ep_route_backward(sh, cfg, logits.cuda(), idx.cuda(), g.cuda(), d, status)
    return d.cpu(), ep.ep_sync_status(status)


def check_backward(logits, idx, g, score, renorm, scale, want_status=ep.EP_OK):
    d, rc = run_backward(logits, idx, g, score, renorm, scale)
    assert rc == want_status
    want = moe_ref.route_backward(logits, idx.clamp(min=-1), g, score, renorm, scale)
    rel = 2.0 ** -8 if logits.dtype == torch.bfloat16 else RTOL
    atol = 4 * RTOL * scale * float(g.abs().max()) if g.numel() else 0.0
    np.testing.assert_allclose(d.double().numpy(), want.numpy(), rtol=rel, atol=atol)
    return d, want


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("renorm", [False, True], ids=["plain", "renorm"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward_matches_formula(shape, score, renorm, dtype):
    R, T, E, K = shape
    l = logits_of(R, T, E, dtype, 8)
    gen = torch.Generator().manual_seed(9)
    idx = torch.rand(R, T, E, generator=gen).argsort(-1)[..., :K].contiguous()
    if T > 1:
        idx[:, 1, K // 2:] = -1
    if T > 2:
        idx[:, 2] = -1  # a row that kept nothing
    g = torch.randn(R, T, K, generator=gen)
    d, _ = check_backward(l, idx, g, score, renorm, 2.5)
    if T > 2:
        assert (d[:, 2] == 0).all()


@pytest.mark.parametrize("renorm", [False, True], ids=["plain", "renorm"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_backward_matches_differences_of_the_forward(score, renorm):
    """Central differences of the float64 weights: error h^2 / 6 * |f'''| (third derivatives of
    the scores are below 1) plus 2^-52 / h, with h = 1e-4 below 1e-8 per unit of gradient."""
    R, T, E, K = 1, 5, 24, 6
    l = logits_of(R, T, E, torch.float32, 10)
    idx, _ = moe_ref.route(l, None, K, score)
    idx = torch.from_numpy(idx).view(R, T, K)
    g = torch.randn(R, T, K, generator=torch.Generator().manual_seed(11))
    d, _ = run_backward(l, idx, g, score, renorm, 1.5)
    ok = torch.ones(R, T, E, dtype=torch.bool)
    h, num = 1e-4, torch.zeros(R, T, E, dtype=torch.float64)
    for e in range(E):
        step = torch.zeros(E, dtype=torch.float64)
        step[e] = h
        up = (moe_ref.weights_of(l.double() + step, ok, idx, score, renorm, 1.5) * g).sum(-1)
        dn = (moe_ref.weights_of(l.double() - step, ok, idx, score, renorm, 1.5) * g).sum(-1)
        num[..., e] = (up - dn) / (2 * h)
    np.testing.assert_allclose(d.double().numpy(), num.numpy(), rtol=RTOL, atol=4 * RTOL * 1.5 * float(g.abs().max()))


@pytest.mark.parametrize("renorm", [False, True], ids=["plain", "renorm"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_backward_masks_repeats_and_bad_ids(score, renorm):
    l = logits_of(1, 9, 16, torch.float32, 12)
    l[0, 0, 3:] = -float("inf")
    l[0, 1, :] = -float("inf")
    l[0, 2, 5] = float("inf")
    gen = torch.Generator().manual_seed(13)
    idx = torch.rand(1, 9, 16, generator=gen).argsort(-1)[..., :4].contiguous()
    idx[0, 0] = torch.tensor([0, 1, 2, -1])
    idx[0, 1] = -1
    idx[0, 2] = torch.tensor([5, 1, -1, -1])
    idx[0, 3] = torch.tensor([7, 7, 2, 7])  # a repeated expert's slots add up
    g = torch.randn(1, 9, 4, generator=gen)
    d, _ = check_backward(l, idx, g, score, renorm, 1.0)
    assert torch.isfinite(d).all()
    bad = idx.clone()
    bad[0, 4, 1], bad[0, 5, 0] = 16, -5
    clean = bad.clone()
    clean[0, 4, 1], clean[0, 5, 0] = -1, -1
    got, rc = run_backward(l, bad, g, score, renorm, 1.0)
    want, ok = run_backward(l, clean, g, score, renorm, 1.0)
    assert rc == ep.EP_ERR_INPUT and ok == ep.EP_OK and torch.equal(got, want)


@pytest.mark.parametrize("E,G,tg,gt,K", [(130, 13, 5, 2, 9), (45, 9, 4, 1, 3), (217, 7, 3, 2, 17), (31, 1, 1, 1, 12),
                                         (390, 6, 2, 2, 8), (511, 1, 1, 1, 8), (66, 33 // 11, 2, 2, 32)], ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_route_groups_of_any_size(E, G, tg, gt, K, dtype):
    bias = torch.round(torch.randn(E, generator=torch.Generator().manual_seed(5)) * 8) / 32
    l = logits_of(1, 29, E, dtype, 6, _mask_some(-float("inf")))
    l[0, 5:] = logits_of(1, 24, E, dtype, 7)[0]
    for score in ("sigmoid", "softmax"):
        check_route(l, None, K, score=score, G=G, topk_groups=tg, group_top=1)
    check_route(l, bias, K, score="sigmoid", G=G, topk_groups=tg, group_top=gt)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_route_close_keys_keep_their_exact_order(dtype):
    """Keys a few ulp apart, below what a cut or an approximate key can tell: the order is the exact
    sigmoid's (fp32, as 1 / (1 + exp(-l)) rounds), ties to the lowest index."""
    g = torch.Generator().manual_seed(8)
    l = (2.0 + torch.randint(-40, 40, (1, 64, 256), generator=g) * 2.0 ** -22).to(dtype)
    bias = torch.randint(-3, 4, (256,), generator=g) * 2.0 ** -23
    idx, _, rc = run_route(l, bias, 8, score="sigmoid", G=8, topk_groups=4, group_top=2)
    s = (1.0 / (1.0 + torch.exp(-l.float().cuda())) + bias.cuda()).cpu()
    per = s.view(64, 8, 32)
    two = per.sort(dim=-1, descending=True).values[..., :2].sum(-1)
    keep = two.sort(dim=-1, descending=True, stable=True).indices[:, :4]
    mask = torch.zeros(64, 8, dtype=torch.bool).scatter_(1, keep, True)
    key = torch.where(mask.unsqueeze(-1), per, -9.0).view(64, 256)
    want = key.sort(dim=-1, descending=True, stable=True).indices[:, :8]
    assert rc == ep.EP_OK and torch.equal(idx.view(64, 8), want)


@pytest.mark.parametrize("E,G,tg,gt,K", [(1536, 8, 1, 1, 3), (2080, 13, 4, 2, 8), (576, 8, 7, 2, 31), (4096, 32, 5, 1, 6)],
                         ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_route_many_experts(E, G, tg, gt, K, dtype):
    bias = torch.round(torch.randn(E, generator=torch.Generator().manual_seed(5)) * 8) / 32
    l = logits_of(1, 9, E, dtype, 6, _mask_some(-float("inf")))
    l[0, 5:] = logits_of(1, 4, E, dtype, 7)[0]
    for score in ("sigmoid", "softmax"):
        check_route(l, None, K, score=score, G=G, topk_groups=tg, group_top=1)
    check_route(l, bias, K, score="sigmoid", G=G, topk_groups=tg, group_top=gt)


@pytest.mark.parametrize("E,K,bias,score", [(8, 2, False, "softmax"), (64, 8, True, "sigmoid"), (40, 5, True, "softmax"),
                                            (640, 4, False, "softmax"), (33, 17, False, "sigmoid"),
                                            (384, 8, False, "softmax")], ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_long_calls_repeat_short_ones(E, K, bias, score, dtype):
    """More tokens than the GPU holds warps for, ending in part of a warp's tokens: every token's
    results are those of a call of 61 tokens, bit for bit, forward and backward."""
    short, times = 61, 2201  # 134261 tokens
    base = logits_of(1, short, E, dtype, 11)
    b = torch.randn(E, generator=torch.Generator().manual_seed(12)) if bias else None
    idx, w, rc = run_route(base, b, K, score=score, renorm=False)
    many_idx, many_w, many_rc = run_route(base.repeat(1, times, 1), b, K, score=score, renorm=False)
    assert rc == many_rc == ep.EP_OK
    assert torch.equal(many_idx, idx.repeat(1, times, 1)) and torch.equal(many_w, w.repeat(1, times, 1))
    g = torch.randn(1, short, K, generator=torch.Generator().manual_seed(13))
    idx[0, 7, 0], idx[0, 11] = -1, idx[0, 11, :1]  # an empty slot, and one expert in every slot
    for renorm in (False, True):
        d, rc = run_backward(base, idx, g, score, renorm, 1.5)
        many, many_rc = run_backward(base.repeat(1, times, 1), idx.repeat(1, times, 1), g.repeat(1, times, 1), score,
                                     renorm, 1.5)
        assert rc == many_rc == ep.EP_OK and torch.equal(many, d.repeat(1, times, 1))


@pytest.mark.parametrize("E,K", [(48, 6), (256, 8), (512, 20), (300, 8), (384, 3)], ids=str)
def test_route_bf16_sigmoids_that_coincide(E, K):
    """Large and tiny bf16 logits whose fp32 sigmoids are equal or a few ulp apart: the order is the
    sigmoids', ties to the lowest index, not the logits'."""
    g = torch.Generator().manual_seed(14)
    scale = torch.tensor([2.0 ** -14, 2.0 ** -9, 1.0, 11.0, 30.0, 100.0])
    l = torch.randn(1, 240, E, generator=g) * scale[torch.arange(240) % 6].view(1, 240, 1)
    l[0, ::7] = -l[0, ::7].abs()       # only the negative side
    l = l.to(torch.bfloat16)
    idx, _, rc = run_route(l, None, K, score="sigmoid")
    s = (1.0 / (1.0 + torch.exp(-l.float().cuda()))).cpu().view(240, E)
    want = s.sort(dim=-1, descending=True, stable=True).indices[:, :K]
    assert rc == ep.EP_OK and torch.equal(idx.view(240, K), want)
