"""Gradients and weights of the router where a bound relative to the row's largest element, or
logits of ordinary size, would not show an error.  References and bounds in float64; each
test derives its own."""
from __future__ import annotations

import pytest
import torch

import moe_ref
from combine_get_dispatch_notify_gb300 import ep
from test_gpu_route import RTOL, SHAPES, logits_of, run_backward, run_route

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.lib()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("E,K,lo,hi,size", [(64, 2, -88.5, -88.0, 2.0), (64, 2, -80.0, -76.0, 65536.0),
                                            (256, 8, -88.5, -70.0, 3e4), (34, 17, -88.5, -84.0, 1.0),
                                            (48, 32, -87.0, -20.0, 1e3)], ids=str)
def test_backward_of_renormalised_sigmoids_that_are_all_small(E, K, lo, hi, size, dtype):
    """Every kept score far below 1, down to where it is no normal fp32 number, and incoming gradients
    as a scaled loss has them: the weights s / sum(s) are ordinary numbers, and so is their gradient.

    With d the error of a score (expf 2 ulp, an addition, a division, 2^-22 more where it is
    subnormal: below 2^-20), a weight v is off by 2 d + 2^-24, a sum of K terms by K 2^-24 more, and
    what is left are four roundings: below (4 + 1) 2^-20 + (K + 6) 2^-24 < 2^-16.5 of v (|g| + sum v |g|)."""
    R, T, scale = 2, 40, 2.5
    gen = torch.Generator().manual_seed(21)
    l = (torch.rand(R, T, E, generator=gen) * (hi - lo) + lo).mul(2).round().div(2).to(dtype)  # exact in bf16 too
    idx = torch.rand(R, T, E, generator=gen).argsort(-1)[..., :K].contiguous()
    g = torch.randn(R, T, K, generator=gen) * size
    d, rc = run_backward(l, idx, g, "sigmoid", True, scale)
    assert rc == ep.EP_OK
    want = moe_ref.route_backward(l, idx, g, "sigmoid", True, scale)
    s = torch.sigmoid(l.double()).gather(-1, idx)
    v = s / s.sum(-1, keepdim=True)
    size_k = v * (g.double().abs() + (v * g.double().abs()).sum(-1, keepdim=True)) * scale
    bound = torch.zeros(R, T, E, dtype=torch.float64).scatter_(-1, idx, size_k * 2.0 ** -16.5)
    if dtype == torch.bfloat16:
        bound = bound + want.abs() * 2.0 ** -8
    assert torch.isfinite(d).all()
    assert ((d.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("renorm", [False, True], ids=["plain", "renorm"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("E,K", [(64, 8), (40, 16), (256, 1), (64, 32)], ids=str)
def test_backward_of_sigmoids_near_one(E, K, dtype, renorm):
    """s (1 - s) keeps its digits where s is near 1 in fp32, or 1: 1 - s is exp(-l) s.

    exp(-l) is within 2^-22, s and s exp(-l) within 2^-20 with their roundings, a weight within 2^-19
    (its sum of K terms K 2^-24 more), what it multiplies within (K + 4) 2^-24 of |g| + sum v |g|:
    together below 2^-18 + K 2^-23 < 2^-16.9 of v (1 - s) (|g| + sum v |g|)."""
    R, T, scale = 2, 40, 2.5
    gen = torch.Generator().manual_seed(26)
    l = (torch.rand(R, T, E, generator=gen) * 44 - 4).mul(4).round().div(4).to(dtype)  # exact in bf16 too
    idx = torch.rand(R, T, E, generator=gen).argsort(-1)[..., :K].contiguous()
    g = torch.randn(R, T, K, generator=gen)
    d, rc = run_backward(l, idx, g, "sigmoid", renorm, scale)
    assert rc == ep.EP_OK
    k, gd = l.double().gather(-1, idx), g.double() * scale
    s = 1 / (1 + torch.exp(-k))
    rest = 1 / (1 + torch.exp(k))  # 1 - s
    v = s / s.sum(-1, keepdim=True) if renorm else s
    dot = (v * gd).sum(-1, keepdim=True) if renorm else 0.0
    mag = (v * gd.abs()).sum(-1, keepdim=True) if renorm else 0.0
    zeros = torch.zeros(R, T, E, dtype=torch.float64)
    want = zeros.scatter(-1, idx, v * rest * (gd - dot))
    bound = zeros.scatter(-1, idx, v * rest * (gd.abs() + mag) * 2.0 ** -16.9)
    if dtype == torch.bfloat16:
        bound = bound + want.abs() * 2.0 ** -8
    assert ((d.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("R,T,E", [(1, 33, 16), (2, 37, 32), (1, 9, 64), (1, 70, 72), (2, 61, 128), (1, 5, 130),
                                   (4, 65, 256), (1, 21, 300), (1, 17, 384), (2, 33, 512), (1, 5, 1000)], ids=str)
def test_backward_of_scores_far_below_the_largest(R, T, E):
    """One expert holds the row and is kept; the others' gradients are -exp(l_e - max) g.  They are as
    exact as an fp32 exponential: l_e - max is a multiple of 2^-10 (no rounding), the sum is 1 and
    the largest score is 1, so expf's 2 ulp (2^-22) and at most six roundings (2^-24) remain: 2^-21.
    A gradient below 2^-126 is a multiple of 2^-149, and so off by up to one of those."""
    gen = torch.Generator().manual_seed(22)
    l = -(torch.rand(R, T, E, generator=gen) * 45 + 40).mul(1024).round().div(1024)  # -40 to -85
    top = torch.randint(0, E, (R, T, 1), generator=gen)
    l.scatter_(-1, top, torch.randint(-3, 4, (R, T, 1), generator=gen).float() / 4)
    g = torch.randn(R, T, 1, generator=gen)
    d, rc = run_backward(l, top, g, "softmax", False, 1.5)
    assert rc == ep.EP_OK
    diff = (l - l.gather(-1, top)).double()
    want = -torch.exp(diff) * (g.double() * 1.5)
    others = torch.ones(R, T, E, dtype=torch.bool).scatter_(-1, top, False)
    assert ((d.double() - want).abs() <= want.abs() * 2.0 ** -21 + 2.0 ** -149)[others].all()
    assert (d.gather(-1, top).abs() <= g.abs() * 1.5 * 2.0 ** -21).all()  # s (1 - s) g with s = 1


@pytest.mark.parametrize("renorm", [False, True], ids=["plain", "renorm"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_weights_of_equal_logits_are_the_nearest_numbers(dtype, renorm):
    """Equal logits: every exponential is 1 and their sum a whole number n, so the one rounding is the
    division's, and each weight is the fp32 number nearest to 1 / n."""
    for E in range(2, 513, 2):
        K = min(E, 32) if renorm else 1
        for k in ({K, max(1, K - E // 2 % 32)} if renorm else {1}):
            idx, w, rc = run_route(torch.full((1, 1, E), 0.75, dtype=dtype), None, k, score="softmax", renorm=renorm)
            assert rc == ep.EP_OK and idx.flatten().tolist() == list(range(k))
            n = k if renorm else E
            assert (w == torch.tensor(1.0) / torch.tensor(float(n))).all(), (E, k)


def gradient_and_sizes(logits, idx, g, score, renorm, scale):
    """(gradient, magnitude of what each element is the sum of) from the formulas, float64 [R, T, E]."""
    l, ok = moe_ref.masked_logits(logits)
    l, ok = torch.from_numpy(l), torch.from_numpy(ok)
    on = (idx >= 0) & ok.gather(-1, idx.clamp(min=0))
    at = idx.clamp(min=0)
    k, g = l.gather(-1, at), torch.where(on, g.double() * scale, 0.0)
    p = torch.softmax(torch.where(ok, l, -1e300), -1)
    if score == "softmax" and renorm:
        s, rest = torch.softmax(torch.where(on, k, -1e300), -1) * on, 1.0
    elif score == "softmax":
        s, rest = p.gather(-1, at) * on, 1.0
    else:
        s, rest = on / (1 + torch.exp(-k)), 1 / (1 + torch.exp(k))
    dot = mag = 0.0
    if renorm:
        total = s.sum(-1, keepdim=True)
        s = torch.where(total > 0, s / total.clamp(min=1e-300), 0.0)
        dot, mag = (s * g).sum(-1, keepdim=True), (s * g).abs().sum(-1, keepdim=True)
    zeros = torch.zeros_like(l)
    grad = zeros.scatter_add(-1, at, s * rest * (g - dot) * on)
    size = zeros.scatter_add(-1, at, s * rest * (g.abs() + mag) * on)
    if score == "softmax" and not renorm:
        grad = grad - p * (s * g).sum(-1, keepdim=True)
        size = size + p * (s * g).abs().sum(-1, keepdim=True)
    return grad, size


@pytest.mark.parametrize("pick", ["largest", "any"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("renorm", [False, True], ids=["plain", "renorm"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shape", SHAPES + [(1, 37, 64, 8), (2, 29, 48, 6), (1, 33, 128, 12), (1, 21, 300, 8)], ids=str)
def test_every_gradient_element_is_held_to_its_own_size(shape, score, renorm, dtype, pick):
    """An element's error is bounded by RTOL of the terms that it is the sum of, not of the row's
    largest: with many experts the dense softmax part is far below that one everywhere."""
    R, T, E, K = shape
    l = logits_of(R, T, E, dtype, 23)
    gen = torch.Generator().manual_seed(24)
    order = l.float() if pick == "largest" else torch.rand(R, T, E, generator=gen)
    idx = order.argsort(-1, descending=True)[..., :K].contiguous()
    if T > 1 and K > 1:
        idx[:, 1, K // 2:] = -1
    g = torch.randn(R, T, K, generator=gen)
    d, rc = run_backward(l, idx, g, score, renorm, 2.5)
    assert rc == ep.EP_OK
    want, size = gradient_and_sizes(l, idx, g, score, renorm, 2.5)
    bound = RTOL * size
    if dtype == torch.bfloat16:
        bound = bound + want.abs() * 2.0 ** -8
    assert ((d.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("E,K", [(24, 6), (64, 8), (130, 3)], ids=str)
@pytest.mark.parametrize("renorm", [False, True], ids=["plain", "renorm"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_every_gradient_element_matches_differences_of_the_forward(score, renorm, E, K):
    """Central differences of the float64 weights with h = 2^-16: h^2 / 6 times third derivatives (below
    2 for a weight) and roundings of 2^-52 / h are each below 1e-10 per unit of scale * sum |g|."""
    R, T = 1, 7
    l = logits_of(R, T, E, torch.float32, 27)
    gen = torch.Generator().manual_seed(28)
    idx = l.argsort(-1, descending=True)[..., :K].contiguous()
    idx[:, 3:] = torch.rand(R, T - 3, E, generator=gen).argsort(-1)[..., :K]
    g = torch.randn(R, T, K, generator=gen)
    d, rc = run_backward(l, idx, g, score, renorm, 1.5)
    assert rc == ep.EP_OK
    ok = torch.ones(R, T, E, dtype=torch.bool)
    h, num = 2.0 ** -16, torch.zeros(R, T, E, dtype=torch.float64)
    for e in range(E):
        step = torch.zeros(E, dtype=torch.float64)
        step[e] = h
        up = (moe_ref.weights_of(l.double() + step, ok, idx, score, renorm, 1.5) * g).sum(-1)
        dn = (moe_ref.weights_of(l.double() - step, ok, idx, score, renorm, 1.5) * g).sum(-1)
        num[..., e] = (up - dn) / (2 * h)
    _, size = gradient_and_sizes(l, idx, g, score, renorm, 1.5)
    bound = RTOL * size + 2e-10 * 1.5 * g.double().abs().sum(-1, keepdim=True)
    assert ((d.double() - num).abs() <= bound).all()
