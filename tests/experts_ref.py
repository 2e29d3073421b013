"""Plain float64 references of the experts' bf16 and int8 products, of their gradients and of the
combine's gradient, one expert at a time, with the bounds of fp32 sums beside them.

Bounds.  Products of two bf16 (or int8) values are exact in fp32.  A sum of k terms, in any order
and each addition off by at most one unit of the last place (2^-23 of the partial sum, so that a
truncating adder is covered too), is within k * 2^-23 of the sum of magnitudes.  A rounding to bf16
is off by 2^-8 of the value, and by half the smallest number (2^-134) near zero."""
from __future__ import annotations

import torch

HALF = 2.0 ** -8
TINY = 2.0 ** -134


def sum_error(k: int) -> float:
    return (k + 2) * 2.0 ** -23


def silu(g: torch.Tensor) -> torch.Tensor:
    return g * torch.sigmoid(g)


def product(a: torch.Tensor, w: torch.Tensor):
    """(a @ w^T, bound of its fp32 sums): a [m, k], w [n, k]."""
    a, w = a.double(), w.double()
    return a @ w.T, (a.abs() @ w.abs().T) * sum_error(a.shape[-1])


def gated(a, w):
    """(h, its bound, [gate, up], their bounds) of unrounded gate and up; w [2, n, k]."""
    (g, dg), (u, du) = product(a, w[0]), product(a, w[1])
    h = silu(g) * u
    # |silu'| <= 1.1; sixteen ulp for the activation itself
    return h, 1.1 * dg * (u.abs() + du) + silu(g).abs() * du + h.abs() * 2.0 ** -20, (g, u), (dg, du)


def gated_gradient(gh, dgh, gate, up):
    """((grad_gate, grad_up), their bounds) from gh with bound dgh."""
    gate, up = gate.double(), up.double()
    s = torch.sigmoid(gate)
    rest = torch.sigmoid(-gate)
    slope = s * (1 + gate * rest)
    return ((gh * up * slope, gh * gate * s),
            (dgh * (up * slope).abs() + gh.abs() * up.abs() * s * (1 + (gate * rest).abs()) * 2.0 ** -20,
             dgh * (gate * s).abs() + (gh * gate * s).abs() * 2.0 ** -20))


def close_bf16(name, got, want, bound) -> None:
    err = (got.double() - want).abs()
    tol = (want.abs() + bound) * HALF + bound + TINY
    bad = ~(err <= tol)  # a NaN is bad
    assert not bad.any(), f"{name}: {int(bad.sum())} off, first {bad.nonzero()[0].tolist()}, " \
                          f"got {got[bad][0]}, want {want[bad][0]}"


def close_fp32(name, got, want, bound) -> None:
    err = (got.double() - want).abs()
    bad = ~(err <= want.abs() * 2.0 ** -23 + bound + 2.0 ** -149)
    assert not bad.any(), f"{name}: {int(bad.sum())} off, first {bad.nonzero()[0].tolist()}, " \
                          f"got {got[bad][0]}, want {want[bad][0]}"


def cast_rows(x: torch.Tensor):
    """fp32 / bf16 [..., n] -> (int8, fp32 scales [...]) with fp32 arithmetic, bit for bit."""
    v = x.float()
    amax = v.abs().amax(-1)  # NaN wins
    scale = torch.where(amax == amax, amax.clamp(min=2.0 ** -100), amax) * torch.tensor(1 / 127, dtype=torch.float32)
    q = torch.round(v / scale.unsqueeze(-1))
    q = torch.where(torch.isfinite(amax).unsqueeze(-1), q, torch.zeros_like(q))
    return q.to(torch.int8), scale
