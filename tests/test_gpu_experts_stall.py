"""Waits of the experts' bf16 and int8 products that run out: reported as a timeout, with the context
usable and the next call right."""
from __future__ import annotations

import pytest
import torch

from combine_get_dispatch_notify_gb300 import ep

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
E, CAP, N, K = 12, 300, 528, 272
ROWS = [300, 0, 17, 129, 64, 300, 1, 33, 256, 300, 5, 200]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.lib()


def normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(BF16).cuda()


def zeros(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def check(call, stalled, outs, status, tile):
    call()
    assert ep.ep_sync_status(status) == ep.EP_OK
    want = [t.clone() for t in outs]
    stalled(0, tile, 20000)
    rc = ep.ep_sync_status(status)
    # every pair of these calls has its first tile; of the others only that the call ends is known here
    assert rc == ep.EP_ERR_TIMEOUT if tile == 0 else rc in (ep.EP_OK, ep.EP_ERR_TIMEOUT)
    status.zero_()
    call()
    assert ep.ep_sync_status(status) == ep.EP_OK
    for a, b in zip(outs, want):
        assert torch.equal(a, b)
    for t in outs:
        t.zero_()
    stalled(-1, 0, 2000000)  # nothing stalled
    assert ep.ep_sync_status(status) == ep.EP_OK
    for a, b in zip(outs, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("tile", [0, 1])
@pytest.mark.parametrize("form", range(6))
def test_bf16_products(form, tile):
    count, status = torch.tensor(ROWS, dtype=torch.int32, device="cuda"), zeros(1, dtype=torch.int32)
    a, gy = normal(1, E, CAP, K), normal(2, E, CAP, N)
    w, w2, gu = normal(3, E, N, K), normal(4, E, 2, N, K), normal(5, E, CAP, 2, K)
    out2 = None
    if form == 0:
        rows, other, out = a, w, zeros(E, CAP, N)
        call = lambda: ep.ep_ll_gemm_bf16(a, w, count, out, status)  # noqa: E731
    elif form == 1:
        rows, other, out, out2 = a, w2, zeros(E, CAP, N), zeros(E, CAP, 2, N)
        call = lambda: ep.ep_ll_gemm_swiglu_bf16(a, w2, count, out, out2, status)  # noqa: E731
    elif form == 2:
        rows, other, out = gy, w, zeros(E, CAP, K)
        call = lambda: ep.ep_ll_gemm_dgrad_bf16(gy, w, count, out, status)  # noqa: E731
    elif form == 3:
        rows, other, out = gy, w, zeros(E, CAP, 2, K)
        call = lambda: ep.ep_ll_gemm_dswiglu_bf16(gy, w, gu, count, out, status)  # noqa: E731
    else:
        rows, other, out = gy, a, zeros(E, N, K, dtype=torch.float32 if form == 4 else BF16)
        call = lambda: ep.ep_ll_gemm_wgrad_bf16(gy, a, count, out, status)  # noqa: E731
    stalled = lambda *s: ep.ep_debug_ll_gemm_bf16_stall(  # noqa: E731
        form, N, K, rows, other, gu if form == 3 else None, count, out, out2, status, *s)
    check(call, stalled, [out] if out2 is None else [out, out2], status, tile)


@pytest.mark.parametrize("cap", [300, 60])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("tile", [0, 1])
def test_int8_products(cap, gated, tile):
    count, status = torch.tensor(ROWS, dtype=torch.int32, device="cuda"), zeros(1, dtype=torch.int32)
    g = torch.Generator().manual_seed(6)
    whole = lambda *s: torch.randint(-127, 128, s, generator=g, dtype=torch.int8).cuda()  # noqa: E731
    two = (2,) if gated else ()
    a, w = whole(E, cap, K), whole(E, *two, N, K)
    s, ws = torch.rand(E, cap, generator=g).cuda() + 0.5, torch.rand(E, *two, N, generator=g).cuda() * 1e-3
    y = zeros(E, cap, N, dtype=torch.int8 if gated else BF16)
    ys = zeros(E, cap, dtype=torch.float32) if gated else None
    work = zeros(E * cap * N * 4, dtype=torch.uint8)
    if gated:
        call = lambda: ep.ep_ll_gemm_swiglu_int8(a, s, w, ws, count, y, ys, work, status)  # noqa: E731
    else:
        call = lambda: ep.ep_ll_gemm_int8(a, s, w, ws, count, y, status)  # noqa: E731
    stalled = lambda *st: ep.ep_debug_ll_gemm_int8_stall(a, s, w, ws, count, y, ys, work, status, *st)  # noqa: E731
    check(call, stalled, [y] if ys is None else [y, ys], status, tile)
