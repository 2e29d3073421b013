"""Order between the experts' products and what stands around them: inputs written by the kernel
just before, results read by the one just after, and the hand-overs between a kernel's own warps.

Every comparison is bit for bit: the products add in a fixed order, so a call on inputs that
lie ready gives the bits that a call in any company has to give.  Those calls themselves are
held to float64 with the bounds of test_gpu_ll_fp8."""
from __future__ import annotations

import pytest
import torch

from combine_get_dispatch_notify_gb300 import ep
from test_gpu_ll_fp8 import check_gemm, check_swiglu, gemm_inputs, run_swiglu, status_word

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.lib()


# rows that both kernels share: whole tiles of 256, last ones of 129 to 255, rests of up to 128
COUNTS = [[300, 256, 384, 1, 0, 513], [1, 640, 128, 129, 385, 0], [520, 0, 257, 640, 255, 31]]


@pytest.mark.parametrize("n,k", [(264, 128), (520, 1040)], ids=str)
def test_product_reads_what_the_kernel_before_it_wrote(n, k):
    """Counts, rows and scales arrive by copies right before the call, other ones each time and
    without a pause between the calls; the output is taken away by a copy right behind it."""
    E, cap = 6, 640
    sets = [gemm_inputs(E, cap, n, k, 20 + i, counts=c) for i, c in enumerate(COUNTS)]
    status = status_word()
    dev = [[t.cuda() for t in s] for s in sets]
    y = torch.empty(E, cap, n, dtype=torch.bfloat16, device="cuda")
    want = []
    for d, s in zip(dev, sets):
        y.fill_(-7.0)
        torch.cuda.synchronize()
        ep.ep_ll_gemm_fp8(*d, y, status)
        torch.cuda.synchronize()
        want.append(y.clone())
        check_gemm(s, y.cpu(), n)
    a, a_s, w, w_s, count = (torch.empty_like(t) for t in dev[0])
    got = []
    for i in range(60):
        for to, t in zip((a, a_s, w, w_s, count), dev[i % 3]):
            to.copy_(t)
        y.fill_(-7.0)
        ep.ep_ll_gemm_fp8(a, a_s, w, w_s, count, y, status)
        got.append(y.clone())
    assert ep.ep_sync_status(status) == ep.EP_OK
    for i, g in enumerate(got):
        assert torch.equal(g, want[i % 3]), i


def test_product_behind_the_casting_dispatch():
    """The dispatch lets the product start early; its rows and scales still are the ones multiplied."""
    R, T, K, E, H, n, cap = 2, 400, 2, 4, 1024, 272, 800
    sh = ep.EpShape.make(R, T, K, E, H, 1)
    g = torch.Generator().manual_seed(30)
    status = status_word()
    _, _, w, w_s, _ = (t.cuda() for t in gemm_inputs(E, 1, n, H, 31))
    slot, rng, count = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((R, T, K), (E, R, 2), (E,)))
    rows = torch.zeros(E, cap, H, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(E, cap, H // 128, device="cuda")
    y = torch.empty(E, cap, n, dtype=torch.bfloat16, device="cuda")
    xs = [(torch.randn(R, T, H, generator=g) * s).to(torch.bfloat16).cuda() for s in (1.0, 30.0)]
    ids = [torch.rand(R, T, E, generator=g).argsort(-1)[..., :K].contiguous().cuda() for _ in xs]

    def step(i, pause):
        y.fill_(-7.0)
        for call in (lambda: ep.ep_ll_layout(sh, ids[i], None, cap, slot, rng, count, status),
                     lambda: ep.ep_ll_dispatch_fp8(sh, xs[i], ids[i], slot, cap, rows, scales, None, status),
                     lambda: ep.ep_ll_gemm_fp8(rows, scales, w, w_s, count, y, status)):
            if pause:
                torch.cuda.synchronize()
            call()
        return y.clone()

    want = [step(i, True) for i in (0, 1)]
    got = [step(i % 2, False) for i in range(60)]
    assert ep.ep_sync_status(status) == ep.EP_OK
    for i, v in enumerate(got):
        assert torch.equal(v, want[i % 2]), i


@pytest.mark.parametrize("k", [128, 512, 640], ids=str)
def test_gated_tiles_with_and_without_rows_in_a_quarter(k):
    """Each pair of SMs walks tiles of 256, 160, 129 and 256 rows by turns: most of its epilogue warps
    have rows on one tile, none on the next and rows again on the one after.  With few k-blocks a
    tile its warps may be far apart; every row's scale still comes from that row's own block."""
    E, cap, n = 8, 256, 76 * 128  # as many column tiles as pairs: a pair keeps its column
    args = gemm_inputs(E, cap, n, k, 32, halves=2, counts=[256, 160, 256, 129, 256, 160, 129, 256])
    # experts of very different size: a neighbouring tile's maximum would be far off
    args[3].mul_(10.0 ** (torch.arange(E) % 5 - 2).view(E, 1, 1, 1))
    y, ys = run_swiglu(args, n)
    check_swiglu(args, y, ys, n)
    for _ in range(10):
        again = run_swiglu(args, n)
        assert torch.equal(again[0], y) and torch.equal(again[1], ys)


@pytest.mark.parametrize("n,k", [(272, 128), (528, 1040)], ids=str)
def test_gated_product_reads_what_the_kernel_before_it_wrote(n, k):
    E, cap = 6, 640
    sets = [gemm_inputs(E, cap, n, k, 40 + i, halves=2, counts=c) for i, c in enumerate(COUNTS)]
    status = status_word()
    dev = [[t.cuda() for t in s] for s in sets]
    want = []
    for s in sets:
        y, ys = run_swiglu(s, n)
        check_swiglu(s, y, ys, n)
        want.append((y.cuda(), ys.cuda()))
    y, ys = torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
    into = [torch.empty_like(t) for t in dev[0]]
    got = []
    for i in range(60):
        for to, t in zip(into, dev[i % 3]):
            to.copy_(t)
        y.fill_(0x55)
        ys.fill_(-7.0)
        ep.ep_ll_gemm_swiglu_fp8(*into, y, ys, status)
        got.append((y.clone(), ys.clone()))
    assert ep.ep_sync_status(status) == ep.EP_OK
    for i, (v, s) in enumerate(got):
        assert torch.equal(v, want[i % 3][0]) and torch.equal(s, want[i % 3][1]), i


# E, capacity, n, k, counts: pairs of SMs with one to four tiles of one and of four k-blocks; few rows; both in one call
STALLS = [(4, 256, 76 * 128, 128, [256, 160, 256, 256]), (4, 256, 76 * 128, 512, [256, 129, 256, 256]),
          (40, 40, 1024, 384, [40] * 40), (8, 400, 4096, 256, [400, 20, 300, 128, 64, 256, 257, 1])]


@pytest.mark.parametrize("tile", [0, 1, 2])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("case", STALLS, ids=str)
def test_a_product_without_products_times_out_and_the_context_survives(case, gated, tile):
    """One place's tensor cores get nothing from one of its tiles on: the call still ends, reports
    EP_ERR_TIMEOUT, and the next call on the same buffers is bit for bit what it was before."""
    E, cap, n, k, counts = case
    a, a_s, w, w_s, count = (t.cuda() for t in gemm_inputs(E, cap, n, k, 50, halves=2 if gated else 1, counts=counts))
    status = status_word()
    y = torch.full((E, cap, n), 0x55 if gated else -7, dtype=torch.uint8 if gated else torch.bfloat16, device="cuda")
    ys = torch.full((E, cap, ep.scale_blocks(n)), -7.0, device="cuda") if gated else None

    def call():
        if gated:
            ep.ep_ll_gemm_swiglu_fp8(a, a_s, w, w_s, count, y, ys, status)
        else:
            ep.ep_ll_gemm_fp8(a, a_s, w, w_s, count, y, status)
        assert ep.ep_sync_status(status) == ep.EP_OK

    call()
    want = y.clone(), None if ys is None else ys.clone()
    # every place has its first tile; of the others only that the call ends is known here
    ep.ep_debug_ll_gemm_fp8_stall(a, a_s, w, w_s, count, y, ys, status, 0, tile, 20000)
    rc = ep.ep_sync_status(status)
    assert rc == ep.EP_ERR_TIMEOUT if tile == 0 else rc in (ep.EP_OK, ep.EP_ERR_TIMEOUT)
    status.zero_()
    call()
    assert torch.equal(y, want[0]) and (ys is None or torch.equal(ys, want[1]))
    ep.ep_debug_ll_gemm_fp8_stall(a, a_s, w, w_s, count, y, ys, status, -1, 0, 2000000)  # nothing stalled
    assert ep.ep_sync_status(status) == ep.EP_OK and torch.equal(y, want[0])


@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("E,cap,n,k", [(3, 128, 640, 7168), (40, 96, 1024, 3328), (2, 300, 784, 7168)], ids=str)
def test_scales_of_every_block_are_its_own(E, cap, n, k, gated):
    """Scales handed over four k-blocks at a time, each four 2^6 larger or smaller than the ones before in
    the same place: a row that read its neighbours' would be far off."""
    args = gemm_inputs(E, cap, n, k, 60, halves=2 if gated else 1, counts=[cap] * E)
    step = 2.0 ** (6.0 * ((torch.arange(args[1].shape[-1]) // 4) % 3 - 1))
    args[1].mul_(step)
    args[3].mul_(step.flip(0))
    if gated:
        y, ys = run_swiglu(args, n)
        check_swiglu(args, y, ys, n)
    else:
        a, a_s, w, w_s, count = (t.cuda() for t in args)
        y, status = torch.full((E, cap, n), -7.0, dtype=torch.bfloat16, device="cuda"), status_word()
        ep.ep_ll_gemm_fp8(a, a_s, w, w_s, count, y, status)
        assert ep.ep_sync_status(status) == ep.EP_OK
        check_gemm(args, y.cpu(), n)
