"""Experts' products at sizes where a tile has two blocks of output columns and a pair several such tiles, with an even
and an odd number of blocks (the last tile's second block is then absent); waits that run out at a later tile; rows
of the gated int8 product that are longer than what its cast holds; projections that are not finite."""
from __future__ import annotations

import pytest
import torch

import experts_ref as ref
import test_gpu_ll_bf16 as bf
import test_gpu_ll_int8 as i8
from combine_get_dispatch_notify_gb300 import ep
from test_gpu_ll_bf16 import BF16, call, dev, fresh, normal, poisoned, untouched

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.lib()


def ceil(a, b):
    return -(-a // b)


def tiling(rows, cap, out, tile_rows):
    """(blocks of a tile, tiles, pairs of SMs) of the forms that choose between one block and two: the rule of RowTiles and
    blocks_of_tiles in whole numbers."""
    columns = ceil(out, 256)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    pairs = min(len(rows) * ceil(cap, tile_rows // 2) * columns, sms // 2)
    tiles = sum(ceil(m, tile_rows) for m in rows)
    halves = sum(ceil(m, tile_rows // 2) for m in rows)
    if cap > tile_rows // 2 and halves * columns <= ceil(tiles * columns, pairs) * pairs:
        tiles = halves
    one, two = ceil(tiles * columns, pairs), ceil(tiles * ceil(columns, 2), pairs)
    blocks = 1 if 8 * one <= 14 * two else 2
    return blocks, tiles * ceil(columns, blocks), pairs


RAGGED = [255, 256, 257, 300, 31, 33, 129, 0]
# output columns, contraction, capacity, rows of each expert, blocks of a tile
SHAPES = {
    "two_blocks_even": (504, 72, 300, RAGGED * 40, 2),
    "two_blocks_odd": (2056, 40, 300, (RAGGED + [300, 64]) * 6, 2),
    "one_block": (200, 72, 300, RAGGED * 40, 1),
}


def shape_of(name):
    out, inner, cap, rows, blocks = SHAPES[name]
    got, tiles, pairs = tiling(rows, cap, out, 256)
    assert got == blocks and tiles > 3 * pairs, (got, tiles, pairs)  # else the case no longer tests what it is for
    return out, inner, cap, rows


@pytest.mark.parametrize("name", sorted(SHAPES))
def test_product(name):
    n, k, cap, rows = shape_of(name)
    E = len(rows)
    a, w = normal(1, E, cap, k), normal(2, E, n, k, scale=k ** -0.5)
    y = fresh(E, cap, n)
    call(ep.ep_ll_gemm_bf16, poisoned(a, rows), w.cuda(), dev(rows), y)
    y = y.cpu()
    untouched(y, rows)
    for e, m in enumerate(rows):
        ref.close_bf16(f"y[{e}]", y[e, :m], *ref.product(a[e, :m], w[e]))


@pytest.mark.parametrize("name", sorted(SHAPES))
def test_rows_gradient(name):
    k, n, cap, rows = shape_of(name)
    E = len(rows)
    gy, w = normal(3, E, cap, n), normal(4, E, n, k, scale=n ** -0.5)
    ga = fresh(E, cap, k)
    call(ep.ep_ll_gemm_dgrad_bf16, poisoned(gy, rows), w.cuda(), dev(rows), ga)
    ga = ga.cpu()
    untouched(ga, rows)
    for e, m in enumerate(rows):
        ref.close_bf16(f"grad_a[{e}]", ga[e, :m], *ref.product(gy[e, :m], w[e].T))


@pytest.mark.parametrize("name", sorted(SHAPES))
def test_activation_gradient(name):
    k, n, cap, rows = shape_of(name)
    E = len(rows)
    gy, w = normal(5, E, cap, n), normal(6, E, n, k, scale=n ** -0.5)
    gu = normal(7, E, cap, 2, k, scale=3.0)
    out = fresh(E, cap, 2, k)
    call(ep.ep_ll_gemm_dswiglu_bf16, poisoned(gy, rows), w.cuda(), poisoned(gu, rows), dev(rows), out)
    out = out.cpu()
    untouched(out, rows)
    for e, m in enumerate(rows):
        gh, dgh = ref.product(gy[e, :m], w[e].T)
        want, bound = ref.gated_gradient(gh, dgh, gu[e, :m, 0], gu[e, :m, 1])
        for i, part in enumerate(("gate", "up")):
            ref.close_bf16(f"grad_{part}[{e}]", out[e, :m, i], want[i], bound[i])


# int8: output columns, contraction, capacity, blocks of a tile; tiles of 128 rows and of 64 (by the capacity)
INT8 = {
    "two_blocks": (512, 80, 300, 2),
    "two_blocks_short": (512, 80, 60, 2),
    "one_block": (208, 80, 300, 1),
    "one_block_short": (208, 80, 60, 1),
}


def int8_shape_of(name):
    n, k, cap, blocks = INT8[name]
    rows = [min(m, cap) for m in RAGGED * 40]
    got, tiles, pairs = tiling(rows, cap, n, 64 if cap <= 64 else 128)
    assert got == blocks and tiles > 3 * pairs, (got, tiles, pairs)
    return n, k, cap, rows


@pytest.mark.parametrize("name", sorted(INT8))
def test_int8_product(name):
    n, k, cap, rows = int8_shape_of(name)
    E = len(rows)
    a, w = i8.whole(8, E, cap, k), i8.whole(9, E, n, k)
    s, ws = i8.near(10, E, cap, scale=1 / 64), i8.near(11, E, n, scale=1 / 64)
    y = i8.run_plain(a.cuda(), i8.poisoned_scales(s, rows), w.cuda(), ws.cuda(), rows,
                     torch.full((E, cap, n), 7.0, dtype=BF16, device="cuda"))
    for e, m in enumerate(rows):
        assert (y[e, m:] == 7.0).all(), e
        ref.close_bf16(f"y[{e}]", y[e, :m], *i8.product(a[e, :m], s[e, :m], w[e], ws[e]))


# ------------------------------------------------------------------ waits that run out later on
def check(run, stalled, outs, status):
    """Every pair has more than three tiles here: the first two stalls are reported, the last one is behind every tile."""
    run()
    assert ep.ep_sync_status(status) == ep.EP_OK
    want = [t.clone() for t in outs]
    for tile, rc in ((1, ep.EP_ERR_TIMEOUT), (2, ep.EP_ERR_TIMEOUT), (1 << 20, ep.EP_OK)):
        for t in outs:
            t.zero_()
        stalled(0, tile, 20000)
        assert ep.ep_sync_status(status) == rc, tile
        status.zero_()
        if rc != ep.EP_OK:
            run()
            assert ep.ep_sync_status(status) == ep.EP_OK
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("name", sorted(SHAPES))
@pytest.mark.parametrize("form", range(6))
def test_bf16_products_stalled_later(name, form):
    out_n, inner, cap, rows = shape_of(name)
    n, k = (out_n, inner) if form in (0, 1, 4, 5) else (inner, out_n)
    E = len(rows)
    count, status = dev(rows), torch.zeros(1, dtype=torch.int32, device="cuda")
    gate_up, out2 = None, None
    if form in (4, 5):
        # its tiles are 512 x 256 of an expert's weights
        assert E * ceil(n, 512) * ceil(k, 256) > 3 * tiling(rows, cap, out_n, 256)[2]
        left, right = poisoned(normal(20, E, cap, n), rows), poisoned(normal(21, E, cap, k), rows)
        outs = [torch.zeros(E, n, k, dtype=torch.float32 if form == 4 else BF16, device="cuda")]
        run = lambda: ep.ep_ll_gemm_wgrad_bf16(left, right, count, outs[0], status)  # noqa: E731
    else:
        left = poisoned(normal(22, E, cap, k if form < 2 else n), rows)
        right = normal(23, E, *((2,) if form == 1 else ()), n, k).cuda()
        two = (2,) if form == 3 else ()
        outs = [torch.zeros(E, cap, *two, n if form < 2 else k, dtype=BF16, device="cuda")]
        if form == 0:
            run = lambda: ep.ep_ll_gemm_bf16(left, right, count, outs[0], status)  # noqa: E731
        elif form == 1:
            out2 = torch.zeros(E, cap, 2, n, dtype=BF16, device="cuda")
            outs.append(out2)
            run = lambda: ep.ep_ll_gemm_swiglu_bf16(left, right, count, outs[0], out2, status)  # noqa: E731
        elif form == 2:
            run = lambda: ep.ep_ll_gemm_dgrad_bf16(left, right, count, outs[0], status)  # noqa: E731
        else:
            gate_up = poisoned(normal(24, E, cap, 2, k), rows)
            run = lambda: ep.ep_ll_gemm_dswiglu_bf16(left, right, gate_up, count, outs[0], status)  # noqa: E731
    stalled = lambda *s: ep.ep_debug_ll_gemm_bf16_stall(  # noqa: E731
        form, n, k, left, right, gate_up, count, outs[0], out2, status, *s)
    check(run, stalled, outs, status)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("name", sorted(INT8))
def test_int8_products_stalled_later(name, gated):
    n, k, cap, rows = int8_shape_of(name)
    E, two = len(rows), (2,) if gated else ()
    count, status = dev(rows), torch.zeros(1, dtype=torch.int32, device="cuda")
    a, w = i8.whole(25, E, cap, k).cuda(), i8.whole(26, E, *two, n, k).cuda()
    s, ws = i8.near(27, E, cap).cuda(), i8.near(28, E, *two, n, scale=1e-3).cuda()
    y = torch.zeros(E, cap, n, dtype=torch.int8 if gated else BF16, device="cuda")
    ys = torch.zeros(E, cap, device="cuda") if gated else None
    work = torch.zeros(E * cap * n * 4 if gated else 0, dtype=torch.uint8, device="cuda")
    if gated:
        run = lambda: ep.ep_ll_gemm_swiglu_int8(a, s, w, ws, count, y, ys, work, status)  # noqa: E731
    else:
        run = lambda: ep.ep_ll_gemm_int8(a, s, w, ws, count, y, status)  # noqa: E731
    stalled = lambda *st: ep.ep_debug_ll_gemm_int8_stall(a, s, w, ws, count, y, ys, work, status, *st)  # noqa: E731
    check(run, stalled, [y] if ys is None else [y, ys], status)


# ------------------------------------------------------------------ long rows, values that are not finite
@pytest.mark.parametrize("n", [4096, 4112, 8208])
def test_int8_rows_longer_than_the_cast_holds(n):
    E, cap, k, rows = 2, 5, 32, [5, 2]
    a, w = i8.whole(30, E, cap, k), i8.whole(31, E, 2, n, k)
    s, ws = i8.near(32, E, cap, scale=1 / 64), i8.near(33, E, 2, n, scale=k ** -0.5 / 64)
    w[0, :, n - 3], ws[0, :, n - 3] = 127, 4.0  # some row's largest value behind what the cast holds
    y, ys = i8.run_gated(a.cuda(), i8.poisoned_scales(s, rows), w.cuda(), ws.cuda(), rows)
    for e, m in enumerate(rows):
        assert (y[e, m:] == 99).all() and (ys[e, m:] == 7.0).all(), e
        (g, dg), (u, du) = (i8.product(a[e, :m], s[e, :m], w[e, i], ws[e, i]) for i in range(2))
        h = ref.silu(g) * u
        dh = 1.1 * dg * (u.abs() + du) + ref.silu(g).abs() * du + h.abs() * 2.0 ** -20
        amax, damax = h.abs().amax(-1), dh.amax(-1)
        ref.close_fp32(f"scale[{e}]", ys[e, :m], amax / 127, damax / 127 + amax / 127 * 2.0 ** -23)
        step = ys[e, :m].double().unsqueeze(-1)
        # half a step, its own error in the quotient, and h's
        assert ((y[e, :m].double() * step - h).abs() <= step * (0.5 + 2.0 ** -15) + dh).all(), e
        assert (y[e, :m].abs().amax(-1) == 127).all()


def test_projections_that_are_not_finite():
    """Gates and ups past fp32's range, and a NaN, each in a row of its own.  gate / (1 + exp(-gate)) is infinite at an
    infinite gate and has no value at minus infinity; a finite gate with an infinite up is infinite; the slope
    s (1 + gate (1 - s)) has no value at either end.  The row that is finite is unmoved."""
    inf, nan, big = float("inf"), float("nan"), 2.0 ** 100
    m, k, n = 6, 8, 8
    a, w = torch.zeros(1, m, k), torch.zeros(1, 2, n, k)
    # row r reads column r of the weights; every column of the output is alike
    gate, up = [big, -big, 1.0, 1.0, nan, 2.0], [1.0, 1.0, big, -big, 1.0, 3.0]
    for r in range(m):
        a[0, r, r] = big if r < 4 else 1.0
        w[0, 0, :, r], w[0, 1, :, r] = gate[r], up[r]
    for r in (2, 3):
        w[0, 0, :, r] = 2.0 ** -100  # gate 1
    for r in (0, 1):
        w[0, 1, :, r] = 2.0 ** -100  # up 1
    w[0, 0, :, 4] = 1.0
    a[0, 4, 4] = nan
    y, gu = fresh(1, m, n), fresh(1, m, 2, n)
    call(ep.ep_ll_gemm_swiglu_bf16, a.to(BF16).cuda(), w.to(BF16).cuda(), dev([m]), y, gu)
    y, kept = y.cpu()[0].float(), gu.cpu()[0].float()
    assert torch.equal(kept[:4, 0, 0], torch.tensor([inf, -inf, 1.0, 1.0]))
    assert torch.equal(kept[:4, 1, 0], torch.tensor([1.0, 1.0, inf, -inf]))
    assert torch.isnan(kept[4]).all() and (kept[5, 0] == 2.0).all() and (kept[5, 1] == 3.0).all()
    assert (y[0] == inf).all() and torch.isnan(y[1]).all() and (y[2] == inf).all() and (y[3] == -inf).all()
    assert torch.isnan(y[4]).all()
    two = ref.silu(torch.full((n,), 2.0, dtype=torch.float64)) * 3
    ref.close_bf16("finite row", y[5], two, two.abs() * 2.0 ** -20)
    # the gradient from the same projections, gh = 1
    gy, wd = torch.zeros(1, m, 8, dtype=BF16), torch.zeros(1, 8, n, dtype=BF16)
    gy[..., 0], wd[0, 0] = 1.0, 1.0
    out = fresh(1, m, 2, n)
    call(ep.ep_ll_gemm_dswiglu_bf16, gy.cuda(), wd.cuda(), gu, dev([m]), out)
    out = out.cpu()[0].float()
    assert torch.isnan(out[[0, 1, 4], 0]).all() and torch.isnan(out[[1, 4], 1]).all()
    assert (out[0, 1] == inf).all() and (out[2, 0] == inf).all() and (out[3, 0] == -inf).all()
    one = torch.ones(m, n, dtype=torch.float64)
    want, bound = ref.gated_gradient(one[:1], 0 * one[:1], 2 * one[:1], 3 * one[:1])
    for i in range(2):
        ref.close_bf16("finite row", out[5:, i], want[i], bound[i])
    want, bound = ref.gated_gradient(one[:2], 0 * one[:2], one[:2], 0 * one[:2])
    ref.close_bf16("gradient of the infinite ups", out[2:4, 1], want[1], bound[1])
