"""ep_ll_dispatch_fp8 and the experts' e4m3 products against plain references.

Tolerances, fixed before the first run.  The cast uses fp32 operations only:
bit-exact.  A product's fp32 sums are off by at most sum_error(k) * sum |a w|
(any order); its bf16 result adds half an ulp, 2^-8 relative to be safe of a
boundary.  The gated activation h carries the products' errors through
|silu'| <= 1.1, plus a few fp32 roundings; its e4m3 value adds half a step:
|h| / 16 for normal values, scale * 2^-10 below."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import moe_ref
import oracle
from combine_get_dispatch_notify_gb300 import ep
from combine_get_dispatch_notify_gb300.workloads import CONFIGS, Workload, gen_routing, gen_x

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.lib()


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ dispatch
DISPATCH = {
    "tiny": (CONFIGS["tiny"], None),
    "low_latency": (CONFIGS["low_latency"], 128),
    "one_token": (Workload("d", R=1, T=1, H=7168, E=8, K=8, C=1), 1),
    "odd_h": (Workload("d", R=3, T=17, H=208, E=9, K=5, C=1, mask=0.3), None),
    "h16": (Workload("d", R=1, T=37, H=16, E=6, K=3, C=1, routing="replace"), None),
    "h1040": (Workload("d", R=2, T=29, H=1040, E=64, K=32, C=1), None),
    "h_2200": (Workload("d", R=8, T=64, H=2192, E=64, K=4, C=1, routing="zipf"), None),
    "capacity_drop": (Workload("d", R=2, T=64, H=512, E=4, K=2, C=1), 7),
    "no_tokens": (Workload("d", R=2, T=0, H=512, E=4, K=2, C=1), 7),
}


def run_dispatch(w, cap, x, idx, slot, info=True):
    sh = ep.EpShape.make(w.R, w.T, w.K, w.E, w.H, w.C)
    nb = ep.scale_blocks(w.H)
    rx = torch.full((w.E, cap, w.H), 0x55, dtype=torch.uint8, device="cuda")
    rs = torch.full((w.E, cap, nb), -7.0, device="cuda")
    si = torch.full((w.E, cap, 2), -7, dtype=torch.int32, device="cuda") if info else None
    status = status_word()
    ep.ep_ll_dispatch_fp8(sh, x.cuda(), idx.cuda(), slot.cuda(), cap, rx, rs, si, status)
    assert ep.ep_sync_status(status) == ep.EP_OK
    return rx.cpu(), rs.cpu(), None if si is None else si.cpu()


def want_dispatch(w, cap, x, idx, slot):
    q, s = moe_ref.cast_blocks(x.reshape(w.R * w.T, w.H))
    rx = torch.full((w.E, cap, w.H), 0x55, dtype=torch.uint8)
    rs = torch.full((w.E, cap, s.shape[-1]), -7.0)
    si = torch.full((w.E, cap, 2), -7, dtype=torch.int32)
    for r in range(w.R):
        for t in range(w.T):
            for k in range(w.K):
                e, p = int(idx[r, t, k]), int(slot[r, t, k])
                if 0 <= e < w.E and 0 <= p < cap:
                    rx[e, p], rs[e, p] = q[r * w.T + t], s[r * w.T + t]
                    si[e, p] = torch.tensor([r, t], dtype=torch.int32)
    return rx, rs, si


@pytest.mark.parametrize("name", sorted(DISPATCH))
def test_dispatch_fp8_is_exact(name):
    w, cap = DISPATCH[name]
    cap = w.R * w.T * w.K if cap is None else cap
    idx, _ = gen_routing(w)
    x = gen_x(w)
    if w.T > 3:
        x[0, 0] = 0.0                     # scale at its floor
        x[0, 1] *= 1e-30                  # below the floor: rounds to zero
        x[0, 2] *= 1e30
        x[0, 3, :5] = torch.tensor([1e-39, -1e-39, 0.0, -0.0, 3e38])
    slot = torch.from_numpy(oracle.ll_layout(oracle.load(), w.R, w.T, w.K, w.E, cap, idx.numpy())["slot_pos"])
    got = run_dispatch(w, cap, x, idx, slot)
    want = want_dispatch(w, cap, x, idx, slot)
    for g, v, what in zip(got, want, ("recv_x", "recv_x_scales", "recv_src_info")):
        assert torch.equal(g, v), what
    rx, rs, _ = run_dispatch(w, cap, x, idx, slot, info=False)
    assert torch.equal(rx, want[0]) and torch.equal(rs, want[1])


def test_dispatch_fp8_skips_bad_slots_and_keeps_infinities_visible():
    w = Workload("d", R=1, T=4, H=256, E=4, K=2, C=1)
    x = gen_x(w)
    x[0, 1, 3] = float("nan")
    x[0, 2, 130] = float("inf")
    idx = torch.tensor([[[0, 9], [1, -1], [2, 3], [-6, 1]]])
    slot = torch.tensor([[[0, 0], [0, 1], [1, 8], [0, -1]]], dtype=torch.int32)
    rx, rs, si = run_dispatch(w, 8, x, idx, slot)
    wx, ws, wi = want_dispatch(w, 8, x, idx, slot)
    assert torch.equal(si, wi) and torch.equal(rs, ws)
    v, u = moe_ref.fp8(rx), moe_ref.fp8(wx)
    assert torch.equal(torch.isnan(v), torch.isnan(u)) and torch.equal(torch.nan_to_num(v), torch.nan_to_num(u))
    back = v[2, 1] * moe_ref.expand(rs[2, 1], 256, -1)
    assert torch.isnan(back[128:]).all() and torch.isfinite(back[:128]).all()
    assert torch.isnan(v[1, 0]).sum() == 1  # a NaN stays one element


# ------------------------------------------------------------------ products
def gemm_inputs(E, cap, n, k, seed, halves=1, counts=None):
    g = torch.Generator().manual_seed(seed)
    q = lambda *s: (torch.randn(*s, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
    sc = lambda *s: torch.exp(torch.randn(*s, generator=g)) / 100  # noqa: E731
    nb, kb = ep.scale_blocks(n), ep.scale_blocks(k)
    ws = (E, n) if halves == 1 else (E, 2, n)
    wss = (E, nb) if halves == 1 else (E, 2, nb)
    a, w = q(E, cap, k), q(*ws, k)
    a_s, w_s = sc(E, cap, kb), sc(*wss, kb) / k ** 0.5
    if counts is None:
        counts = torch.randint(0, cap + 3, (E,), generator=g)
        counts[0] = cap
        counts[-1] = 0 if E > 1 else cap
    return a, a_s, w, w_s, torch.as_tensor(counts, dtype=torch.int32)


GEMMS = [  # E, cap, n, k
    (1, 1, 8, 16), (2, 3, 128, 128), (3, 16, 136, 144), (4, 17, 256, 256), (2, 64, 384, 512), (5, 33, 120, 400),
    (2, 130, 512, 640), (3, 260, 264, 1040), (1, 400, 1024, 7168), (8, 8, 2048, 128), (40, 20, 256, 384),
    (2, 520, 776, 2048), (1, 129, 40, 48), (300, 2, 16, 32),
]


def check_gemm(args, y, n):
    a, a_s, w, w_s, count = args
    k = a.shape[-1]
    for e in range(a.shape[0]):
        m = min(int(count[e]), a.shape[1])
        assert (y[e, max(m, 0):] == -7.0).all(), "rows beyond the count were written"
        if m <= 0:
            continue
        want, mag = moe_ref.product(a[e, :m], a_s[e, :m], w[e], w_s[e])
        err = (y[e, :m].double() - want).abs()
        assert (err <= want.abs() * 2.0 ** -8 + mag * moe_ref.sum_error(k)).all(), e


def run_gemm(args, n, stream=None):
    a, a_s, w, w_s, count = (t.cuda() for t in args)
    y = torch.full((a.shape[0], a.shape[1], n), -7.0, dtype=torch.bfloat16, device="cuda")
    status = status_word()
    torch.cuda.synchronize()
    ep.ep_ll_gemm_fp8(a, a_s, w, w_s, count, y, status, stream=stream)
    assert ep.ep_sync_status(status, stream=stream) == ep.EP_OK
    return y.cpu()


@pytest.mark.parametrize("dims", GEMMS, ids=str)
def test_gemm_matches_float64(dims):
    E, cap, n, k = dims
    args = gemm_inputs(E, cap, n, k, 1)
    check_gemm(args, run_gemm(args, n), n)


def silu(x):
    return x / (1 + torch.exp(-x))


def check_swiglu(args, y, ys, n):
    a, a_s, w, w_s, count = args
    k = a.shape[-1]
    nb = ep.scale_blocks(n)
    for e in range(a.shape[0]):
        m = max(0, min(int(count[e]), a.shape[1]))
        assert (y[e, m:] == 0x55).all() and (ys[e, m:] == -7.0).all(), "rows beyond the count were written"
        if m == 0:
            continue
        gate, gm = moe_ref.product(a[e, :m], a_s[e, :m], w[e, 0], w_s[e, 0])
        up, um = moe_ref.product(a[e, :m], a_s[e, :m], w[e, 1], w_s[e, 1])
        h = silu(gate) * up
        c = moe_ref.sum_error(k)
        dh = 1.1 * gm * c * (up.abs() + um * c) + silu(gate).abs() * um * c + h.abs() * 2.0 ** -20
        pad = torch.nn.functional.pad
        blocks = lambda t: pad(t, (0, nb * 128 - n)).view(m, nb, 128).amax(-1)  # noqa: E731
        want = blocks(h.abs()).clamp(min=2.0 ** -100) / 448
        dscale = blocks(dh) / 448 + want * 2.0 ** -22
        assert ((ys[e, :m].double() - want).abs() <= dscale).all(), e
        sc = moe_ref.expand(ys[e, :m], n, -1)
        back = moe_ref.fp8(y[e, :m]) * sc
        tol = h.abs() / 16 + sc * 2.0 ** -10 + 2 * dh + 448 * moe_ref.expand(dscale, n, -1)
        assert ((back - h).abs() <= tol).all(), e


def run_swiglu(args, n):
    a, a_s, w, w_s, count = (t.cuda() for t in args)
    y = torch.full((a.shape[0], a.shape[1], n), 0x55, dtype=torch.uint8, device="cuda")
    ys = torch.full((a.shape[0], a.shape[1], ep.scale_blocks(n)), -7.0, device="cuda")
    status = status_word()
    ep.ep_ll_gemm_swiglu_fp8(a, a_s, w, w_s, count, y, ys, status)
    assert ep.ep_sync_status(status) == ep.EP_OK
    return y.cpu(), ys.cpu()


@pytest.mark.parametrize("dims", [(E, cap, max(16, n // 16 * 16), k) for E, cap, n, k in GEMMS], ids=str)
def test_swiglu_matches_float64(dims):
    E, cap, n, k = dims
    args = gemm_inputs(E, cap, n, k, 2, halves=2)
    check_swiglu(args, *run_swiglu(args, n), n)


def test_products_without_rows_write_nothing():
    args = gemm_inputs(4, 8, 256, 256, 3, counts=[0, 0, 0, 0])
    assert (run_gemm(args, 256) == -7.0).all()
    args = gemm_inputs(3, 8, 256, 256, 3, counts=[-4, 0, 2])  # a negative count has no rows
    check_gemm(args, run_gemm(args, 256), 256)
    args = gemm_inputs(4, 8, 256, 256, 3, halves=2, counts=[0, 0, 0, 0])
    y, ys = run_swiglu(args, 256)
    assert (y == 0x55).all() and (ys == -7.0).all()
    a, a_s, w, w_s, count = gemm_inputs(2, 0, 256, 256, 3, counts=[0, 0])
    run_gemm((a, a_s, w, w_s, count), 256)


def test_rows_do_not_mix():
    """Infinite and NaN rows (and the garbage beyond the count) stay in their rows."""
    E, cap, n, k = 2, 40, 256, 384
    args = gemm_inputs(E, cap, n, k, 4, counts=[33, 21])
    clean = run_gemm(args, n)
    a = args[0].clone()
    a_s = args[1].clone()
    a[:, 21:] = torch.where(torch.arange(cap)[21:, None] < 33, a[:, 21:], torch.tensor(0x7f, dtype=torch.uint8))
    a[1, 21:] = 0x7f       # NaN bytes beyond the count of expert 1
    a[0, 33:] = 0x7f
    a_s[0, 33:] = float("nan")
    a[0, 5, 7] = 0x7f      # one NaN element of one row
    a_s[0, 6, 1] = float("inf")
    y = run_gemm((a, a_s, *args[2:]), n)
    assert torch.isnan(y[0, 5]).all() and not torch.isfinite(y[0, 6]).any()
    keep = [r for r in range(33) if r not in (5, 6)]
    assert torch.equal(y[0, keep], clean[0, keep]) and torch.equal(y[1, :21], clean[1, :21])


def test_products_repeat_bit_for_bit_on_any_stream():
    args = gemm_inputs(6, 200, 640, 1024, 5)
    first = run_gemm(args, 640)
    side = torch.cuda.Stream()
    for stream in (None, side, side):
        assert torch.equal(run_gemm(args, 640, stream), first)


def test_input_gradient_is_the_call_on_the_transposed_weights():
    """dx = g @ w: the same product with the weights' blocks and scales transposed."""
    E, cap, n, k = 2, 24, 256, 384
    g, g_s, w, w_s, count = gemm_inputs(E, cap, k, n, 6)       # w [E, k, n]
    y = run_gemm((g, g_s, w, w_s, count), k)
    for e in range(E):
        m = min(int(count[e]), cap)
        wv = moe_ref.fp8(w[e]) * moe_ref.expand(moe_ref.expand(w_s[e], k, 0), n, 1)
        want = (moe_ref.fp8(g[e, :m]) * moe_ref.expand(g_s[e, :m], n, -1)) @ wv.T
        mag = (moe_ref.fp8(g[e, :m]).abs() * moe_ref.expand(g_s[e, :m], n, -1)) @ wv.abs().T
        assert ((y[e, :m].double() - want).abs() <= want.abs() * 2.0 ** -8 + mag * moe_ref.sum_error(n)).all()


def test_large_offsets():
    """Buffers whose byte offsets pass 32 bits: the last expert's rows and weights are the right ones."""
    E, cap, n, k = 40, 65536, 16, 2048     # a: 5.4e9 bytes
    a = torch.zeros(E, cap, k, dtype=torch.uint8, device="cuda")
    a_s = torch.zeros(E, cap, k // 128, device="cuda")
    small = gemm_inputs(E, 4, n, k, 7, counts=[2] * E)
    count = torch.zeros(E, dtype=torch.int32)
    count[-1] = cap
    a[-1, -4:] = small[0][-1].cuda()
    a_s[-1, -4:] = small[1][-1].cuda()
    y = torch.empty(E, cap, n, dtype=torch.bfloat16, device="cuda")
    status = status_word()
    ep.ep_ll_gemm_fp8(a, a_s, small[2].cuda(), small[3].cuda(), count.cuda(), y, status)
    assert ep.ep_sync_status(status) == ep.EP_OK
    want, mag = moe_ref.product(small[0][-1], small[1][-1], small[2][-1], small[3][-1])
    got = y[-1, -4:].double().cpu()
    assert ((got - want).abs() <= want.abs() * 2.0 ** -8 + mag * moe_ref.sum_error(k)).all()
    assert (y[-1, :-4] == 0).all()


def off16(t):
    """A copy of `t` on the device that starts on a 16-byte boundary and on no wider one."""
    step = 16 // t.element_size()
    buf = torch.empty(t.numel() + step, dtype=t.dtype, device="cuda")
    assert buf.data_ptr() % 32 == 0
    return buf[step:].view(t.shape).copy_(t)


@pytest.mark.parametrize("cap,n,k", [(300, 512, 384), (40, 272, 256)])
def test_products_with_arrays_on_16_byte_boundaries(cap, n, k):
    E = 3
    a, a_s, w, w_s, count = gemm_inputs(E, cap, n, k, 8)
    y = off16(torch.full((E, cap, n), -7.0, dtype=torch.bfloat16))
    status = status_word()
    ep.ep_ll_gemm_fp8(off16(a), off16(a_s), off16(w), off16(w_s), count.cuda(), y, status)
    assert ep.ep_sync_status(status) == ep.EP_OK
    check_gemm((a, a_s, w, w_s, count), y.cpu(), n)
    a, a_s, w, w_s, count = gemm_inputs(E, cap, n, k, 9, halves=2)
    y = off16(torch.full((E, cap, n), 0x55, dtype=torch.uint8))
    ys = off16(torch.full((E, cap, ep.scale_blocks(n)), -7.0))
    ep.ep_ll_gemm_swiglu_fp8(off16(a), off16(a_s), off16(w), off16(w_s), count.cuda(), y, ys, status)
    assert ep.ep_sync_status(status) == ep.EP_OK
    check_swiglu((a, a_s, w, w_s, count), y.cpu(), ys.cpu(), n)


@pytest.mark.parametrize("E,cap,n,k", [(48, 300, 512, 128), (40, 270, 768, 640), (90, 140, 1024, 48), (150, 40, 512, 272)],
                         ids=str)
def test_products_with_many_tiles(E, cap, n, k):
    """Several tiles for every SM, of few k-blocks each: the tiles' hand-over runs ahead as far as it can."""
    args = gemm_inputs(E, cap, n, k, 10)
    args[4][1::3] = cap
    check_gemm(args, run_gemm(args, n), n)
    args = gemm_inputs(E, cap, n, k, 11, halves=2)
    args[4][1::3] = cap
    check_swiglu(args, *run_swiglu(args, n), n)
