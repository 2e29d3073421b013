"""Host-side refusals of the experts' bf16 and int8 products, their gradients, the combine's
gradient and the int8 dispatch (no kernel runs)."""
import ctypes
import os
import shutil

import pytest
import torch

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")


@pytest.fixture(scope="module")
def ep():
    from combine_get_dispatch_notify_gb300 import build, ep as binding
    build.build()
    binding.lib()
    return binding


def vp(v):
    return ctypes.c_void_p(v)


FAKE, FAKE2 = vp(1 << 20), vp(1 << 21)  # never dereferenced: the call fails first
ODD, NUL = vp((1 << 20) + 2), vp(None)


def test_bf16_shape_rules(ep):
    G = ep.EpGemmShape
    for s in (G(1, 0, 8, 8), G(8192, 128, 1 << 17, 1 << 20), G(1, 1, 8, 1 << 20), G(3, 5, 136, 24), G(127, 1 << 24, 8, 8)):
        assert ep.ep_check_gemm_shape_bf16(s) == ep.EP_OK
    for s in (G(0, 1, 8, 8), G(8193, 1, 8, 8), G(1, -1, 8, 8), G(1, (1 << 24) + 1, 8, 8), G(1, 1, 4, 8), G(1, 1, 8, 12),
              G(1, 1, 0, 8), G(1, 1, 8, 0), G(1, 1, -8, 8), G(1, 1, 8, -8), G(1, 1, (1 << 20) + 8, 8),
              G(1, 1, 8, (1 << 20) + 8), G(128, 1 << 24, 8, 8), G(1, 1 << 18, 8, 1 << 20), G(1, 1 << 18, 1 << 20, 8),
              G(1, 1, 1 << 18, 1 << 20)):
        assert ep.ep_check_gemm_shape_bf16(s) == ep.EP_ERR_INVALID_ARG


def test_int8_workspace_follows_the_shape(ep):
    G = ep.EpGemmShape
    assert ep.ep_ll_gemm_swiglu_int8_workspace_bytes(G(4, 10, 48, 32)) == 4 * 10 * 48 * 4
    assert ep.ep_ll_gemm_swiglu_int8_workspace_bytes(G(4, 0, 48, 32)) == 0
    assert ep.ep_ll_gemm_swiglu_int8_workspace_bytes(G(4, 10, 40, 32)) == 0  # n % 16
    assert ep.ep_ll_gemm_swiglu_int8_workspace_bytes(G(4, 10, 48, 24)) == 0  # k % 16


BF16_CALLS = {  # name: number of pointers (all required), those that may be NULL, those that take no 2-byte alignment
    "ep_ll_gemm_bf16": (5, ()),
    "ep_ll_gemm_swiglu_bf16": (6, (4,)),
    "ep_ll_gemm_dgrad_bf16": (5, ()),
    "ep_ll_gemm_dswiglu_bf16": (6, ()),
}


@pytest.mark.parametrize("name", sorted(BF16_CALLS))
def test_bf16_products_refuse_bad_pointers(ep, name):
    fn, inv = getattr(ep.lib(), name), ep.EP_ERR_INVALID_ARG
    count, nullable = BF16_CALLS[name]
    good = ep.EpGemmShape(2, 4, 16, 24)
    pointers = lambda: [FAKE] * 4 + [FAKE2] * (count - 4)  # noqa: E731
    for i in range(count):
        for wrong in (NUL, ODD):
            if wrong is NUL and i in nullable:
                continue
            p = pointers()
            p[i] = wrong
            assert fn(ctypes.byref(good), *p, vp(0)) == inv, (i, wrong)
    assert fn(None, *pointers(), vp(0)) == inv
    for bad in (ep.EpGemmShape(2, 4, 12, 24), ep.EpGemmShape(2, 4, 16, 20), ep.EpGemmShape(0, 4, 16, 24)):
        assert fn(ctypes.byref(bad), *pointers(), vp(0)) == inv
    # no rows: nothing is enqueued
    empty = ep.EpGemmShape(2, 0, 16, 24)
    assert fn(ctypes.byref(empty), *pointers(), vp(0)) == ep.EP_OK


def test_activation_gradient_refuses_its_own_input_as_output(ep):
    good = ep.EpGemmShape(2, 4, 16, 24)
    assert ep.lib().ep_ll_gemm_dswiglu_bf16(ctypes.byref(good), FAKE, FAKE, FAKE2, FAKE, FAKE2, FAKE, vp(0)) == \
        ep.EP_ERR_INVALID_ARG


def test_weight_gradient_refuses_bad_arguments(ep):
    fn, inv = ep.lib().ep_ll_gemm_wgrad_bf16, ep.EP_ERR_INVALID_ARG
    good = ep.EpGemmShape(2, 4, 16, 24)
    for i in range(5):
        for wrong in (NUL, ODD):
            p = [FAKE] * 5
            p[i] = wrong
            assert fn(ctypes.byref(good), *p[:4], 0, p[4], vp(0)) == inv, i
    for flag in (-1, 2):
        assert fn(ctypes.byref(good), FAKE, FAKE, FAKE, FAKE, flag, FAKE, vp(0)) == inv
    # without rows the weights' gradient is still written, so its array is still wanted
    empty = ep.EpGemmShape(2, 0, 16, 24)
    assert fn(ctypes.byref(empty), NUL, NUL, FAKE, NUL, 0, FAKE, vp(0)) == inv


def test_int8_products_refuse_bad_arguments(ep):
    L, inv = ep.lib(), ep.EP_ERR_INVALID_ARG
    good = ep.EpGemmShape(2, 4, 16, 32)
    for i in range(7):  # a, a_scales, w, w_scales, count, y, status
        for wrong in (NUL, ODD):
            p = [FAKE] * 7
            p[i] = wrong
            assert L.ep_ll_gemm_int8(ctypes.byref(good), *p, vp(0)) == inv, i
    need = 2 * 4 * 16 * 4
    for i in range(9):  # a, a_scales, w, w_scales, count, y, y_scales, workspace, status
        for wrong in (NUL, ODD):
            p = [FAKE] * 9
            p[i] = wrong
            assert L.ep_ll_gemm_swiglu_int8(ctypes.byref(good), *p[:8], need, p[8], vp(0)) == inv, i
    assert L.ep_ll_gemm_swiglu_int8(ctypes.byref(good), *[FAKE] * 8, need - 1, FAKE, vp(0)) == inv
    for bad in (ep.EpGemmShape(2, 4, 8, 32), ep.EpGemmShape(2, 4, 16, 24), ep.EpGemmShape(2, -1, 16, 32)):
        assert L.ep_ll_gemm_swiglu_int8(ctypes.byref(bad), *[FAKE] * 8, 1 << 20, FAKE, vp(0)) == inv
    assert L.ep_ll_gemm_int8(ctypes.byref(ep.EpGemmShape(2, 4, 12, 32)), *[FAKE] * 7, vp(0)) == inv
    empty = ep.EpGemmShape(2, 0, 16, 32)
    assert L.ep_ll_gemm_int8(ctypes.byref(empty), NUL, NUL, FAKE, FAKE, FAKE, NUL, FAKE, vp(0)) == ep.EP_OK
    assert L.ep_ll_gemm_swiglu_int8(ctypes.byref(empty), NUL, NUL, FAKE, FAKE, FAKE, NUL, NUL, NUL, 0, FAKE, vp(0)) == \
        ep.EP_OK


def test_combine_gradient_and_int8_dispatch_refuse_bad_arguments(ep):
    L, inv = ep.lib(), ep.EP_ERR_INVALID_ARG
    sh = ep.EpShape.make(2, 4, 2, 4, 16, 1)
    for i in range(8):  # grad_combined, y, topk_idx, topk_w, slot_pos, grad_y, grad_topk_w, status
        for wrong in (NUL, ODD):
            p = [FAKE] * 8
            p[i] = wrong
            assert L.ep_ll_combine_backward(ctypes.byref(sh), *p[:2], 4, *p[2:], vp(0)) == inv, i
    assert L.ep_ll_combine_backward(ctypes.byref(sh), FAKE, FAKE, -1, *[FAKE] * 6, vp(0)) == inv
    assert L.ep_ll_combine_backward(None, FAKE, FAKE, 4, *[FAKE] * 6, vp(0)) == inv
    for i in (0, 1, 2, 3, 4, 6):  # all but recv_src_info
        for wrong in (NUL, ODD):
            p = [FAKE] * 7
            p[i] = wrong
            assert L.ep_ll_dispatch_int8(ctypes.byref(sh), *p[:3], 4, *p[3:], vp(0)) == inv, i
    assert L.ep_ll_dispatch_int8(ctypes.byref(sh), FAKE, FAKE, FAKE, 4, FAKE, FAKE, ODD, FAKE, vp(0)) == inv
    assert L.ep_ll_dispatch_int8(ctypes.byref(sh), FAKE, FAKE, FAKE, -1, *[FAKE] * 4, vp(0)) == inv
    h24 = ep.EpShape.make(2, 4, 2, 4, 24, 1)  # rows of int8 are whole 16-byte vectors
    assert L.ep_ll_dispatch_int8(ctypes.byref(h24), FAKE, FAKE, FAKE, 4, *[FAKE] * 4, vp(0)) == inv
    none = ep.EpShape.make(2, 0, 2, 4, 16, 1)
    assert L.ep_ll_combine_backward(ctypes.byref(none), NUL, FAKE, 4, NUL, NUL, NUL, FAKE, NUL, FAKE, vp(0)) == ep.EP_OK
    assert L.ep_ll_dispatch_int8(ctypes.byref(none), NUL, NUL, NUL, 4, FAKE, FAKE, NUL, FAKE, vp(0)) == ep.EP_OK


def test_binding_checks_its_tensors(ep):
    z = torch.zeros
    with pytest.raises(ValueError):
        ep.ep_ll_gemm_bf16(z(2, 4), z(2, 8, 16), None, None, None)
    with pytest.raises(ValueError):
        ep.ep_ll_gemm_bf16(z(2, 4, 16, dtype=torch.bfloat16), z(2, 8, 16, dtype=torch.bfloat16), None, None, None)  # CPU
    with pytest.raises(ValueError):
        ep.ep_ll_gemm_swiglu_bf16(z(2, 4, 16), z(2, 8, 16), None, None, None, None)
    with pytest.raises(ValueError):
        ep.ep_ll_gemm_dgrad_bf16(None, z(2, 8, 16), None, None, None)
    with pytest.raises(ValueError):
        ep.ep_ll_gemm_dswiglu_bf16(z(2, 4, 16), z(8, 16), None, None, None, None)
    with pytest.raises(ValueError):
        ep.ep_ll_gemm_wgrad_bf16(z(2, 4, 16), z(2, 4, 8), None, z(2, 16, 8, dtype=torch.float16), None)
    with pytest.raises(ValueError):
        ep.ep_ll_gemm_swiglu_int8(z(2, 4, 16), None, z(2, 8, 16), None, None, None, None, None, None)
    with pytest.raises(ValueError):
        ep.MoELayer(ep.EpShape.make(1, 2, 2, 4, 16, 1), ep.EpRoute.make(), 16, 4, weights="int4")


def test_channel_cast():
    from combine_get_dispatch_notify_gb300 import ep
    w = torch.randn(2, 2, 24, 40, generator=torch.Generator().manual_seed(3)) * 3
    w[0, 1, 5] = 0
    q, s = ep.cast_weight_channels(w)
    assert q.dtype == torch.int8 and q.shape == w.shape and s.shape == (2, 2, 24) and q.is_contiguous()
    assert int(q.abs().max()) == 127 and (q[0, 1, 5] == 0).all() and float(s[0, 1, 5]) > 0
    # half a step, and the roundings of scale and quotient
    assert ((q.double() * s.double().unsqueeze(-1) - w.double()).abs() <= s.double().unsqueeze(-1) * (0.5 + 2.0 ** -15)).all()


def test_stall_hooks_refuse_bad_arguments(ep):
    L, inv = ep.lib(), ep.EP_ERR_INVALID_ARG
    good = ctypes.byref(ep.EpGemmShape(2, 4, 16, 32))
    bf16 = lambda form, p, *stall: L.ep_debug_ll_gemm_bf16_stall(good, form, *p, *stall, vp(0))  # noqa: E731
    p = [FAKE, FAKE, FAKE, FAKE, FAKE2, NUL, FAKE]  # rows, other, gate_up, count, out, gate_up_out, status
    i8 = lambda p, *stall: L.ep_debug_ll_gemm_int8_stall(good, *p[:8], 1 << 20, p[8], *stall, vp(0))  # noqa: E731
    q = [FAKE] * 9
    for stall in ((-2, 0, 1000), (0, -1, 1000), (0, (1 << 20) + 1, 1000), (0, 0, 0), (0, 0, 2000001)):
        assert bf16(0, p, *stall) == inv and i8(q, *stall) == inv
    for form in (-1, 6):
        assert bf16(form, p, 0, 0, 1000) == inv
    assert bf16(0, p[:5] + [FAKE] + p[6:], 0, 0, 1000) == inv  # only the gated product has a second output
    assert bf16(3, p[:2] + [NUL] + p[3:], 0, 0, 1000) == inv
    for i in (0, 1, 3, 4, 6):
        assert bf16(0, p[:i] + [NUL] + p[i + 1:], 0, 0, 1000) == inv
    for i in (0, 1, 2, 3, 4, 5, 7, 8):
        assert i8(q[:i] + [NUL] + q[i + 1:], 0, 0, 1000) == inv
