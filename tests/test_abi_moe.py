"""Host-side refusals of the router and the experts' products (no kernel runs)."""
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


FAKE, ODD, NUL = vp(1 << 20), vp((1 << 20) + 4), vp(None)  # never dereferenced: the call fails first


def test_route_rules(ep):
    sh = ep.EpShape.make(2, 4, 8, 256, 8, 1)
    mk = ep.EpRoute.make
    ok = [mk(), mk("sigmoid", 8, 4, 2, True, 2.5), mk("softmax", 32, 1, 2), mk("softmax", 1, 1, 2), mk(scale=-1.0)]
    bad = [mk(num_groups=0), mk(num_groups=3), mk(num_groups=64), mk("softmax", 8, 9), mk("softmax", 8, 0),
           mk(group_top=0), mk(group_top=3), mk(scale=float("nan")), mk(scale=float("inf")),
           ep.EpRoute(2, 1, 1, 1, 0, 1.0), ep.EpRoute(-1, 1, 1, 1, 0, 1.0), ep.EpRoute(0, 1, 1, 1, 2, 1.0)]
    for r in ok:
        assert ep.ep_check_route(sh, r) == ep.EP_OK
    for r in bad:
        assert ep.ep_check_route(sh, r) == ep.EP_ERR_INVALID_ARG
    # K experts must be left by the groups, a group must have group_top members, the shape must be one
    assert ep.ep_check_route(ep.EpShape.make(1, 4, 9, 32, 8, 1), mk("softmax", 8, 2)) == ep.EP_ERR_INVALID_ARG
    assert ep.ep_check_route(ep.EpShape.make(1, 4, 8, 32, 8, 1), mk("softmax", 8, 2)) == ep.EP_OK
    assert ep.ep_check_route(ep.EpShape.make(1, 4, 2, 8, 8, 1), mk("softmax", 8, 2, 2)) == ep.EP_ERR_INVALID_ARG
    assert ep.ep_check_route(ep.EpShape.make(1, 4, 9, 8, 8, 1), mk()) == ep.EP_ERR_INVALID_ARG
    assert ep.ep_check_route(ep.EpShape.make(12, 4, 2, 12, 8, 1), mk()) == ep.EP_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        mk("tanh")


def test_gemm_shape_rules(ep):
    G = ep.EpGemmShape
    for s in (G(1, 0, 8, 16), G(8192, 1 << 24, 1 << 20, 1 << 15), G(1, 1, 8, 1 << 20), G(3, 5, 136, 144)):
        assert ep.ep_check_gemm_shape(s) == ep.EP_OK
    for s in (G(0, 1, 8, 16), G(8193, 1, 8, 16), G(1, -1, 8, 16), G(1, (1 << 24) + 1, 8, 16), G(1, 1, 4, 16),
              G(1, 1, 0, 16), G(1, 1, 8, 8), G(1, 1, 8, 0), G(1, 1, 8, 24), G(1, 1, 12, 16), G(1, 1, (1 << 20) + 8, 16),
              G(1, 1, 8, (1 << 20) + 16), G(1, 1 << 20, 8, 1 << 20), G(1, 1, 1 << 20, 1 << 20), G(1, 1, -8, 16), G(1, 1, 8, -16)):
        assert ep.ep_check_gemm_shape(s) == ep.EP_ERR_INVALID_ARG


def test_bad_pointers_are_refused(ep):
    L, inv = ep.lib(), ep.EP_ERR_INVALID_ARG
    sh, cfg = ep.EpShape.make(2, 4, 2, 4, 16, 1), ep.EpRoute.make()
    s, c = ctypes.byref(sh), ctypes.byref(cfg)
    for i in (0, 2, 3, 4):  # logits, topk_idx, topk_w, status
        for wrong in (NUL, ODD if i != 4 else vp((1 << 20) + 2)):
            p = [FAKE] * 5
            p[i] = wrong
            assert L.ep_route(s, c, p[0], 0, p[1], p[2], p[3], p[4], vp(0)) == inv
    assert L.ep_route(s, c, FAKE, 0, ODD, FAKE, FAKE, FAKE, vp(0)) == inv       # bias, misaligned
    assert L.ep_route(s, c, FAKE, 2, NUL, FAKE, FAKE, FAKE, vp(0)) == inv       # unknown logits type
    assert L.ep_route(None, c, FAKE, 0, NUL, FAKE, FAKE, FAKE, vp(0)) == inv
    assert L.ep_route(s, None, FAKE, 0, NUL, FAKE, FAKE, FAKE, vp(0)) == inv
    for i in range(5):  # logits, topk_idx, grad_topk_w, grad_logits, status
        p = [FAKE] * 5
        p[i] = NUL
        assert L.ep_route_backward(s, c, p[0], 1, *p[1:], vp(0)) == inv
    for i in (0, 1, 2, 3, 4, 6):  # all but recv_src_info
        p = [FAKE] * 7
        p[i] = NUL
        assert L.ep_ll_dispatch_fp8(s, *p[:3], 4, *p[3:], vp(0)) == inv
    assert L.ep_ll_dispatch_fp8(s, FAKE, FAKE, FAKE, -1, FAKE, FAKE, FAKE, FAKE, vp(0)) == inv
    assert L.ep_ll_dispatch_fp8(s, FAKE, FAKE, FAKE, 4, FAKE, FAKE, ODD, FAKE, vp(0)) == inv
    h24 = ep.EpShape.make(2, 4, 2, 4, 24, 1)  # rows of e4m3 are whole 16-byte vectors
    assert L.ep_ll_dispatch_fp8(ctypes.byref(h24), FAKE, FAKE, FAKE, 4, FAKE, FAKE, FAKE, FAKE, vp(0)) == inv
    g = ep.EpGemmShape(2, 4, 16, 32)
    for i in range(7):  # a, a_scales, w, w_scales, count, y, status
        for wrong in (NUL, vp((1 << 20) + 2)):
            p = [FAKE] * 7
            p[i] = wrong
            assert L.ep_ll_gemm_fp8(ctypes.byref(g), *p, vp(0)) == inv
    for i in range(8):
        p = [FAKE] * 8
        p[i] = NUL
        assert L.ep_ll_gemm_swiglu_fp8(ctypes.byref(g), *p, vp(0)) == inv
    n8 = ep.EpGemmShape(2, 4, 8, 32)  # the gated product's rows are e4m3: a multiple of 16
    assert L.ep_ll_gemm_swiglu_fp8(ctypes.byref(n8), *[FAKE] * 8, vp(0)) == inv


def test_empty_calls_enqueue_nothing(ep):
    """No tokens or no rows: EP_OK without a launch (this machine may have no GPU)."""
    L = ep.lib()
    sh, cfg = ep.EpShape.make(2, 0, 2, 4, 16, 1), ep.EpRoute.make()
    s, c = ctypes.byref(sh), ctypes.byref(cfg)
    assert L.ep_route(s, c, NUL, 0, NUL, NUL, NUL, FAKE, vp(0)) == ep.EP_OK
    assert L.ep_route_backward(s, c, NUL, 0, NUL, NUL, NUL, FAKE, vp(0)) == ep.EP_OK
    assert L.ep_ll_dispatch_fp8(s, NUL, NUL, NUL, 4, FAKE, FAKE, NUL, FAKE, vp(0)) == ep.EP_OK
    g = ep.EpGemmShape(2, 0, 16, 32)
    assert L.ep_ll_gemm_fp8(ctypes.byref(g), NUL, NUL, FAKE, FAKE, FAKE, NUL, FAKE, vp(0)) == ep.EP_OK


def test_binding_checks_its_tensors(ep):
    sh = ep.EpShape.make(1, 2, 2, 4, 16, 1)
    cpu = torch.zeros(1, 2, 4)
    with pytest.raises(ValueError):
        ep.ep_route(sh, ep.EpRoute.make(), cpu, None, None, None, None)
    with pytest.raises(ValueError):
        ep.ep_route(sh, ep.EpRoute.make(), cpu.double(), None, None, None, None)
    with pytest.raises(ValueError):
        ep.ep_ll_gemm_fp8(torch.zeros(2, 4), None, torch.zeros(2, 8, 16), None, None, None, None)
    with pytest.raises(ValueError):
        ep.ep_ll_gemm_swiglu_fp8(torch.zeros(2, 4, 16), None, torch.zeros(2, 8, 16), None, None, None, None, None)
