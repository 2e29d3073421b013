"""Host-side refusals of the experts' products' testing hook (no kernel runs)."""
import ctypes

from test_abi_moe import FAKE, NUL, ep, pytestmark, vp  # noqa: F401  (the fixture builds the library)


def test_stall_hook_rules(ep):  # noqa: F811
    L, inv = ep.lib(), ep.EP_ERR_INVALID_ARG
    good, n8 = ctypes.byref(ep.EpGemmShape(2, 4, 16, 32)), ctypes.byref(ep.EpGemmShape(2, 4, 8, 32))

    def call(shape, pointers, cta, tile, limit):
        return L.ep_debug_ll_gemm_fp8_stall(shape, *pointers, cta, tile, limit, vp(0))

    p = [FAKE] * 8
    for cta, tile, limit in ((-2, 0, 1000), (0, -1, 1000), (0, (1 << 20) + 1, 1000), (0, 0, 0), (0, 0, 2000001)):
        assert call(good, p, cta, tile, limit) == inv
    for i in (0, 1, 2, 3, 4, 5, 7):  # a, a_scales, w, w_scales, count, y, status
        assert call(good, p[:i] + [NUL] + p[i + 1:], 0, 0, 1000) == inv
    assert call(n8, p, 0, 0, 1000) == inv  # with y_scales the gated product's rules hold
    assert call(None, p, 0, 0, 1000) == inv
    empty = ctypes.byref(ep.EpGemmShape(2, 0, 16, 32))
    assert call(empty, [NUL, NUL, FAKE, FAKE, FAKE, NUL, NUL, FAKE], 0, 0, 1000) == ep.EP_OK
