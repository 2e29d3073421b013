"""Outputs of the experts' bf16 and int8 products and of the combine's gradient that overlap an input or each other are
refused on the host (no kernel runs); arrays that touch are not."""
import ctypes
import os
import shutil

import pytest
import torch

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")

E, CAP, N, K = 3, 5, 32, 48
ROW_N, ROW_K = 2 * E * CAP * N, 2 * E * CAP * K  # bytes of bf16 rows
W = 2 * E * N * K
GEMM = (E, CAP, N, K)
# name: arrays in the order of the call with their bytes (0: a number of the call, not an array), and the outputs' places
CALLS = {
    "ep_ll_gemm_bf16": ([ROW_K, W, 4 * E, ROW_N, 4], (3,)),
    "ep_ll_gemm_swiglu_bf16": ([ROW_K, 2 * W, 4 * E, ROW_N, 2 * ROW_N, 4], (3, 4)),
    "ep_ll_gemm_dgrad_bf16": ([ROW_N, W, 4 * E, ROW_K, 4], (3,)),
    "ep_ll_gemm_dswiglu_bf16": ([ROW_N, W, 2 * ROW_K, 4 * E, 2 * ROW_K, 4], (4,)),
    "ep_ll_gemm_wgrad_bf16": ([ROW_N, ROW_K, 4 * E, 2 * W, 0, 4], (3,)),
    "ep_ll_gemm_int8": ([ROW_K // 2, 4 * E * CAP, W // 2, 4 * E * N, 4 * E, ROW_N, 4], (5,)),
    "ep_ll_gemm_swiglu_int8": ([ROW_K // 2, 4 * E * CAP, W, 8 * E * N, 4 * E, ROW_N // 2, 4 * E * CAP, 2 * ROW_N, 0, 4],
                               (5, 6, 7)),
}


@pytest.fixture(scope="module")
def ep():
    from combine_get_dispatch_notify_gb300 import build, ep as binding
    build.build()
    binding.lib()
    return binding


def spread(sizes):
    """Places with room between them, never dereferenced: every call here is refused."""
    at, out = 1 << 20, []
    for s in sizes:
        out.append(at)
        at += s + 4096 & ~255
    return out


def collisions(sizes, outputs):
    """Places of all arrays with one output moved onto another array: its start, and its last 16 bytes (4 where it is that
    short)."""
    for o in outputs:
        for other, size in enumerate(sizes):
            if other == o or size == 0:
                continue
            for inside in {0, max(0, (size - 1) // 16 * 16)}:
                at = spread(sizes)
                at[o] = at[other] + inside
                yield o, other, inside, at
                if sizes[o] > 16:  # and the other array within the output
                    at = spread(sizes)
                    at[other] = at[o] + (sizes[o] - 1) // 16 * 16
                    yield o, other, inside, at


@pytest.mark.parametrize("name", sorted(CALLS))
def test_products_refuse_outputs_that_overlap(ep, name):
    sizes, outputs = CALLS[name]
    fn, shape = getattr(ep.lib(), name), ep.EpGemmShape(*GEMM)
    for o, other, inside, at in collisions(sizes, outputs):
        args = [ctypes.c_void_p(p) if s else None for p, s in zip(at, sizes)]
        if name == "ep_ll_gemm_wgrad_bf16":
            args[4] = 0  # fp32
        elif name == "ep_ll_gemm_swiglu_int8":
            args[8] = sizes[7]
        assert fn(ctypes.byref(shape), *args, ctypes.c_void_p(0)) == ep.EP_ERR_INVALID_ARG, (o, other, inside)


def test_weight_gradient_in_the_place_of_its_rows_counts_the_type(ep):
    """bf16 gradients take half of the fp32 ones' bytes, and all of those."""
    sizes, _ = CALLS["ep_ll_gemm_wgrad_bf16"]
    at = spread(sizes)
    at[0] = at[3] + W - 16  # the last bytes of bf16 gradients
    args = [ctypes.c_void_p(p) for p in at]
    assert ep.lib().ep_ll_gemm_wgrad_bf16(ctypes.byref(ep.EpGemmShape(*GEMM)), *args[:4], 1, args[5], ctypes.c_void_p(0)) == \
        ep.EP_ERR_INVALID_ARG


def test_combine_gradient_refuses_outputs_that_overlap(ep):
    R, T, k, H = 1, 7, 2, 16
    shape = ep.EpShape.make(R, T, k, E, H, 1)
    # grad_combined, y, topk_idx, topk_w, slot_pos, grad_y, grad_topk_w, status
    sizes = [2 * R * T * H, 2 * E * CAP * H, 8 * R * T * k, 4 * R * T * k, 4 * R * T * k, 2 * E * CAP * H, 4 * R * T * k, 4]
    for o, other, inside, at in collisions(sizes, (5, 6)):
        p = [ctypes.c_void_p(v) for v in at]
        assert ep.lib().ep_ll_combine_backward(ctypes.byref(shape), *p[:2], CAP, *p[2:], ctypes.c_void_p(0)) == \
            ep.EP_ERR_INVALID_ARG, (o, other, inside)


@pytest.mark.gpu
def test_arrays_that_touch_are_taken(ep):
    """All arrays of a product one behind the other in one buffer, no byte between them."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    e, cap, n, k = 2, 16, 64, 64
    g = torch.Generator().manual_seed(1)
    a, w = (torch.randn(s, generator=g).bfloat16().cuda() for s in ((e, cap, k), (e, n, k)))
    count, status = torch.tensor([16, 9], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    want = torch.zeros(e, cap, n, dtype=torch.bfloat16, device="cuda")
    ep.ep_ll_gemm_bf16(a, w, count, want, status)
    one = torch.zeros(e * cap * (k + n) + e * n * k, dtype=torch.bfloat16, device="cuda")
    y, a2, w2 = one.split([e * cap * n, e * cap * k, e * n * k])
    y, a2, w2 = y.view(e, cap, n), a2.view(e, cap, k), w2.view(e, n, k)
    a2.copy_(a)
    w2.copy_(w)
    ep.ep_ll_gemm_bf16(a2, w2, count, y, status)
    assert ep.ep_sync_status(status) == ep.EP_OK
    assert torch.equal(y, want) and torch.equal(a2, a) and torch.equal(w2, w)
    with pytest.raises(ep.EpError):  # n == k: the rows' gradient in the place of what it is made from
        ep.ep_ll_gemm_dgrad_bf16(a, w, count, a, status)
    assert torch.equal(a2, a)
