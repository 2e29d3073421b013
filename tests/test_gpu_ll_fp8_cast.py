"""The gated product's activation and its cast to e4m3, on inputs whose products are exact."""
from __future__ import annotations

import pytest
import torch

from combine_get_dispatch_notify_gb300 import ep
from test_gpu_ll_fp8 import run_swiglu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.lib()


def e4m3(v):
    return torch.as_tensor(v, dtype=torch.float32).to(torch.float8_e4m3fn).view(torch.uint8)


@pytest.mark.parametrize("rows", [1, 77, 128, 256, 400])
def test_gated_rows_are_cast_by_division(rows):
    """q = e4m3_rne(h / scale) with one fp32 division, as the casting dispatch has it, bit for bit.

    h is exact: gate = 32, whose exp(-32) does not change 1 + exp(-gate), times up, a whole number
    below 4096 put together from three columns.  A block's largest is 28 q, so its scale is
    a multiple of q and q (17 + 2 i) lies halfway between two e4m3 numbers: a quotient that is
    one ulp off goes to the wrong one of them."""
    blocks = 146
    n = blocks * 128
    gen = torch.Generator().manual_seed(25)
    q = torch.arange(1, blocks + 1).view(-1, 1)
    up = (torch.rand(blocks, 128, generator=gen) * (28 * q + 1)).long()
    up[:, 0] = 28 * q[:, 0]
    up[:, 1:7] = q * (17 + 2 * torch.arange(6))
    up[:, 7:13] = q * (17 + 2 * torch.arange(6)) // 2
    up[:, 13:19] = q * (17 + 2 * torch.arange(6)) // 4
    up = up[:, torch.randperm(128, generator=gen)].reshape(n)
    w = torch.zeros(1, 2, n, 16)
    w[0, 0, :, 3] = 32.0
    for j in range(3):
        w[0, 1, :, j] = (up >> 4 * j & 15).float()
    a = torch.zeros(1, rows, 16)
    a[0, :, :4] = torch.tensor([1.0, 16.0, 256.0, 1.0])
    args = (e4m3(a), torch.ones(1, rows, 1), e4m3(w), torch.ones(1, 2, blocks, 1), torch.tensor([rows], dtype=torch.int32))
    y, ys = run_swiglu(args, n)
    h = (32 * up).float().view(blocks, 128)
    scale = h.amax(-1) / 448.0
    assert torch.equal(ys[0], scale.expand(rows, blocks))
    assert torch.equal(y[0], e4m3(h / scale.unsqueeze(-1)).view(1, n).expand(rows, n))


@pytest.mark.parametrize("rows", [64, 128, 256, 389])
def test_activation_has_fp32_precision_at_every_gate(rows):
    """silu(gate) * up over gates from 20 to -88.6, seen through the scale of a block whose other columns
    are zero: |h| / 448.  gate = -x and up = 2^40 x are exact; expf's 2 ulp (2^-22), an addition, two
    divisions and a product (2^-24 each) make 2^-21 relative."""
    x = torch.linspace(-20.0, 88.6, rows)
    x[x == 0] = 0.5
    a = torch.zeros(1, rows, 16)
    a[0, :, 0] = 1.0
    w = torch.zeros(1, 2, 128, 16)
    w[0, 0, 5, 0], w[0, 1, 5, 0] = -1.0, 1.0
    ws = torch.tensor([1.0, 2.0 ** 40]).view(1, 2, 1, 1)
    args = (e4m3(a), x.view(1, rows, 1), e4m3(w), ws, torch.tensor([rows], dtype=torch.int32))
    y, ys = run_swiglu(args, 128)
    xd = x.double()
    h = -xd / (1 + torch.exp(xd)) * (xd * 2.0 ** 40)
    want = h.abs() / 448
    assert (want > 2.0 ** -100).all()
    assert ((ys[0, :, 0].double() - want).abs() <= want * 2.0 ** -21).all()
    assert (y[0, :, 5] == e4m3(torch.where(h < 0, -448.0, 448.0))).all()
    assert (y[0, :, :5] & 0x7f == 0).all() and (y[0, :, 6:] & 0x7f == 0).all()
