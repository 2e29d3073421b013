"""Waits of the experts' weight gradient in calls that are far longer than the wait limit: the limit is for work that
stands still, not for the length of a call."""
from __future__ import annotations

import pytest
import torch

from combine_get_dispatch_notify_gb300 import ep

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.lib()


def run(form, n, k, counts, cap, limit_us):
    """All operands 1, so that an expert's gradients are its rows, which bf16 holds here: (status, gradients' minima and
    maxima)."""
    E = len(counts)
    gy, a = (torch.ones(E, cap, m, dtype=BF16, device="cuda") for m in (n, k))
    gw = torch.full((E, n, k), 7.0, dtype=torch.float32 if form == 4 else BF16, device="cuda")
    count = torch.tensor(counts, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.ep_debug_ll_gemm_bf16_stall(form, n, k, gy, a, None, count, gw, None, status, -1, 0, limit_us)
    return ep.ep_sync_status(status), gw.flatten(1).amin(1).tolist(), gw.flatten(1).amax(1).tolist()


@pytest.mark.parametrize("form", [4, 5])
def test_one_ragged_expert_behind_many_whole_ones(form):
    """Only the last expert's rows end inside a step: what zeroes behind them has nothing to do for the 8 ms before (1.8e13
    operations at 2 PFLOP/s), four times the limit, while no step takes more than microseconds and no tile more than 40 of them."""
    counts = [2048] * 256 + [5]
    rc, low, high = run(form, 4096, 4096, counts, 2048, 2000)
    assert rc == ep.EP_OK
    assert low == counts and high == counts


def test_many_tiles_of_one_block_between_those_of_two():
    """The last of three tiles of output rows has one block, and a pair, whose next tile is one column further, has all of
    its columns in a row: the second accumulator's warps have nothing to do for 4 ms, twice the limit."""
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    columns = (pairs - 1) // 3
    if 3 * columns != pairs - 1:
        pytest.skip("the walk over the tiles does not advance by one column on this number of SMs")
    counts = [32768] * 32
    rc, low, high = run(5, 1280, 256 * columns, counts, 32768, 2000)
    assert rc == ep.EP_OK
    assert low == counts and high == counts
