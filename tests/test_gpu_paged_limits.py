"""The paged calls at the ends of their documented ranges."""
import math

import pytest
import torch

from tests import test_gpu_paged as paged

pytestmark = pytest.mark.gpu
SENT = 123.0


def test_layout_of_lengths_past_31_bits(gpu_lib):
    """A table row with pages for more than 2^31 - 1 tokens: the last length
    that there is, and one beyond it, whose second position has no 32 bits."""
    api = gpu_lib
    i32, dev = torch.int32, "cuda"
    page, width = 256, (1 << 31) // 256 + 1
    plan = api.PagedPlan(4, 4, 64, page, max_rows=2)
    table = torch.full((2, width), -1, dtype=i32, device=dev)
    table[:, width - 2] = torch.tensor([3, 5], dtype=i32, device=dev)     # the page of the last positions
    held = torch.full((2,), width - 1, dtype=i32, device=dev)
    free = torch.tensor([0, 4], device=dev)
    ring = torch.arange(4, dtype=i32, device=dev)
    last = (1 << 31) - 1
    start, lens, pos, slots = api.markov_paged_layout(
        plan, torch.tensor([last, last - 2], dtype=i32, device=dev), torch.tensor([2, 2], dtype=i32, device=dev),
        torch.arange(2, device=dev), table, held, ring, free, 4)
    assert api.markov_paged_plan_status(plan) == 0
    assert start.tolist() == [0, 2, 4] and lens.tolist() == [0, last]
    assert pos.tolist() == [0, 0, last - 2, last - 1]
    assert slots.tolist() == [-1, -1, 5 * page + 253, 5 * page + 254]
    assert held.tolist() == [width - 1] * 2 and free.tolist() == [0, 4] and ring.tolist() == [0, 1, 2, 3]
    plan.close()


def attend_absent_pages(api, keys, timeout_ms=0):
    """One token, 256 key heads of 64, over `keys` keys in pages that are not
    there: they read as zeros, so the outputs are zeros and lse is ln(keys)."""
    i32 = dict(dtype=torch.int32, device="cuda")
    plan = api.PagedPlan(256, 256, 64, 256, torch.bfloat16, max_rows=1, timeout_ms=timeout_ms)
    cache = torch.ones((1, 256, 256, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.ones((1, 256, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.full_like(q, SENT), torch.full((1, 256), SENT, device="cuda")
    api.markov_paged_attention(plan, q, cache, cache, torch.full((1, keys // 256), -1, **i32),
                               torch.zeros(1, dtype=torch.int64, device="cuda"), torch.tensor([0, 1], **i32),
                               torch.tensor([keys], **i32), out=out, lse=lse)
    status = api.markov_paged_plan_status(plan)
    plan.close()
    return status, out, lse


def test_a_request_of_2_to_the_27_key_tiles(gpu_lib):
    """A sixteenth of the documented bound, in one request."""
    keys = 1 << 26
    status, out, lse = attend_absent_pages(gpu_lib, keys)
    assert status == 0
    assert bool((out == 0).all())
    # sums of ones are exact here; the logarithm is within a few units of fp32
    assert float((lse.double() - math.log(keys)).abs().max()) <= 1e-5 * math.log(keys)


def test_items_that_take_longer_than_the_wait_limit(gpu_lib):
    """A block's next item waits for the one before it: several milliseconds
    of work, which is not a wait that went wrong."""
    keys = 1 << 20
    status, out, lse = attend_absent_pages(gpu_lib, keys, timeout_ms=1)
    assert status == 0
    assert bool((out == 0).all())
    assert float((lse.double() - math.log(keys)).abs().max()) <= 1e-5 * math.log(keys)


def test_a_walk_that_takes_longer_than_the_wait_limit(gpu_lib):
    """32768 pairs of row tiles in one request are counted before the first
    item is known; its tokens see nothing."""
    api = gpu_lib
    T = 65536
    i32 = dict(dtype=torch.int32, device="cuda")
    plan = api.PagedPlan(128, 1, 64, 16, torch.bfloat16, max_rows=1, timeout_ms=1)
    cache = torch.zeros((1, 16, 1, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.ones((T, 128, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.full_like(q, SENT), torch.full((T, 128), SENT, device="cuda")
    api.markov_paged_attention(plan, q, cache, cache, torch.zeros((1, 1), **i32),
                               torch.zeros(1, dtype=torch.int64, device="cuda"), torch.tensor([0, T], **i32),
                               torch.tensor([0], **i32), out=out, lse=lse)
    assert api.markov_paged_plan_status(plan) == 0
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    plan.close()


@pytest.mark.parametrize("window,sinks", [(1 << 30, 0), ((1 << 30) + 100, 5), ((1 << 31) - 1, 0)])
def test_windows_past_30_bits(gpu_lib, window, sinks):
    """A length beyond the table's keys, of which a window of 2^30 keys and more
    still hides the first ones."""
    for behind in (40, 130, 300):
        c = paged.Case([(383, 1), (380, 4)], 4, 2, 64, 16, seed=behind, width_extra=0)
        c.lens[:] = min(window + behind, (1 << 31) - 1)
        paged.both(gpu_lib, c, window=window, sinks=sinks)


@pytest.mark.parametrize("window,sinks", [(5, 3), (200, 130), (7, 0), (0, 0)])
def test_the_last_positions_that_there_are(gpu_lib, window, sinks):
    """Lengths up to 2^31 - 1 over a short table: of a window nothing is left but
    the first tokens, in whole key tiles too."""
    for n in (1, 3):
        c = paged.Case([(512 - n, n), (300, 2)], 4, 4, 64, 16, seed=n, width_extra=0)
        c.lens[0] = (1 << 31) - 1
        paged.both(gpu_lib, c, window=window, sinks=sinks)
