"""The paged calls at the ends of their documented ranges."""
import pytest
import torch

pytestmark = pytest.mark.gpu


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
