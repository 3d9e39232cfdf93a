"""Rotary plans that are used as soon as they are there."""
import pytest
import torch

from tests import serving_ref as ref

pytestmark = pytest.mark.gpu


def test_a_plans_first_call_on_a_stream_of_its_own(gpu_lib):
    """Plans of other frequencies one after the other, most likely in the same memory, each
    called at once on a stream that does not wait for the default one."""
    api = gpu_lib
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn((64, 2, 128), generator=g, device="cuda")
    pos = torch.randint(0, 100000, (64,), generator=g, device="cuda").int()
    out = torch.empty_like(x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(50):
        theta = 1000.0 * (i + 2)
        plan = api.RotaryPlan(128, theta=theta)
        api.markov_rotary(plan, x, None, pos, q_out=out, stream=side)
        side.synchronize()
        want, tol = ref.rotary(x, pos, ref.frequencies(128, theta), False)
        assert float(((out.double() - want).abs() - tol).max()) <= 0, i
        torch.cuda.synchronize()
        plan.close()
