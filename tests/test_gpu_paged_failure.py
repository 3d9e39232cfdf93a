"""The paged attention's waits give up without faulting the GPU, and calls work
after that."""
import time

import pytest

from tests import test_gpu_paged as paged

pytestmark = pytest.mark.gpu
ETIMEOUT = 4


def test_a_wait_that_gives_up_ends_the_others(gpu_lib):
    """The second wait's limit is 2 seconds; had it run out, no status would be there."""
    t0 = time.perf_counter()
    assert gpu_lib.markov_selftest_wait(2, 2000) == ETIMEOUT
    assert time.perf_counter() - t0 < 5.0
    c = paged.Case([(200, 3), (40, 70)], 4, 2, 64, 16, seed=1)
    paged.both(gpu_lib, c)


def test_a_status_of_an_earlier_call_stops_both_launches(gpu_lib):
    """Split items' parts are not joined either: nothing of the call is written."""
    c = paged.Case([(20000, 1), (300, 200)], 4, 2, 64, 64, seed=2)
    plan = c.plan(gpu_lib)
    want = paged.run(gpu_lib, c, plan=plan)
    gpu_lib.markov_paged_plan_inject_status(plan, ETIMEOUT, 0x100)
    d = c.dev()
    out, lse = (x.clone().fill_(paged.SENT) for x in want)
    gpu_lib.markov_paged_attention(plan, d["q"], d["kc"], d["vc"], d["table"], d["idx"], d["start"], d["lens"],
                                   out=out, lse=lse)
    assert gpu_lib.markov_paged_plan_status(plan) == ETIMEOUT
    assert bool((out == paged.SENT).all()) and bool((lse == paged.SENT).all())
    again = paged.run(gpu_lib, c, plan=plan)
    assert all(bool((a == b).all()) for a, b in zip(again, want))
    plan.close()
