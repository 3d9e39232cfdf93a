"""Outputs that the binding allocates for a call on a stream given as a raw
handle: their memory may still be in use by the current stream."""
import pytest
import torch

from tests import test_gpu_paged as paged
from tests import test_gpu_verify as verify

pytestmark = pytest.mark.gpu


def _left_by_pending_work(shape, dtype):
    """Memory that goes back to the allocator while the current stream has
    still to write it: the next allocation of this size there gets it."""
    x = torch.empty(shape, dtype=dtype, device="cuda")
    torch.cuda._sleep(int(3e8))
    x.fill_(7)
    return x.data_ptr()


def test_attention_on_a_raw_handle(gpu_lib):
    c = paged.Case([(300, 300), (700, 200)], 16, 2, 128, 16, seed=1)
    d = c.dev()
    plan = c.plan(gpu_lib)
    want, _ = paged.run(gpu_lib, c, d=d, plan=plan)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    at = _left_by_pending_work(want.shape, c.dtype)
    out, _ = gpu_lib.markov_paged_attention(plan, d["q"], d["kc"], d["vc"], d["table"], d["idx"], d["start"],
                                            d["lens"], stream=s.cuda_stream)
    assert out.data_ptr() == at
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    plan.close()


def test_acceptance_on_a_raw_handle(gpu_lib):
    s = verify.make(200, 16, 1040, seed=2)
    want = verify.run(gpu_lib, s, probs=False)
    d = {k: v.cuda() for k, v in s.items()}
    plan = gpu_lib.Plan(1040, 64, 16, 200)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    at = _left_by_pending_work((200, 17), torch.int64)
    toks, acc = gpu_lib.markov_verify(plan, d["target"], d["tokens"], d["draft"], d["T"], d["u"], d["noise"],
                                      d["idx"], stream=st.cuda_stream)
    assert toks.data_ptr() == at
    torch.cuda.synchronize()
    assert (toks.cpu().numpy() == want[0]).all() and (acc.cpu().numpy() == want[1]).all()
    plan.close()


def test_the_default_streams_handle(gpu_lib):
    """0 is a handle too; the current stream is another one."""
    c = paged.Case([(40, 3)], 4, 2, 64, 16, seed=3)
    d = c.dev()
    plan = c.plan(gpu_lib)
    want, wl = paged.run(gpu_lib, c, d=d, plan=plan)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, lse = gpu_lib.markov_paged_attention(plan, d["q"], d["kc"], d["vc"], d["table"], d["idx"], d["start"],
                                                  d["lens"], lse=True, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)
    plan.close()
