"""Attention over an e4m3 cache whose scales take long to come: they lie in pinned host
memory, which the device reads over its link, while keys, values and the table are in its
own.  Whatever takes part in a tile's softmax has to wait for them."""
import ctypes

import pytest
import torch

from tests.test_gpu_e4m3 import SENT, Case, check

pytestmark = pytest.mark.gpu


def _view(api, plan, t, scales):
    v = api._E4m3View()
    pages, blocks, heads = scales.shape
    s, c = t.stride(), scales.stride()
    v.data, v.num_pages, v.s_page, v.s_slot, v.s_head = t.data_ptr(), pages, s[0], s[1], s[2]
    v.scales, v.ss_page, v.ss_block, v.ss_head = scales.data_ptr(), c[0], c[1], c[2]
    v.block = plan.page_size // blocks
    return v


@pytest.mark.parametrize("host", ["values", "keys", "both"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("reqs,page,block", [
    ([(4000, 9), (100, 9), (0, 9), (700, 9)], 64, 16),            # items of one row tile
    ([(3000, 60), (500, 33)], 32, 32),                            # of two
    ([(300, 200), (129, 1), (2000, 2)], 128, 16),                 # of two and of one
    ([(3000, 1), (40, 1), (900, 1)], 16, 16)])                    # single tokens
def test_scales_that_come_late(gpu_lib, reqs, page, block, d, dtype, host):
    api = gpu_lib
    # neighbouring blocks' scales lie far apart, so that another's would show
    case = Case(reqs, 16, 2, d, page, block, dtype=dtype, seed=page + d, spread=(-10, -3))
    x = case.dev()
    ks = case.ks.pin_memory() if host != "values" else x["ks"]
    vs = case.vs.pin_memory() if host != "keys" else x["vs"]
    plan = case.plan(api)
    k, v = _view(api, plan, x["kc"], ks), _view(api, plan, x["vc"], vs)
    for _ in range(3):
        out = torch.full((case.T, case.hq, case.d), SENT, dtype=case.dtype, device="cuda")
        lse = torch.full((case.T, case.hq), SENT, device="cuda")
        q, table = x["q"], x["table"]
        code = api.lib().markov_paged_attention_e4m3(
            plan.handle, q.data_ptr(), q.stride(0), q.stride(1), ctypes.byref(k), ctypes.byref(v), table.data_ptr(),
            table.stride(0), table.shape[0], table.shape[1], x["idx"].data_ptr(), x["start"].data_ptr(), x["lens"].data_ptr(),
            len(case.idx), case.T, case.d ** -0.5, 0, 0, out.data_ptr(), out.stride(0), out.stride(1), lse.data_ptr(),
            torch.cuda.current_stream().cuda_stream)
        assert code == 0 and api.markov_paged_plan_status(plan) == 0
    plan.close()
    check(case, out, lse)
