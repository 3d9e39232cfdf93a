"""markov_verify where its arguments are unusual."""
import math

import numpy as np
import pytest
import torch

from tests import test_gpu_verify as base

pytestmark = pytest.mark.gpu
F = [torch.bfloat16, torch.float32]


def call(api, s, target=None, draft=None):
    R, N, V = s["draft"].shape
    d = {k: v.cuda() for k, v in s.items()}
    plan = api.Plan(V, 64, N, R)
    toks, acc = api.markov_verify(plan, d["target"] if target is None else target, d["tokens"],
                                  d["draft"] if draft is None else draft, d["T"], d["u"], d["noise"], d["idx"])
    assert api.markov_plan_status(plan) == 0
    plan.close()
    return toks.cpu().numpy(), acc.cpu().numpy()


def test_the_stride_of_a_lone_row_says_nothing(gpu_lib):
    """Logits [N + 1, 1, V] of a sequence-first model, transposed."""
    s = base.make(1, 4, 4096, seed=1, temps=(1.0,))
    want = base.run(gpu_lib, s)
    base.check(s, want)
    t, c = (s[k].cuda()[0].unsqueeze(1).transpose(0, 1) for k in ("target", "draft"))
    assert t.stride(0) == c.stride(0) == 4096
    for target, draft in ((t, None), (None, c), (t, c)):
        toks, acc = call(gpu_lib, s, target, draft)
        assert np.array_equal(toks, want[0]) and np.array_equal(acc, want[1])
    # not a multiple of 16 bytes either
    t = s["target"].cuda().as_strided((1, 5, 4096), (3, 4096, 1))
    toks, acc = call(gpu_lib, s, t)
    assert np.array_equal(toks, want[0]) and np.array_equal(acc, want[1])
    s["noise"] = torch.cat([s["noise"], torch.zeros((1, 1))], 1).cuda()[:, :4096]
    assert s["noise"].stride(0) == 4097
    toks, acc = call(gpu_lib, s)
    assert np.array_equal(toks, want[0]) and np.array_equal(acc, want[1])


def test_the_stride_of_a_lone_step_says_nothing(gpu_lib):
    s = base.make(3, 1, 4096, seed=2, temps=(1.0,))
    want = base.run(gpu_lib, s)
    base.check(s, want)
    for stride in (1, 4095):
        toks, acc = call(gpu_lib, s, draft=s["draft"].cuda().as_strided((3, 1, 4096), (4096, stride, 1)))
        assert np.array_equal(toks, want[0]) and np.array_equal(acc, want[1])


@pytest.mark.parametrize("dtype", F)
@pytest.mark.parametrize("V", [2064, 4096, 20000])
def test_infinite_temperature(gpu_lib, dtype, V):
    """Every logit over +inf is 0: the distributions are uniform."""
    s = base.make(5, 3, V, seed=3, target=dtype, draft=dtype, temps=(math.inf, 1.0))
    got = base.run(gpu_lib, s)
    assert base.check(s, got) >= 4
    # ids that are masked stay without probability
    s["target"][..., ::2] = -math.inf
    s["draft"][..., ::2] = -math.inf
    s["tokens"] = s["tokens"] // 2 * 2 + 1
    _, _, p, q = got = base.run(gpu_lib, s)
    for b in (0, 2, 4):
        assert np.allclose(p[b], 2 / V, rtol=5e-5) and np.allclose(q[b], 2 / V, rtol=5e-5)
        assert (got[0][b][:3] % 2 == 1).all() and got[1][b] == 3 and got[0][b][3] % 2 == 1
