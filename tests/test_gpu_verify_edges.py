"""markov_verify where its arguments are unusual."""
import math

import numpy as np
import pytest
import torch

from tests import test_gpu_verify as base

pytestmark = pytest.mark.gpu
F = [torch.bfloat16, torch.float32]


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
