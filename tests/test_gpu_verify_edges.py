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


def test_noise_where_one_id_has_it_all(gpu_lib):
    """Greedy rows, and rows whose token comes from a one-hot target: whatever
    the noise is, NaN included."""
    s = base.make(4, 3, 20000, seed=4, temps=(0.0, 1.0))
    s["u"][1], s["u"][3] = 0.0, 0.0                           # what p allows is accepted
    s["target"][1, 1, 777] = math.nan                         # refused there
    s["target"][3, 3, 5] = math.inf                           # all accepted, then this one
    s["tokens"][1, 1] = 5
    want = base.run(gpu_lib, s)
    base.check(s, want)
    assert list(want[1][[1, 3]]) == [1, 3] and want[0][1][1] == 777 and want[0][3][3] == 5
    for bad in (math.nan, math.inf, -math.inf):
        s["noise"][:] = bad
        got = base.run(gpu_lib, s)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_tokens_in_the_drafts_place(gpu_lib):
    """One buffer [rows, N + 1] that holds the drafts and takes the tokens, while
    other work keeps a row's blocks from starting together."""
    api = gpu_lib
    R, N, V = 64, 8, 129280
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    draft = (3 * rnd(R, N, V)).to(torch.bfloat16)
    target = torch.cat([draft, draft[:, :1]], 1)
    rows = torch.arange(R, device="cuda")
    T, noise = torch.ones(R, device="cuda"), -torch.log(-torch.log(
        torch.rand((R, V), generator=g, device="cuda").clamp(1e-9, 1 - 1e-7)))
    drafts = torch.randint(1, V, (R, N), generator=g, device="cuda")
    u = torch.zeros((R, N), device="cuda")
    # half of the rows are refused by a one-hot target at once, the others take all
    target[::2, 0, 0] = math.inf
    plan = api.Plan(V, 64, N, R)
    want, want_n = api.markov_verify(plan, target, drafts, draft, T, u, noise, rows)
    assert want_n[::2].eq(0).all() and want_n[1::2].eq(N).all() and want[::2, 0].eq(0).all()
    other, x = torch.cuda.Stream(), rnd(8192, 8192).to(torch.bfloat16)
    other.wait_stream(torch.cuda.current_stream())
    for k in range(30):
        with torch.cuda.stream(other):
            x @ x
        buf = torch.cat([drafts, torch.full((R, 1), -9, device="cuda")], 1)
        toks, n = api.markov_verify(plan, target, buf[:, :N], draft, T, u, noise, rows, tokens=buf)
        assert torch.equal(toks, want) and torch.equal(n, want_n), k
        toks, n = api.markov_verify(plan, target, drafts, draft, T, u, noise, rows)
        assert torch.equal(toks, want) and torch.equal(n, want_n), k
    assert api.markov_plan_status(plan) == 0
    plan.close()
