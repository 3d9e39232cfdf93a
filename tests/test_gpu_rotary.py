"""Rotary positions on the GPU against the formula in 64 bits."""
import math

import numpy as np
import pytest
import torch

from tests import serving_ref as ref

pytestmark = pytest.mark.gpu

SCALED = dict(factor=8.0, original_len=8192, low=1.0, high=32.0)


def _check(got, x, positions, f, interleaved, amplitude=1.0):
    want, tol = ref.rotary(x, positions, f, interleaved, amplitude)
    far = (got.double() - want).abs() - tol
    assert float(far.max()) <= 0, float(far.max())
    n = 2 * len(f)
    assert torch.equal(got[..., n:], x[..., n:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hk,d,rot", [(1, 1, 1, 16, 16), (1, 64, 8, 128, 128), (7, 5, 1, 64, 16), (72, 12, 3, 128, 64),
                                           (130, 2, 2, 96, 48), (5000, 3, 1, 64, 32), (3, 1, 1, 512, 512)])
def test_rotary(gpu_lib, dtype, interleaved, T, hq, hk, d, rot):
    api = gpu_lib
    g = torch.Generator(device="cuda").manual_seed(T + d)
    q = torch.randn((T, hq, d), generator=g, device="cuda").to(dtype)
    k = torch.randn((T, hk, d), generator=g, device="cuda").to(dtype)
    pos = torch.randint(0, 2 ** 31 - 1, (T,), generator=g, device="cuda", dtype=torch.int64).int()
    pos[0] = 0
    plan = api.RotaryPlan(d, rot, theta=10000.0, interleaved=interleaved)
    f = ref.frequencies(rot)
    qo, ko = api.markov_rotary(plan, q, k, pos)
    # an angle is p f_i with f_i in 64 bits: at 2^31 the plain form's is off by 2^-22 itself
    for got, x in ((qo, q), (ko, k)):
        near = pos < 2 ** 24
        near[0] = True
        _check(got[near], x[near], pos[near], f, interleaved)
    # in place
    q2, k2 = q.clone(), k.clone()
    api.markov_rotary(plan, q2, k2, pos, q_out=q2, k_out=k2)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    # one at a time
    assert torch.equal(api.markov_rotary(plan, q, None, pos)[0], qo)
    assert torch.equal(api.markov_rotary(plan, None, k, pos)[1], ko)
    plan.close()


def test_far_positions_keep_their_angle(gpu_lib):
    """Positions up to 2^31 - 1 and negative ones, against exact whole-number angles."""
    api = gpu_lib
    # 1/16, 1/1024 and 3/2^20 of a turn a position
    turns = [(1, 16), (1, 1024), (3, 2 ** 20), (1, 2 ** 31), (1, 3 * 2 ** 20), (0, 1), (-1, 64), (1, 1)]
    f = [2 * math.pi * a / b for a, b in turns]
    plan = api.RotaryPlan(16, 16, scaling="given", frequencies=f)
    pos = torch.tensor([0, 1, 2 ** 24 + 1, 2 ** 30 + 12345, 2 ** 31 - 1, -1, -2 ** 31, -987654321], dtype=torch.int32, device="cuda")
    x = torch.zeros((len(pos), 1, 16), device="cuda")
    x[..., :8] = 1.0
    got, _ = api.markov_rotary(plan, x, None, pos)
    for i, (a, b) in enumerate(turns):
        for t, p in enumerate(pos.tolist()):
            angle = 2 * math.pi * ((p * a) % b) / b
            # a frequency is a double: its rounding is worth 2^-53 of up to 2^31 turns; fp32 values of a
            # fp32 angle: 2^-22
            tol = 2.0 ** -22 + 2.0 ** -52 * abs(p) * abs(f[i])
            assert abs(float(got[t, 0, i]) - math.cos(angle)) <= tol, (i, p)
            assert abs(float(got[t, 0, 8 + i]) - math.sin(angle)) <= tol, (i, p)
    plan.close()


@pytest.mark.parametrize("scaling", ["linear", "base", "parts", "wavelength"])
@pytest.mark.parametrize("rot", [16, 64, 128])
def test_scaled_frequencies(gpu_lib, scaling, rot):
    api = gpu_lib
    f = ref.frequencies(rot, 500000.0, scaling, 8.0, 8192, 1.0, 32.0)
    amplitude = 0.1 * math.log(8.0) + 1 if scaling == "parts" else 1.0
    g = torch.Generator(device="cuda").manual_seed(rot)
    x = torch.randn((40, 3, 128), generator=g, device="cuda")
    pos = torch.randint(0, 70000, (40,), generator=g, device="cuda").int()
    plan = api.RotaryPlan(128, rot, theta=500000.0, scaling=scaling, **SCALED)
    _check(api.markov_rotary(plan, x, None, pos)[0], x, pos, f, False, amplitude)
    plan.close()
    plan = api.RotaryPlan(128, rot, theta=500000.0, scaling=scaling, amplitude=0.5, **SCALED)
    _check(api.markov_rotary(plan, x, None, pos)[0], x, pos, f, False, 0.5)
    plan.close()


def test_strides_streams_and_graphs(gpu_lib):
    api = gpu_lib
    g = torch.Generator(device="cuda").manual_seed(1)
    # queries and keys as slices of one projection's output, tokens inside heads
    qkv = torch.randn((37, 12, 64), generator=g, device="cuda").bfloat16()
    q, k = qkv[:, :6], qkv[:, 6:9]
    pos = torch.randint(0, 5000, (37,), generator=g, device="cuda").int()
    f = ref.frequencies(32)
    plan = api.RotaryPlan(64, 32)
    out = torch.zeros((6, 37, 64), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    before = qkv.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _, ko = api.markov_rotary(plan, q, k, pos, q_out=out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    _check(out, q, pos, f, False)
    _check(ko, k, pos, f, False)
    api.markov_rotary(plan, q, k, pos, q_out=q, k_out=k)          # in place in the projection
    assert torch.equal(q, out) and torch.equal(k, ko) and torch.equal(qkv[:, 9:], before[:, 9:])
    graph = torch.cuda.CUDAGraph()
    x, y = before[:, :6].contiguous(), torch.empty_like(out.contiguous())
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        api.markov_rotary(plan, x, None, pos, q_out=y)
    pos.add_(17)
    graph.replay()
    _check(y, x, pos, f, False)
    plan.close()


@pytest.mark.parametrize("interleaved", [False, True])
def test_wide_strides_of_each_type(gpu_lib, interleaved):
    """Keys of another number of heads and other strides than the queries, one of them in place."""
    api = gpu_lib
    g = torch.Generator(device="cuda").manual_seed(2)
    plan = api.RotaryPlan(96, 64, interleaved=interleaved)
    f = ref.frequencies(64)
    for dtype in (torch.float32, torch.float16, torch.bfloat16):
        wide = torch.randn((33, 7, 120), generator=g, device="cuda").to(dtype)
        q, k = wide[:, :4, :96], torch.randn((3, 33, 96), generator=g, device="cuda").to(dtype).transpose(0, 1)
        pos = torch.randint(0, 10 ** 6, (33,), generator=g, device="cuda").int()
        q0, k0, rest = q.clone(), k.clone(), wide[..., 96:].clone()
        _, ko = api.markov_rotary(plan, q, k, pos, q_out=q)
        _check(q, q0, pos, f, interleaved)
        _check(ko, k0, pos, f, interleaved)
        assert torch.equal(k, k0) and torch.equal(wide[..., 96:], rest)
    plan.close()


def test_nothing_to_do_and_special_values(gpu_lib):
    api = gpu_lib
    plan = api.RotaryPlan(16)
    q = torch.empty((0, 4, 16), dtype=torch.float16, device="cuda")
    api.markov_rotary(plan, q, None, torch.empty(0, dtype=torch.int32, device="cuda"))
    x = torch.zeros((2, 1, 16), device="cuda")
    x[0, 0, 1], x[1, 0, 2] = math.inf, math.nan
    y, _ = api.markov_rotary(plan, x, None, torch.zeros(2, dtype=torch.int32, device="cuda"))
    # only a NaN's or an infinity's own pair is touched
    assert math.isinf(float(y[0, 0, 1])) and math.isnan(float(y[1, 0, 2]))
    keep = np.ones((2, 16), bool)
    keep[0, [1, 9]], keep[1, [2, 10]] = False, False
    assert (y.cpu().numpy()[:, 0][keep] == 0).all()
    plan.close()


def test_refusals(gpu_lib):
    api = gpu_lib
    plan = api.RotaryPlan(64, 32)
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    q = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        api.markov_rotary(plan, q.double(), None, pos)
    with pytest.raises(TypeError):
        api.markov_rotary(plan, q, q.float(), pos)
    with pytest.raises(TypeError):
        api.markov_rotary(plan, q, None, pos.long())
    with pytest.raises(ValueError):
        api.markov_rotary(plan, q, None, pos[:2])
    with pytest.raises(ValueError):
        api.markov_rotary(plan, q[..., :32], None, pos)
    with pytest.raises(ValueError):
        api.markov_rotary(plan, None, None, pos)
    with pytest.raises(api.MarkovError):                          # rows 2 bytes off
        wide = torch.zeros((3, 2, 72), dtype=torch.bfloat16, device="cuda")
        api.markov_rotary(plan, wide[..., 1:65], None, pos)
    with pytest.raises(api.MarkovError):                          # in place with other strides
        a = torch.zeros((3, 4, 64), dtype=torch.bfloat16, device="cuda")
        api.markov_rotary(plan, a[:, :2], None, pos, q_out=a.view(4, 3, 64).transpose(0, 1)[:, :2])
    for bad in (dict(rot_dim=8), dict(rot_dim=80), dict(scaling="linear", factor=0.0), dict(theta=1.0),
                dict(scaling="parts", factor=2.0), dict(scaling="linear", factor=0.01)):
        with pytest.raises(api.MarkovError):
            api.RotaryPlan(64, **bad)
    with pytest.raises(ValueError):
        api.RotaryPlan(64, scaling="given")
    plan.close()


def test_head_counts_are_refused(gpu_lib):
    """More heads than 4096 together, and counts whose sum leaves 32 bits."""
    api = gpu_lib
    plan = api.RotaryPlan(64)
    pos = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = torch.zeros(64, dtype=torch.bfloat16, device="cuda")
    p, n = x.data_ptr(), pos.data_ptr()
    for hq, hk in ((4097, 0), (2048, 2049), (2 ** 31 - 1, 0), (2 ** 31 - 1, 1), (2 ** 31 - 1, 2 ** 31 - 1)):
        code = api.lib().markov_rotary(plan.handle, p, 64, 64, hq, p, 64, 64, hk, api.MARKOV_BF16, n, 1, p, 64, 64, p, 64, 64, None)
        assert code == 1                                          # EINVAL
    plan.close()
