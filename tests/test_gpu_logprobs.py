"""Log probabilities, ranks, entropies and alternatives on the GPU against their
plain 64-bit form."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests import serving_ref as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _compare(api, logits, tokens, temperature, top, stream=None):
    """Whole numbers equal.  Log probabilities: l - m is rounded once, as are its
    product with log2(e) / T and the constant (3 * 2^-24 of d), 2^x, sums and ln are
    within 2^-20 together, the last steps within 2^-22 of the result: 1e-6 (1 + |d|)
    covers them.  Entropies are means of as much."""
    rows, V = logits.shape
    got = api.markov_logprobs(logits, tokens, temperature, top, stream=stream)
    l = logits.double().cpu().numpy()
    for i in range(rows):
        t = -1 if tokens is None else int(tokens[i])
        T = 1.0 if temperature is None else float(temperature[i])
        if tokens is not None and not 0 <= t < V:
            continue
        p, rank, entropy, ids, top_p = ref.logprobs(l[i], t, T, top)
        near = lambda x, y: x == y or abs(x - y) <= 1e-6 * (1 + abs(y))  # noqa: E731
        if tokens is not None:
            assert near(float(got.logprobs[i]), p), (i, float(got.logprobs[i]), p)
            assert int(got.ranks[i]) == rank, i
        assert abs(float(got.entropy[i]) - entropy) <= 1e-6 * (1 + entropy) * 4, (i, float(got.entropy[i]), entropy)
        if top:
            assert got.top_ids[i].tolist() == ids.tolist(), i
            for a, b in zip(got.top_logprobs[i].tolist(), top_p):
                assert near(a, b), (i, a, b)
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,V,top", [(1, 1, 1), (3, 2, 2), (5, 7, 3), (2, 33, 32), (4, 1000, 20), (3, 4096, 5),
                                        (9, 16384, 32), (3, 16385, 8), (2, 50257, 20), (5, 129280, 20), (2, 262144, 32),
                                        (1, 262143, 0)])
def test_logprobs(gpu_lib, dtype, rows, V, top):
    g = torch.Generator(device="cuda").manual_seed(V + rows)
    logits = (torch.randn((rows, V), generator=g, device="cuda") * 3).to(dtype)
    tokens = torch.randint(0, V, (rows,), generator=g, device="cuda")
    T = torch.tensor([0.7, 1.0, 0.0, 2.0, math.nan, -1.0, 0.05, 1.3, 5.0], device="cuda")[:rows]
    _compare(gpu_lib, logits, tokens, T, top)
    _compare(gpu_lib, logits, tokens, None, top)
    _compare(gpu_lib, logits, None, T, top)


def test_unaligned_rows(gpu_lib):
    """Rows that begin at every place of a 16-byte vector."""
    g = torch.Generator(device="cuda").manual_seed(3)
    for dtype, V in ((torch.bfloat16, 20001), (torch.float32, 10003)):
        wide = torch.full((9, V + 1), 1000.0, device="cuda").to(dtype)      # what lies beside a row is larger
        wide[:, :V] = torch.randn((9, V), generator=g, device="cuda").to(dtype)
        tokens = torch.randint(0, V, (9,), generator=g, device="cuda")
        _compare(gpu_lib, wide[:, :V], tokens, None, 7)
        _compare(gpu_lib, wide.view(-1)[3:].as_strided((8, V), (V + 1, 1), 3), None, None, 4)


def test_ties_and_masks(gpu_lib):
    inf = math.inf
    V = 70000
    rows = []
    rows.append(torch.zeros(V))                                             # every logit the same
    x = torch.full((V,), -inf); x[[5, 69999, 40000]] = torch.tensor([1.0, 2.0, 1.0]); rows.append(x)   # three allowed
    x = torch.full((V,), -inf); x[12345] = -3.0; rows.append(x)             # one
    x = torch.full((V,), float(torch.finfo(torch.bfloat16).min)); x[::1000] = 0.5; rows.append(x)       # masked by the lowest value
    rows.append(torch.where(torch.arange(V) % 3 == 0, 1.0, -0.0))           # many ties at the bound
    x = torch.zeros(V); x[V // 2:] = -0.0; rows.append(x)                   # -0 equals 0
    rows.append(torch.arange(V).float() / 1000)                             # rising: the last ids
    rows.append(-torch.arange(V).float() / 1000)
    x = torch.zeros(V); x[torch.arange(0, 2048 * 8, 8)] = torch.arange(2048) / 512.0; rows.append(x)   # the large ones with few threads
    logits = torch.stack(rows).cuda()
    g = torch.Generator().manual_seed(1)
    for dtype in (torch.bfloat16, torch.float32):
        l = logits.to(dtype)
        for tokens in (torch.tensor([0, 5, 12345, 1000, 3, V // 2, V - 1, 0, 16376]), torch.randint(0, V, (9,), generator=g),
                       torch.full((9,), V - 1)):
            for top in (1, 20, 32):
                _compare(gpu_lib, l, tokens.cuda(), None, top)


def test_rows_that_are_not_finite(gpu_lib):
    inf, nan = math.inf, math.nan
    V = 40000
    g = torch.Generator(device="cuda").manual_seed(5)
    l = torch.randn((8, V), generator=g, device="cuda")
    l[0] = -inf                                                             # nothing is left
    l[1, 777] = inf
    l[2, [39999, 5000]] = inf
    l[3, 39000] = nan
    l[4, [100, 30000]] = nan
    l[4, 50] = inf
    l[5] = nan
    l[6, :V // 2] = -inf                                                    # half of the slices empty
    l[7, 3] = -inf
    for dtype in (torch.bfloat16, torch.float32):
        for tokens in ([0, 777, 5000, 39000, 30000, 0, 3, 3], [1, 0, 39999, 0, 50, V - 1, V - 1, 4]):
            _compare(gpu_lib, l.to(dtype), torch.tensor(tokens, device="cuda"), None, 6)


def test_temperatures(gpu_lib):
    g = torch.Generator(device="cuda").manual_seed(6)
    l = torch.randn((6, 5000), generator=g, device="cuda") * 4
    l[:, 100:200] = -math.inf
    T = torch.tensor([math.inf, 1e-3, 1e-30, 100.0, 1e30, 0.3], device="cuda")
    tokens = l.argmax(1)
    tokens[0] = 17
    got = gpu_lib.markov_logprobs(l, tokens, T, 3)
    # uniform over what is not masked
    assert abs(float(got.logprobs[0]) + math.log(4900)) < 1e-5 and abs(float(got.entropy[0]) - math.log(4900)) < 1e-5
    # a temperature near 0: the argmax alone
    assert got.logprobs[2] == 0 and got.entropy[2] == 0 and got.top_logprobs[2, 1] < -1e29
    keep = [1, 3, 4, 5]
    _compare(gpu_lib, l[keep], tokens[keep], T[keep], 3)


def test_rows_left_alone(gpu_lib):
    api = gpu_lib
    g = torch.Generator(device="cuda").manual_seed(7)
    l = torch.randn((6, 3000), generator=g, device="cuda")
    l[2] = math.nan
    tokens = torch.tensor([4, -1, 3000, 2 ** 40, -2 ** 62, 2999], device="cuda")
    out = dict(logprobs=torch.full((6,), -7.0, device="cuda"), entropy=torch.full((6,), -7.0, device="cuda"),
               ranks=torch.full((6,), -7, dtype=torch.int32, device="cuda"),
               top_ids=torch.full((6, 4), -7, dtype=torch.int32, device="cuda"),
               top_logprobs=torch.full((6, 4), -7.0, device="cuda"))
    api.markov_logprobs(l, tokens, None, 4, **out)
    for x in out.values():
        assert (x[1:5] == -7).all() and not (x[0] == -7).any() and not (x[5] == -7).any()


def test_streams_graphs_and_two_calls_at_once(gpu_lib):
    api = gpu_lib
    g = torch.Generator(device="cuda").manual_seed(8)
    l = torch.randn((40, 30000), generator=g, device="cuda").bfloat16()
    tokens = torch.randint(0, 30000, (40,), generator=g, device="cuda")
    want = api.markov_logprobs(l, tokens, None, 5)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [api.markov_logprobs(l, tokens, None, 5, stream=s) for s in streams]
    torch.cuda.synchronize()
    for x in got:
        assert all(torch.equal(a, b) for a, b in zip(x, want))
    graph = torch.cuda.CUDAGraph()
    out = dict(logprobs=torch.zeros_like(want.logprobs), ranks=torch.zeros_like(want.ranks),
               entropy=torch.zeros_like(want.entropy), top_ids=torch.zeros_like(want.top_ids),
               top_logprobs=torch.zeros_like(want.top_logprobs))
    with torch.cuda.graph(graph):
        api.markov_logprobs(l, tokens, None, 5, **out)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[n], getattr(want, n)) for n in out)


def test_the_first_call_may_be_captured():
    """In a process of its own: nothing has to be called before a capture."""
    code = """
import torch
from draft_token_markov_gb300 import api
l = torch.randn((3, 5000), device="cuda")
t = torch.tensor([1, 2, 3], device="cuda")
out = [torch.zeros(3, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(3, device="cuda")]
api.lib()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    api.markov_logprobs(l, t, None, 0, logprobs=out[0], ranks=out[1], entropy=out[2])
g.replay()
torch.cuda.synchronize()
want = torch.log_softmax(l.double(), -1).gather(1, t[:, None])[:, 0]
assert (out[0].double() - want).abs().max() < 1e-5
"""
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert done.returncode == 0, done.stderr[-2000:]


def test_many_rows(gpu_lib):
    """More rows than a grid's second dimension has."""
    api = gpu_lib
    g = torch.Generator(device="cuda").manual_seed(9)
    l = torch.randn((70001, 24), generator=g, device="cuda")
    tokens = torch.randint(0, 24, (70001,), generator=g, device="cuda")
    got = api.markov_logprobs(l, tokens, None, 2)
    want = torch.log_softmax(l.double(), -1)
    assert (got.logprobs.double() - want.gather(1, tokens[:, None])[:, 0]).abs().max() < 1e-5
    assert torch.equal(got.top_ids[:, 0].long(), l.argmax(1))
    assert torch.equal(got.ranks.long(), (l > l.gather(1, tokens[:, None])).sum(1))


def test_refusals(gpu_lib):
    api = gpu_lib
    l = torch.zeros((3, 100), device="cuda")
    tokens = torch.zeros(3, dtype=torch.int64, device="cuda")
    with pytest.raises(TypeError):
        api.markov_logprobs(l.half(), tokens)
    with pytest.raises(TypeError):
        api.markov_logprobs(l.cpu(), tokens)
    with pytest.raises(TypeError):
        api.markov_logprobs(l, tokens.int())
    with pytest.raises(ValueError):
        api.markov_logprobs(l[None], tokens)
    with pytest.raises(ValueError):
        api.markov_logprobs(l, tokens[:2])
    with pytest.raises(ValueError):
        api.markov_logprobs(l.t().contiguous().t(), tokens)
    with pytest.raises(ValueError):
        api.markov_logprobs(l, logprobs=torch.zeros(3, device="cuda"))
    for top in (33, -1):
        with pytest.raises(api.MarkovError):
            api.markov_logprobs(l, tokens, None, top, top_ids=torch.zeros((3, 33), dtype=torch.int32, device="cuda"),
                                top_logprobs=torch.zeros((3, 33), device="cuda"))
    with pytest.raises(api.MarkovError):
        api.markov_logprobs(l[:, :5], tokens, None, 6)
    with pytest.raises(api.MarkovError):
        api.markov_logprobs(torch.zeros((3, 262145), device="cuda"), tokens)
    with pytest.raises(api.MarkovError):                          # rows that overlap
        api.markov_logprobs(l.view(-1).as_strided((3, 100), (50, 1)), tokens)
    assert np.isfinite(api.markov_logprobs(l, tokens).entropy.cpu().numpy()).all()
