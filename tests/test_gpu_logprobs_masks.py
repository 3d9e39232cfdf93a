"""Log probabilities of rows whose masked logits are large finite values, and of
logits far from 0, against their 64-bit form.

Tolerance of ln p = (d - log2 Z) ln 2: the difference to the maximum, log2(e) / T, their
product, the subtraction and the last product are rounded, six times 2^-24 of the
result, which 2^-21 of it covers; 2^x, the sums and log2 are within 2^-20 together; the
maximum's own product with log2(e) / T, which the weights are taken against, is below
2^27, so an exponent is below 4 where its weight is 1 and rounded by 2^-22, in the sums
and where they are put right: 2^-21.  Entropies are means of as much, of terms as large
as themselves."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

V = 129280
TEMPERATURES = (0.3, 0.6, 0.7, 1.0, 2.0)
TOP = 20


def _masks(g):
    """[patterns, V]: which ids are left out."""
    ids = torch.arange(V, device="cuda")
    u = torch.rand((3, V), generator=g, device="cuda")
    masks = [u[0] < 0.5, u[1] < 0.9, u[2] < 0.99, ids < 8192, ids < V // 2, ids >= V - 8192, (ids // 4096) % 2 == 0]
    return torch.stack(masks)


def _check(api, l, tokens, T, top=TOP, copies=1):
    """A call on `copies` of the rows, one after the other; compares the first and the last."""
    rows = len(l)
    x = l.double()
    own = x.gather(1, tokens[:, None])
    ids = torch.arange(l.shape[1], device="cuda")
    rank = ((x > own) | ((x == own) & (ids < tokens[:, None]))).sum(1)
    first = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :top]
    p = torch.log_softmax((x - x.amax(1, keepdim=True)) / T.double()[:, None], 1)
    q = p.exp()
    entropy = -torch.where(q > 0, q * p, 0.0).sum(1)
    got = api.markov_logprobs(l.repeat(copies, 1), tokens.repeat(copies), T.repeat(copies), top)

    def near(a, b, what):
        b32 = b.float().double()                      # beyond fp32's range: -inf
        tol = 1.5 * 2.0 ** -20 + 2.0 ** -21 * b.abs()
        ok = (a.double() == b32) | ((a.double() - b).abs() <= tol)
        assert bool(ok.all()), (what, ok.logical_not().nonzero()[:3].tolist(), a[~ok][:3].tolist(), b[~ok][:3].tolist())

    for i in {0, copies - 1}:
        part = slice(i * rows, (i + 1) * rows)
        assert torch.equal(got.ranks[part].long(), rank)
        assert torch.equal(got.top_ids[part].long(), first)
        near(got.logprobs[part], p.gather(1, tokens[:, None])[:, 0], "logprobs")
        near(got.top_logprobs[part], p.gather(1, first), "alternatives")
        worst = ((got.entropy[part].double() - entropy).abs() - 4 * (1.5 * 2.0 ** -20 + 2.0 ** -21 * entropy)).max()
        assert float(worst) <= 0, ("entropy", got.entropy[part].tolist(), entropy.tolist())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("value", ["min", -1e32, -1e31, -1e30, -1e20, -1e10, -1e9, -3e8, -1e4, -math.inf])
def test_finite_masks(gpu_lib, dtype, value):
    """A cluster of blocks a row, then one block a row."""
    g = torch.Generator(device="cuda").manual_seed(11)
    value = torch.finfo(dtype).min if value == "min" else value
    masks = _masks(g)
    l = (torch.randn(masks.shape, generator=g, device="cuda") * 3).masked_fill(masks, value).to(dtype)
    n = len(TEMPERATURES)
    T = torch.tensor(TEMPERATURES, device="cuda").repeat(len(l))
    l, masks = l.repeat_interleave(n, 0), masks.repeat_interleave(n, 0)
    live = torch.where(masks, -1.0, torch.rand(masks.shape, generator=g, device="cuda")).argmax(1)
    hidden = torch.where(masks, torch.rand(masks.shape, generator=g, device="cuda"), -1.0).argmax(1)
    for copies in (1, 10):
        _check(gpu_lib, l, live, T, copies=copies)
        _check(gpu_lib, l, hidden, T, copies=copies)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("base,spread", [(0.0, 1e10), (0.0, 1e30), (1e10, 1e4), (-1e10, 1e4), (3e9, 300.0), (-3e9, 300.0),
                                         (9.3e7, 30.0), (-9.3e7, 30.0), (1.9e8, 30.0), (-1.9e8, 30.0), (1e6, 3.0), (-1e6, 3.0)])
def test_logits_far_from_zero(gpu_lib, dtype, base, spread):
    """Around 2^27 = max / T log2(e), where the weights are taken in another way, and beyond."""
    g = torch.Generator(device="cuda").manual_seed(12)
    l = (torch.randn((len(TEMPERATURES), V), generator=g, device="cuda").double() * spread + base).to(dtype)
    # few ids at the top, so that the order of equals ends among them
    at = torch.randint(0, V, (len(l), 24), generator=g, device="cuda")
    step = max(spread, abs(base) / 64) / 2
    l.scatter_(1, at, (base + 6 * spread + step * torch.arange(24, device="cuda").double())[None].expand(len(l), -1).to(dtype))
    T = torch.tensor(TEMPERATURES, device="cuda")
    tokens = torch.randint(0, V, (len(l),), generator=g, device="cuda")
    for copies in (1, 70):
        _check(gpu_lib, l, tokens, T, copies=copies)
        _check(gpu_lib, l, at[:, 3].contiguous(), T, copies=copies)


def test_a_thread_may_meet_masks_first_or_last(gpu_lib):
    """Rows of several turns where some threads see masked logits alone in their first turns, in
    their last ones, or in all of them."""
    g = torch.Generator(device="cuda").manual_seed(13)
    for dtype, lowest in ((torch.bfloat16, -1e31), (torch.float32, -3.4e38)):
        vec = 8 if dtype == torch.bfloat16 else 4
        lane = torch.arange(V, device="cuda") // vec % 256           # the thread, rows being aligned and whole
        turn = torch.arange(V, device="cuda") // (vec * 1024)
        masks = torch.stack([turn == 0, turn == int(turn.max()), lane < 128, lane % 32 == 5, (turn + lane) % 2 == 0,
                             (lane < 250) | (turn > 0)])
        l = (torch.randn(masks.shape, generator=g, device="cuda") * 3).masked_fill(masks, lowest).to(dtype)
        T = torch.tensor([0.6, 0.7, 1.0, 2.0, 0.05, 1.0], device="cuda")
        tokens = torch.randint(0, V, (len(l),), generator=g, device="cuda")
        for copies in (1, 60):
            _check(gpu_lib, l, tokens, T, copies=copies)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("top", [1e37, 3.3e38, -2e38])
def test_differences_that_leave_the_range_of_fp32(gpu_lib, dtype, top):
    """The lowest value's distance to the maximum need not be a float where the log
    probability is one."""
    lowest = torch.finfo(dtype).min
    l = torch.full((6, 3000), lowest, dtype=dtype, device="cuda")
    l[:, 7::500] = top
    T = torch.tensor([1.0, 2.0, 5.5, 9.0, 0.5, 0.01], device="cuda")
    for token in (0, 7, 2999):
        _check(gpu_lib, l, torch.full((6,), token, device="cuda"), T, top=9, copies=1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_uniform_over_finite_masks_too(gpu_lib, dtype):
    """T = +inf: every logit but -inf counts alike, however far from the maximum; one block
    of a cluster may have nothing but masks."""
    l = torch.full((3, V), torch.finfo(dtype).min, dtype=dtype, device="cuda")
    l[:, :100] = 3e38
    l[1, 5000:] = -math.inf
    l[2, 50:V - 7] = -math.inf
    T = torch.full((3,), math.inf, device="cuda")
    for copies in (1, 150):
        got = gpu_lib.markov_logprobs(l.repeat(copies, 1), torch.full((3 * copies,), 49, device="cuda"), T.repeat(copies), 3)
        for i, n in enumerate((V, 5000, 57)):
            # the logarithm of a count: 2^-20 and two roundings of it
            tol = 2.0 ** -20 + 2.0 ** -22 * math.log(n)
            for x, want in ((got.logprobs, -math.log(n)), (got.entropy, math.log(n)), (got.top_logprobs[:, 2], -math.log(n))):
                assert float((x[i::3].double() - want).abs().max()) <= tol, (i, n)


@pytest.mark.parametrize("base", [1e8, -1e8, 4e8])
def test_many_equal_logits_far_from_zero(gpu_lib, base):
    """fp32 logits a few units in the last place apart: sums of many equal terms."""
    g = torch.Generator(device="cuda").manual_seed(14)
    l = (torch.randn((8, V), generator=g, device="cuda").double() + base).float()
    l[4:, ::7] = -1e9
    T = torch.tensor([0.46, 0.55, 0.63, 0.68, 0.69, 0.91, 0.98, 0.5], device="cuda")
    tokens = torch.randint(0, V, (8,), generator=g, device="cuda")
    for copies in (1, 50):
        _check(gpu_lib, l, tokens, T, copies=copies)
