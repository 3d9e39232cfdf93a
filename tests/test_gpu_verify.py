"""markov_verify on the GPU against its plain 64-bit form: sampled and greedy
rows, both logit types, masked and non-finite logits, refusals of drafts,
padding rows, odd shapes and strides, and its distribution."""
import math

import numpy as np
import pytest
import torch

from tests import paged_ref as ref

pytestmark = pytest.mark.gpu
SENT = -7
# a decision that fp32 may turn: probabilities are within 1e-5 of each other
NEAR = 1e-4


def make(R, N, V, seed=0, target=torch.bfloat16, draft=torch.bfloat16, temps=(0.0, 0.6, 1.0), std=3.0, shift=0.7):
    g = torch.Generator().manual_seed(seed)
    d = torch.randn((R, N, V), generator=g) * std
    t = torch.cat([d, torch.randn((R, 1, V), generator=g) * std], 1) + torch.randn((R, N + 1, V), generator=g) * shift
    T = torch.tensor([temps[b % len(temps)] for b in range(R)], dtype=torch.float32)
    d, t = d.to(draft), t.to(target)
    Ts = torch.where(T > 0, T, 1.0)[:, None, None]
    e = -torch.log(-torch.log(torch.rand((R, N, V), generator=g).clamp(1e-9, 1 - 1e-7)))
    x = (d.float() / Ts + torch.where(T > 0, 1.0, 0.0)[:, None, None] * e).argmax(-1)
    return dict(target=t, draft=d, tokens=x, T=T, u=torch.rand((R, N), generator=g),
                noise=-torch.log(-torch.log(torch.rand((R, V), generator=g).clamp(1e-9, 1 - 1e-7))),
                idx=torch.arange(R))


def run(api, s, plan=None, probs=True):
    R, N, V = s["draft"].shape
    own = plan is None
    plan = plan or api.Plan(V, 64, N, R)
    d = {k: v.cuda() for k, v in s.items()}
    toks = torch.full((R, N + 1), SENT, dtype=torch.int64, device="cuda")
    acc = torch.full((R,), SENT, dtype=torch.int32, device="cuda")
    p, q = (torch.full((R, N), float(SENT), device="cuda") for _ in range(2)) if probs else (None, None)
    api.markov_verify(plan, d["target"], d["tokens"], d["draft"], d["T"], d["u"], d["noise"], d["idx"], toks, acc, p, q)
    assert api.markov_plan_status(plan) == 0
    if own:
        plan.close()
    return [None if x is None else x.cpu().numpy() for x in (toks, acc, p, q)]


def check(s, got):
    toks, acc, p, q = got
    R, N, V = s["draft"].shape
    t, d = s["target"].float().numpy(), s["draft"].float().numpy()
    sure = 0
    for b in range(R):
        if s["idx"][b] < 0:
            assert (toks[b] == SENT).all() and acc[b] == SENT and (p[b] == SENT).all() and (q[b] == SENT).all()
            continue
        wt, wn, wp, wq, near = ref.verify_row(t[b], s["tokens"][b].numpy(), d[b], float(s["T"][b]),
                                              s["u"][b].numpy(), s["noise"][b].numpy())
        # exponents of fp32 logits are within 2^-22 of |l - m| / T <= 100, sums within 1e-6
        assert np.allclose(p[b], wp, rtol=5e-5, atol=1e-30) and np.allclose(q[b], wq, rtol=5e-5, atol=1e-30), b
        if near > NEAR:
            sure += 1
            assert list(toks[b]) == wt and acc[b] == wn, (b, list(toks[b]), wt, near)
    return sure


F = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("target", F)
@pytest.mark.parametrize("draft", F)
@pytest.mark.parametrize("R,N,V", [(1, 1, 16), (3, 4, 4096), (6, 8, 5008), (2, 16, 2064), (40, 2, 1040)])
def test_rows(gpu_lib, R, N, V, target, draft):
    s = make(R, N, V, seed=R + N, target=target, draft=draft)
    s["idx"][2::5] = -1
    live = int((s["idx"] >= 0).sum())
    assert check(s, run(gpu_lib, s)) >= 0.9 * live


@pytest.mark.parametrize("R", [1, 8, 64])
def test_full_vocabulary(gpu_lib, R):
    s = make(R, 2, 129280, seed=R, temps=(0.8, 0.0, 1.3))
    assert check(s, run(gpu_lib, s)) >= 0.9 * R
    s = make(2, 1, 262144, seed=R, temps=(0.7,), target=torch.float32)
    assert check(s, run(gpu_lib, s)) >= 1


def test_all_accepted_and_none(gpu_lib):
    s = make(4, 5, 4096, seed=1, shift=0.0, temps=(0.0, 1.0))
    toks, acc, p, q = got = run(gpu_lib, s)
    check(s, got)
    assert (acc == 5).all() and (toks[:, :5] == s["tokens"].numpy()).all() and (toks[:, 5] >= 0).all()
    s["tokens"] = (s["tokens"] + 1) % 4096
    s["u"] = torch.full_like(s["u"], 0.9999)
    s["draft"], s["target"] = -s["target"][:, :5].clone(), s["target"]
    check(s, run(gpu_lib, s))


def test_equal_distributions_refused_by_a_uniform_of_one(gpu_lib):
    """u q < p fails although p == q everywhere: the token is drawn from p."""
    s = make(3, 2, 4096, seed=2, shift=0.0, temps=(1.0,))
    s["u"][:, 1] = 1.0
    toks, acc, _, _ = run(gpu_lib, s)
    t = s["target"].float()[:, 1]
    want = (torch.log_softmax(t, -1) + s["noise"]).argmax(-1).numpy()
    assert (acc == 1).all() and (toks[:, 1] == want).all() and (toks[:, 2] == -1).all()


def test_masked_logits(gpu_lib):
    """-inf and the types' lowest values in most places, whole segments of them."""
    for low in (-math.inf, float(torch.finfo(torch.bfloat16).min)):
        s = make(6, 3, 20000, seed=3)
        keep = torch.zeros(20000, dtype=torch.bool)
        keep[12000:12040] = True
        x = s["target"].clone()
        x[..., ~keep] = low
        s["target"] = x
        s["tokens"][:, :2] = 12000 + s["tokens"][:, :2] % 40
        assert check(s, run(gpu_lib, s)) >= 5
        y = s["draft"].clone()
        y[..., ~keep] = low
        s["draft"] = y
        assert check(s, run(gpu_lib, s)) >= 5


def test_one_key_left_and_none(gpu_lib):
    s = make(4, 2, 4096, seed=4, temps=(1.0,))
    s["target"][0] = -math.inf
    s["target"][0, :, 77] = 1.0
    s["target"][1] = -math.inf                                # nothing left: id 0
    s["draft"][2, :, :] = -math.inf
    s["draft"][3, 0, :] = -math.inf
    s["draft"][3, 0, 5] = 0.0
    s["tokens"][0] = 77
    s["tokens"][3, 0] = 5
    got = run(gpu_lib, s)
    check(s, got)
    assert got[1][0] == 2 and list(got[0][0]) == [77, 77, 77] and got[0][1][got[1][1]] == 0


def test_nan_and_infinite_logits(gpu_lib):
    """The lowest NaN id, else the lowest +inf id, has all the probability."""
    s = make(6, 3, 20000, seed=5, temps=(1.0, 0.0))
    s["target"][0, 0, [9000, 15000]] = math.nan
    s["target"][1, 1, [19999, 3]] = math.inf
    s["target"][2, 0, 7] = math.inf
    s["target"][2, 0, 8] = math.nan
    s["draft"][3, 0, 10] = math.nan
    s["draft"][4, 1, [11, 12]] = math.inf
    s["tokens"][3, 0], s["tokens"][4, 1], s["tokens"][0, 0] = 10, 11, 9000
    s["noise"][0, :100] = math.nan                            # not read where one id has it all
    s["u"][0] = 0.0
    s["u"][0, 1] = 1.0
    s["noise"][0] = torch.randn(20000)
    check(s, run(gpu_lib, s))


def test_extreme_temperatures_and_logits(gpu_lib):
    s = make(5, 2, 4096, seed=6, target=torch.float32, draft=torch.float32, temps=(1e-3, 1e-38, 100.0, -1.0, math.nan))
    check(s, run(gpu_lib, s))
    s = make(2, 2, 4096, seed=7, target=torch.float32, draft=torch.float32, temps=(0.5,))
    s["target"][0, 0, 100], s["target"][0, 1, 50] = 3e38, -3e38
    s["tokens"][0, 0] = 100
    check(s, run(gpu_lib, s))


def test_draft_ids_outside_the_vocabulary_are_refused(gpu_lib):
    s = make(4, 3, 4096, seed=8, shift=0.0, temps=(1.0, 0.0))
    s["tokens"][0, 0], s["tokens"][1, 1], s["tokens"][2, 2] = -1, 4096, 2 ** 40
    toks, acc, p, q = got = run(gpu_lib, s)
    check(s, got)
    assert list(acc) == [0, 1, 2, 3] and p[0, 0] == 0 and q[1, 1] == 0


def test_strides_streams_and_repeats(gpu_lib):
    api = gpu_lib
    R, N, V = 5, 3, 4096
    s = make(R, N, V, seed=9)
    want = run(api, s)
    check(s, want)
    d = {k: v.cuda() for k, v in s.items()}
    wide_t = torch.full((R, N + 3, V + 64), math.nan, dtype=torch.bfloat16, device="cuda")
    wide_t[:, 1:N + 2, 8:V + 8] = d["target"]
    wide_c = torch.full((R, N + 1, V + 16), math.nan, dtype=torch.bfloat16, device="cuda")
    wide_c[:, :N, :V] = d["draft"]
    tk = torch.zeros((R, N + 2), dtype=torch.int64, device="cuda")
    tk[:, :N] = d["tokens"]
    un = torch.zeros((R, N + 1), device="cuda")
    un[:, 1:] = d["u"]
    nz = torch.zeros((R, V + 4), device="cuda")
    nz[:, 4:] = d["noise"]
    out = torch.full((R, N + 5), SENT, dtype=torch.int64, device="cuda")
    plan = api.Plan(V, 64, N, R)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for stream in (None, st, st):
        out.fill_(SENT)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        toks, acc = api.markov_verify(plan, wide_t[:, 1:N + 2, 8:V + 8], tk[:, :N], wide_c[:, :N, :V], d["T"], un[:, 1:],
                                      nz[:, 4:], d["idx"], tokens=out[:, 1:N + 2], stream=stream)
        torch.cuda.synchronize()
        assert np.array_equal(toks.cpu().numpy(), want[0]) and np.array_equal(acc.cpu().numpy(), want[1])
        assert bool((out[:, 0] == SENT).all()) and bool((out[:, N + 2:] == SENT).all())
    plan.close()


def test_distribution(gpu_lib):
    """Over many draws the first token out is distributed as the target's,
    whatever the draft: each count is within five deviations."""
    api = gpu_lib
    R, V, calls = 250, 16, 16
    g = torch.Generator().manual_seed(10)
    tl, dl = torch.randn(V, generator=g), torch.randn(V, generator=g)
    plan = api.Plan(V, 64, 1, R)
    seen = np.zeros(V)
    for _ in range(calls):
        s = make(R, 1, V, seed=0, temps=(1.0,))
        s["target"], s["draft"] = tl.to(torch.bfloat16).expand(R, 2, V).contiguous(), dl.to(torch.bfloat16).expand(R, 1, V).contiguous()
        rnd = lambda *sh: torch.rand(sh, generator=g).clamp(1e-9, 1 - 1e-7)  # noqa: E731
        s["tokens"] = (s["draft"][:, 0].float() - torch.log(-torch.log(rnd(R, V)))).argmax(-1)[:, None]
        s["u"], s["noise"] = torch.rand((R, 1), generator=g), -torch.log(-torch.log(rnd(R, V)))
        seen += np.bincount(run(api, s, plan, probs=False)[0][:, 0], minlength=V)
    n = R * calls
    p = torch.softmax(tl.to(torch.bfloat16).double(), -1).numpy()
    assert (np.abs(seen - n * p) <= 5 * np.sqrt(n * p * (1 - p)) + 1).all()
    plan.close()


def test_after_a_chain_call(gpu_lib):
    """The drafts and the cache of a chain call, greedy: the target that drew
    them accepts them all."""
    api = gpu_lib
    from draft_token_markov_gb300 import workloads as W
    w = W.small(4096, 64, 5, 4, W.GUMBEL, seed=5, padding_rows=(1,), temperatures=(0.0, 1.0))
    h, e = W.make_weights(w)
    c = {k: v.cuda() for k, v in W.make_call(w).items()}
    plan = api.Plan(w.vocab, w.rank, w.steps, w.rows)
    toks, cache = api.markov_chain_sample(plan, c["base"], h.cuda(), e.cuda(), c["anchor"], c["temperature"],
                                          c["seeds"], c["row_state_idx"], w.mode)
    target = torch.cat([cache, cache[:, :1]], 1).contiguous()
    noise = api.markov_gumbel_noise(c["seeds"] + 1, c["temperature"], c["row_state_idx"], 1, w.vocab)
    u = torch.full((w.rows, w.steps), 0.99, device="cuda")
    out, acc = api.markov_verify(plan, target, toks, cache, c["temperature"], u, noise, c["row_state_idx"])
    assert api.markov_plan_status(plan) == 0
    for b in range(w.rows):
        if b != 1:
            assert int(acc[b]) == w.steps and torch.equal(out[b, :w.steps], toks[b])
            assert 0 <= int(out[b, w.steps]) < w.vocab
    plan.close()


def test_refusals(gpu_lib):
    api = gpu_lib
    s = make(3, 2, 4096, seed=11)
    d = {k: v.cuda() for k, v in s.items()}
    plan = api.Plan(4096, 64, 2, 3)

    def verify(**kw):
        a = dict(d)
        out = kw.pop("out", torch.full((3, 3), SENT, dtype=torch.int64, device="cuda"))
        more = {k: kw.pop(k) for k in ("target_probs", "draft_probs") if k in kw}
        a.update(kw)
        try:
            api.markov_verify(plan, a["target"], a["tokens"], a["draft"], a["T"], a["u"], a["noise"], a["idx"], out, **more)
        finally:
            torch.cuda.synchronize()
            assert bool((out == SENT).all())

    big = torch.zeros((3, 3, 4104), dtype=torch.bfloat16, device="cuda")
    for kw, err in [(dict(target=d["target"].half()), TypeError), (dict(target=d["target"][:, :2]), ValueError),
                    (dict(target=d["target"].cpu()), TypeError), (dict(tokens=d["tokens"].int()), TypeError),
                    (dict(draft=d["draft"][:, :1]), ValueError), (dict(T=d["T"].double()), TypeError),
                    (dict(u=d["u"][:, :1]), ValueError), (dict(noise=d["noise"][:, :4000]), ValueError),
                    (dict(idx=d["idx"][:2]), ValueError), (dict(target=big[:, :, 4:4100]), api.MarkovError),
                    (dict(target_probs=torch.zeros((3, 2), device="cuda")), api.MarkovError),
                    (dict(out=torch.full((3, 2), SENT, dtype=torch.int64, device="cuda")), ValueError)]:
        with pytest.raises(err):
            verify(**kw)
    four = {k: torch.cat([v, v[:1]]) for k, v in d.items()}
    with pytest.raises(api.MarkovError):                      # more rows than the plan's
        api.markov_verify(plan, four["target"], four["tokens"], four["draft"], four["T"], four["u"], four["noise"], four["idx"])
    api.markov_plan_inject_status(plan, 4)
    verify()                                                  # a pending status: nothing is written
    assert api.markov_plan_status(plan) == 4
    plan.close()
