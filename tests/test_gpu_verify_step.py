"""The verify step's calls together (examples/verify_step.py): at temperature 0
every token that comes out is the target model's greedy choice after the
tokens before it, computed densely in 64 bits; pages come back."""
import importlib.util
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(gpu_lib):
    spec = importlib.util.spec_from_file_location("verify_step", os.path.join(ROOT, "examples", "verify_step.py"))
    m = sys.modules[spec.name] = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def dense_logits(model, tokens, window, sinks):
    """The toy target's logits after each prefix, in 64 bits on its BF16 weights."""
    d = lambda w: w.double()  # noqa: E731
    x = d(model.embed)[tokens]
    q, k, v = ((x @ d(w).t()).view(len(tokens), -1, model.head_dim) for w in (model.wq, model.wk, model.wv))
    group = model.q_heads // model.kv_heads
    k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
    s = torch.einsum("thd,ihd->hti", q, k) * model.head_dim ** -0.5
    t, i = torch.arange(len(tokens), device=x.device)[:, None], torch.arange(len(tokens), device=x.device)[None]
    hide = i > t
    if window:
        hide |= (i <= t - window) & (i >= sinks)
    o = torch.einsum("hti,ihd->thd", torch.softmax(s.masked_fill(hide, -torch.inf), -1), v)
    return (x + o.reshape(len(tokens), -1) @ d(model.wo).t()) @ d(model.head).t()


@pytest.mark.parametrize("window,sinks,head_dim", [(0, 0, 64), (9, 2, 128)])
def test_greedy_tokens_are_the_targets(example, window, sinks, head_dim):
    r = example.generate(requests=5, new_tokens=40, temperature=0.0, window=window, sinks=sinks, head_dim=head_dim,
                         seed=3)
    model = example.ToyTarget(4096, 256, 8, 2, head_dim, 3)
    assert 0 < r.accepted < r.drafted and r.free_pages == r.total_pages
    for tokens in r.tokens:
        assert len(tokens) > 40
        tokens = tokens[:41]
        logits = dense_logits(model, torch.tensor(tokens, device="cuda"), window, sinks)
        # BF16 states and logits: four roundings of 2^-8 in what a logit sums,
        # five deviations over the tokens, and the logit's own (at most 2^-8 of 16)
        slack = 5 * 4 * 2.0 ** -8 * logits.std() + 2 * 2.0 ** -8 * 16
        for t in range(40):
            assert float(logits[t].max() - logits[t, tokens[t + 1]]) <= float(slack), t


def test_sampled_run_keeps_its_pages(example):
    r = example.generate(requests=7, new_tokens=33, temperature=0.9, drafts=3, page_size=8, seed=4)
    assert r.free_pages == r.total_pages and 0 < r.accepted < r.drafted
    assert all(0 <= t < 4096 for row in r.tokens for t in row)
