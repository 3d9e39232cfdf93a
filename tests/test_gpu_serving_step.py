"""A step of a serving loop with rotary positions, an e4m3 cache and log
probabilities, its calls together: each against its plain 64-bit form on what the
calls before it left, the whole captured in a graph, and the example."""
import importlib.util
import math
import os
import sys

import pytest
import torch

from tests import serving_ref as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E4M3 = torch.float8_e4m3fn


class Loop:
    """Requests of a serving loop, their state on the GPU."""

    def __init__(self, api, R=5, N=4, hq=8, hkv=2, d=64, page=32, block=16, V=4000, seed=0):
        self.api, self.R, self.N, self.hq, self.hkv, self.d, self.page, self.V = api, R, N, hq, hkv, d, page, V
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.T = R * (N + 1)
        self.paged = api.PagedPlan(hq, hkv, d, page, max_rows=R)
        self.verify = api.Plan(V, 64, N, R)
        self.rotary = api.RotaryPlan(d, d // 2, scaling="parts", factor=4.0, original_len=4096)
        width = 8
        pages = R * width
        self.cache = [torch.zeros((pages, page, hkv, d), dtype=E4M3, device="cuda") for _ in range(2)]
        self.scales = [torch.zeros((pages, page // block, hkv), device="cuda") for _ in range(2)]
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table, self.held = torch.full((R, width), -1, **i32), torch.zeros(R, **i32)
        self.ring, self.free = torch.arange(pages, **i32), torch.tensor([0, pages], device="cuda")
        self.context, self.query = torch.zeros(R, **i32), torch.full((R,), N + 1, **i32)
        self.state = torch.arange(R, device="cuda")
        self.state[2] = -1                                    # a padding row
        rand = lambda *s: torch.randn(s, generator=self.g, device="cuda")  # noqa: E731
        self.qkv = [rand(self.T, hq + 2 * hkv, d).bfloat16()]
        self.draft = rand(R, N, self.V).bfloat16() * 3
        self.drafted = torch.randint(0, self.V, (R, N), generator=self.g, device="cuda")
        self.temp = torch.tensor([0.0, 0.7, 1.0, 1.3, 0.9], device="cuda")[:R]
        self.uniforms = torch.rand((R, N), generator=self.g, device="cuda")
        self.noise = -torch.log(-torch.log(torch.rand((R, self.V), generator=self.g, device="cuda").clamp(1e-9, 1 - 1e-7)))
        self.target = (torch.cat([self.draft, rand(R, 1, self.V).bfloat16() * 3], 1) + rand(R, N + 1, self.V)).bfloat16()

    def step(self, stream=None):
        api, R, N, hq, hkv = self.api, self.R, self.N, self.hq, self.hkv
        qkv = self.qkv[0].clone()
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        start, lens, positions, slots = api.markov_paged_layout(self.paged, self.context, self.query, self.state, self.table,
                                                                self.held, self.ring, self.free, self.T)
        api.markov_rotary(self.rotary, q, k, positions, q_out=q, k_out=k)
        api.markov_paged_write_e4m3(self.paged, k, v, *self.cache, *self.scales, slots)
        out = torch.zeros((self.T, hq, self.d), dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros((self.T, hq), device="cuda")
        api.markov_paged_attention_e4m3(self.paged, q, *self.cache, *self.scales, self.table, self.state, start, lens,
                                        out=out, lse=lse)
        tokens = torch.full((R, N + 1), -1, device="cuda")
        accepted = torch.zeros(R, dtype=torch.int32, device="cuda")
        api.markov_verify(self.verify, self.target, self.drafted, self.draft, self.temp, self.uniforms, self.noise, self.state,
                          tokens=tokens, num_accepted=accepted)
        said = api.markov_logprobs(self.target.view(-1, self.V), tokens.view(-1), self.temp.repeat_interleave(N + 1), 4)
        return dict(q=q, k=k, v=v, start=start, lens=lens, positions=positions, slots=slots, out=out, lse=lse, tokens=tokens,
                    accepted=accepted, said=said)

    def close(self):
        assert self.api.markov_paged_plan_status(self.paged) == 0 and self.api.markov_plan_status(self.verify) == 0
        for p in (self.paged, self.verify, self.rotary):
            p.close()


def test_each_call_on_what_the_others_left(gpu_lib):
    loop = Loop(gpu_lib)
    f = ref.frequencies(32, scaling="parts", factor=4.0, length=4096)
    amplitude = 0.1 * math.log(4.0) + 1
    for step in range(4):
        cache = [c.cpu() for c in loop.cache]
        scales = [s.cpu() for s in loop.scales]
        before = loop.qkv[0].cpu()
        r = {k: v.cpu() if isinstance(v, torch.Tensor) else v for k, v in loop.step().items()}
        live = (r["slots"] >= 0)
        assert int(live.sum()) == 4 * (loop.N + 1)
        # turned by the positions that the layout gave
        for name, x in (("q", before[:, :8]), ("k", before[:, 8:10])):
            want, tol = ref.rotary(x, r["positions"], f, False, amplitude)
            assert float(((r[name].double() - want).abs() - tol).max()) <= 0
        # stored at its slots
        for new, c0, s0, c1, s1 in ((r["k"], cache[0], scales[0], loop.cache[0], loop.scales[0]),
                                    (r["v"], cache[1], scales[1], loop.cache[1], loop.scales[1])):
            want, want_s = ref.store(new, c0, s0, r["slots"], False)
            assert torch.equal(c1.cpu().double(), want) and torch.equal(s1.cpu().double(), want_s)
        # attended to
        want, wl, tol, tl = ref.attention(r["q"], loop.cache[0].cpu(), loop.cache[1].cpu(), loop.scales[0].cpu(),
                                          loop.scales[1].cpu(), loop.table.cpu(), loop.state.cpu(), r["start"], r["lens"],
                                          loop.d ** -0.5, 0, 0)
        seen = ~wl.isnan()
        assert float(((r["out"].double() - want).abs() - tol)[seen].max()) <= 0
        assert float(((r["lse"].double() - wl).abs() - tl)[seen].max()) <= 0
        assert bool((r["out"][~seen] == 0).all())
        # reported
        said = r["said"]
        for i, (t, T) in enumerate(zip(r["tokens"].view(-1).tolist(), loop.temp.repeat_interleave(loop.N + 1).tolist())):
            if t < 0:
                continue
            l = loop.target.view(-1, loop.V)[i].double().cpu().numpy()
            p, rank, entropy, ids, top = ref.logprobs(l, t, T, 4)
            assert abs(float(said.logprobs[i]) - p) <= 1e-6 * (1 + abs(p)) and int(said.ranks[i]) == rank
            assert said.top_ids[i].tolist() == ids.tolist()
            assert abs(float(said.entropy[i]) - entropy) <= 4e-6 * (1 + entropy)
        assert bool((r["tokens"][2] == -1).all())             # the padding row
        # greedy rows give their argmax
        n = int(r["accepted"][0])
        assert int(said.ranks.view(loop.R, -1)[0, n]) == 0
        # what was not accepted is written over by the next step
        loop.context += loop.state.ge(0).int() * (r["accepted"].cuda() + 1).int()
        loop.qkv[0] = (torch.randn(loop.qkv[0].shape, generator=loop.g, device="cuda") * 2.0 ** (step - 1)).bfloat16()
    loop.close()


def test_the_step_in_a_graph(gpu_lib):
    """Captured once, replayed with other lengths and queries: what an eager step gives."""
    eager, loop = Loop(gpu_lib, seed=3), Loop(gpu_lib, seed=3)
    first = eager.step()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured = loop.step()
    graph.replay()
    for again in range(3):
        torch.cuda.synchronize()
        for name in ("positions", "slots", "k", "out", "lse", "tokens", "accepted"):
            assert torch.equal(captured[name], first[name]), (again, name)
        for a, b in zip(captured["said"], first["said"]):
            # of tokens that were given: others are not written
            given = first["tokens"].view(-1) >= 0
            assert torch.equal(a[given], b[given])
        for a, b in zip(loop.cache + loop.scales, eager.cache + eager.scales):
            assert torch.equal(a.float(), b.float())
        for x in (eager, loop):
            x.context += x.state.ge(0).int() * (first["accepted"] + 1).int()
            x.qkv[0].mul_(1.5)
        first = eager.step()
        graph.replay()
    eager.close()
    loop.close()


@pytest.fixture(scope="module")
def example(gpu_lib):
    spec = importlib.util.spec_from_file_location("verify_step_serving", os.path.join(ROOT, "examples", "verify_step.py"))
    m = sys.modules[spec.name] = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("temperature", [0.0, 0.9])
def test_the_example_with_all_of_it(example, temperature):
    r = example.generate(requests=5, new_tokens=30, temperature=temperature, seed=5, cache="e4m3", rotary=True, alternatives=3)
    assert r.free_pages == r.total_pages and 0 < r.accepted <= r.drafted
    for tokens, logprobs, ids in zip(r.tokens, r.logprobs, r.alternatives):
        assert len(tokens) > 30 and len(logprobs) == len(tokens) - 1 == len(ids)
        assert all(x <= 0 and math.isfinite(x) for x in logprobs)
        if temperature == 0:
            assert [x[0] for x in ids] == tokens[1:]          # the argmax


def test_the_example_is_what_it_was(example):
    """Without the new options it draws the tokens that it drew."""
    a = example.generate(requests=3, new_tokens=20, temperature=0.0, seed=6)
    b = example.generate(requests=3, new_tokens=20, temperature=0.0, seed=6, alternatives=2)
    assert a.tokens == b.tokens and a.logprobs == [[], [], []]


def test_a_cache_beyond_32_bits(gpu_lib):
    """Pages whose bytes lie past 2^32: stored, read back and attended to."""
    api = gpu_lib
    page, hkv, d, pages = 64, 8, 128, 66000                   # 4.3 GB a side
    plan = api.PagedPlan(8, hkv, d, page, max_rows=1)
    big = dict(k=torch.zeros((pages, page, hkv, d), dtype=E4M3, device="cuda"),
               v=torch.zeros((pages, page, hkv, d), dtype=E4M3, device="cuda"))
    scales = [torch.ones((pages, 1, hkv), device="cuda") for _ in range(2)]
    g = torch.Generator(device="cuda").manual_seed(1)
    x, y = (torch.randn((100, hkv, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    pos = torch.arange(100, device="cuda")
    slots = table[0, pos // page].long() * page + pos % page
    idx, start, lens = (torch.tensor(v, dtype=t, device="cuda") for v, t in (([0], torch.int64), ([0, 100], torch.int32), ([100], torch.int32)))
    api.markov_paged_write_e4m3(plan, x, y, big["k"], big["v"], *scales, slots)
    k, v = api.markov_paged_read_e4m3(plan, big["k"], big["v"], *scales, table, idx, start, lens, 100)
    assert float((k.float() - x.float()).abs().max()) <= 2.0 ** -4 * float(x.abs().max())
    small = [c[-2:].flip(0).contiguous() if c.dtype != E4M3 else c[-2:].view(torch.uint8).flip(0).contiguous().view(E4M3)
             for c in (big["k"], big["v"], *scales)]
    near = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    for n in (1, 30):
        q = torch.randn((n, 8, d), generator=g, device="cuda").bfloat16()
        at = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        a, _ = api.markov_paged_attention_e4m3(plan, q, big["k"], big["v"], *scales, table, idx, at, lens)
        b, _ = api.markov_paged_attention_e4m3(plan, q, *small, near, idx, at, lens)
        assert torch.equal(a, b) and float(a.abs().max()) > 0
    assert api.markov_paged_plan_status(plan) == 0
    plan.close()
    assert float((v.float() - y.float()).abs().max()) <= 2.0 ** -4 * float(y.abs().max())
