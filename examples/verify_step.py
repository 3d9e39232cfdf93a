"""Speculative decoding with the library's calls, on a toy target model.

Every step, for all requests at once:
  1. markov_chain_sample draws N draft tokens after each request's last one
     (its base logits come from a toy draft head here);
  2. markov_paged_layout gives the last token and its drafts room in the paged
     cache, markov_rotary turns queries and keys by their positions (optional),
     markov_paged_write stores keys and values, and markov_paged_attention lets
     the tokens attend to them (window and sinks too); with an e4m3 cache
     markov_paged_write_e4m3 and markov_paged_attention_e4m3 do;
  3. markov_verify accepts a prefix of the drafts against the target's logits
     and draws the token after it, and markov_logprobs reports the tokens' log
     probabilities and the most probable alternatives (optional).
What was not accepted is forgotten by not counting it in the context: its
pages are reused or go back to the ring with the next layout.  Requests that
reached their length release their pages and become padding rows.

    python examples/verify_step.py [--requests 6] [--tokens 40] [--temperature 0.7]
        [--cache e4m3] [--rotary] [--alternatives 3]
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass, field

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from draft_token_markov_gb300 import api  # noqa: E402


class ToyTarget:
    """Embedding, one attention layer with a residual, and an LM head; BF16."""

    def __init__(self, vocab, hidden, q_heads, kv_heads, head_dim, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def w(rows, cols, std):
            return (torch.randn((rows, cols), generator=g, device="cuda") * std).to(torch.bfloat16)

        self.embed = w(vocab, hidden, 1.0)
        self.wq, self.wk, self.wv = (w(h * head_dim, hidden, hidden ** -0.5)
                                     for h in (q_heads, kv_heads, kv_heads))
        self.wo = w(hidden, q_heads * head_dim, 0.5 * (q_heads * head_dim) ** -0.5)
        self.head = w(vocab, hidden, 4 * hidden ** -0.5)
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim

    def project(self, x):
        """Queries, keys and values [tokens, heads, head_dim] of hidden states."""
        return [(x @ w.t()).view(len(x), -1, self.head_dim) for w in (self.wq, self.wk, self.wv)]

    def logits(self, x, attended):
        return (x + attended.reshape(len(x), -1) @ self.wo.t()) @ self.head.t()


@dataclass
class Result:
    tokens: list = field(default_factory=list)      # of each request, its first token included
    logprobs: list = field(default_factory=list)    # of each request's tokens after the first, where asked for
    alternatives: list = field(default_factory=list)    # ids at each of those, the most probable first
    drafted: int = 0
    accepted: int = 0
    free_pages: int = 0
    total_pages: int = 0


def generate(requests=6, new_tokens=40, temperature=0.7, drafts=4, vocab=4096, hidden=256, q_heads=8,
             kv_heads=2, head_dim=64, page_size=16, window=0, sinks=0, seed=0, cache="bf16", rotary=False,
             alternatives=0) -> Result:
    R, N = requests, drafts
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed + 1)
    model = ToyTarget(vocab, hidden, q_heads, kv_heads, head_dim, seed)
    # a draft model that mostly agrees: the target's own head on the embedding
    markov_head = (torch.randn((vocab, 64), generator=g, device=dev) * 0.02).to(torch.bfloat16)
    markov_embed = (torch.randn((vocab, 64), generator=g, device=dev) * 0.02).to(torch.bfloat16)

    chain = api.Plan(vocab, 64, N, R)
    paged = api.PagedPlan(q_heads, kv_heads, head_dim, page_size, torch.bfloat16, max_rows=R)
    width = -(-(new_tokens + 2 * N + 4) // page_size)
    pages = R * width
    shape = (pages, page_size, kv_heads, head_dim)
    e4m3 = cache == "e4m3"
    k_cache, v_cache = (torch.zeros(shape, dtype=torch.float8_e4m3fn if e4m3 else torch.bfloat16, device=dev)
                        for _ in range(2))
    # a scale for each 16 tokens and key head
    scales = [torch.zeros((pages, page_size // 16, kv_heads), device=dev) for _ in range(2)] if e4m3 else []
    turn = api.RotaryPlan(head_dim) if rotary else None
    table = torch.full((R, width), -1, dtype=torch.int32, device=dev)
    held = torch.zeros(R, dtype=torch.int32, device=dev)
    ring = torch.arange(pages, dtype=torch.int32, device=dev)
    free = torch.tensor([0, pages], device=dev)

    context = torch.zeros(R, dtype=torch.int32, device=dev)      # tokens in the cache
    query = torch.full((R,), N + 1, dtype=torch.int32, device=dev)    # padding rows keep their place
    state = torch.arange(R, device=dev)                          # -1 once a request is done
    last = torch.randint(0, vocab, (R,), generator=g, device=dev)
    temp = torch.full((R,), float(temperature), device=dev)
    out = Result(tokens=[[int(t)] for t in last.tolist()], logprobs=[[] for _ in range(R)],
                 alternatives=[[] for _ in range(R)], total_pages=pages)

    step = 0
    while bool((state >= 0).any()):
        seeds = torch.full((R,), 1000 * seed + 2 * step, device=dev)
        base = (model.embed[last] @ model.head.t())[:, None].expand(R, N, vocab).contiguous()
        # padding rows are not written: what they hold has to be a token
        drafted = torch.zeros((R, N), dtype=torch.int64, device=dev)
        drafted, draft_logits = api.markov_chain_sample(
            chain, base, markov_head, markov_embed, last.int(), temp, seeds, state, api.GUMBEL,
            draft_tokens=drafted)
        chunk = torch.cat([last[:, None], drafted], 1).reshape(-1)

        start, lens, positions, slots = api.markov_paged_layout(paged, context, query, state, table, held, ring, free,
                                                                R * (N + 1))
        x = model.embed[chunk]
        q, k, v = model.project(x)
        if turn is not None:
            api.markov_rotary(turn, q, k, positions, q_out=q, k_out=k)
        attended = torch.zeros_like(q)               # padding rows stay zero
        write, attend = ((api.markov_paged_write_e4m3, api.markov_paged_attention_e4m3) if e4m3 else
                         (api.markov_paged_write, api.markov_paged_attention))
        write(paged, k, v, k_cache, v_cache, *scales, slots)
        attend(paged, q, k_cache, v_cache, *scales, table, state, start, lens, window=window, sinks=sinks,
               out=attended)
        target = model.logits(x, attended).view(R, N + 1, vocab)

        uniforms = torch.rand((R, N), generator=g, device=dev)
        # noise of seeds that the drafts were not drawn with
        noise = api.markov_gumbel_noise(seeds + 1, temp, state, 1, vocab)
        tokens, accepted = api.markov_verify(chain, target, drafted, draft_logits, temp, uniforms, noise, state)

        if alternatives:
            # ids of padding rows and past the accepted ones are -1: left alone
            given = torch.where(state[:, None] >= 0, tokens, -1).reshape(-1)
            said = api.markov_logprobs(target.view(-1, vocab), given, temp.repeat_interleave(N + 1), alternatives)
            logprobs = said.logprobs.view(R, N + 1).tolist()
            top_ids = said.top_ids.view(R, N + 1, alternatives).tolist()
        taken, counts, live = tokens.tolist(), accepted.tolist(), state.tolist()
        for b in range(R):
            if live[b] < 0:
                continue
            n = counts[b]
            out.tokens[b] += taken[b][:n + 1]
            if alternatives:
                out.logprobs[b] += logprobs[b][:n + 1]
                out.alternatives[b] += top_ids[b][:n + 1]
            out.drafted, out.accepted = out.drafted + N, out.accepted + n
            if len(out.tokens[b]) > new_tokens:
                context[b] = 0                       # its pages go back with the next layout
            else:
                context[b] += n + 1
                last[b] = taken[b][n]
        done = torch.tensor([len(t) > new_tokens for t in out.tokens], device=dev)
        if bool((done & (state >= 0)).any()):
            api.markov_paged_layout(paged, context, torch.zeros_like(query), state, table, held, ring, free, 0)
            state[done] = -1
        step += 1
    for status in (api.markov_plan_status(chain), api.markov_paged_plan_status(paged)):
        if status != 0:
            raise RuntimeError(f"device status {status}")
    out.free_pages = int(free[1])
    chain.close()
    paged.close()
    if turn is not None:
        turn.close()
    return out


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--requests", type=int, default=6)
    p.add_argument("--tokens", type=int, default=40)
    p.add_argument("--drafts", type=int, default=4)
    p.add_argument("--temperature", type=float, default=0.7)
    p.add_argument("--window", type=int, default=0)
    p.add_argument("--sinks", type=int, default=0)
    p.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    p.add_argument("--rotary", action="store_true")
    p.add_argument("--alternatives", type=int, default=0)
    a = p.parse_args()
    r = generate(a.requests, a.tokens, a.temperature, a.drafts, window=a.window, sinks=a.sinks, cache=a.cache,
                 rotary=a.rotary, alternatives=a.alternatives)
    print(f"{r.accepted} of {r.drafted} drafts accepted; {r.free_pages} of {r.total_pages} pages free at the end")
    for b, t in enumerate(r.tokens):
        print(b, t)
        if a.alternatives:
            print("  log probabilities", [round(x, 2) for x in r.logprobs[b]])


if __name__ == "__main__":
    main()
