"""The cases that the verify step's operators are timed on: room for new
tokens in a paged cache (layout), storing their keys and values (write),
attention of the new tokens over the cache (attend) and acceptance of draft
tokens against the target's logits (verify).

Where ``own`` is false ``run`` computes a case with elementary torch
operations in 32 bits; where it is true it calls the library."""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ----------------------------------------------------------------- the cases

def _attend(name, rows, q, ctx, hq, hkv, d=128, page=16, dtype="bf16", window=0, sinks=0,
            order="nhd", lens=1):
    return {"name": name, "op": "attend", "rows": rows, "q_lo": q[0], "q_hi": q[1],
            "ctx_lo": ctx[0], "ctx_hi": ctx[1], "hq": hq, "hkv": hkv, "d": d, "page": page,
            "dtype": dtype, "window": window, "sinks": sinks, "order": order, "lens": lens}


def _layout(name, rows, q, ctx, page, long_q=0, lens=1):
    return {"name": name, "op": "layout", "rows": rows, "q_lo": q[0], "q_hi": q[1],
            "ctx_lo": ctx[0], "ctx_hi": ctx[1], "page": page, "long_q": long_q, "lens": lens}


def _write(name, tokens, hkv, d, page, dtype="bf16", order="nhd"):
    return {"name": name, "op": "write", "tokens": tokens, "hkv": hkv, "d": d, "page": page,
            "dtype": dtype, "order": order}


def _verify(name, rows, steps, vocab, target="bf16", draft="bf16", padding=0):
    return {"name": name, "op": "verify", "rows": rows, "steps": steps, "vocab": vocab,
            "target": target, "draft": draft, "padding": padding}


def listed():
    return [
        # the draft step of a full chain call: 8 requests, 8 drafts and the token before them
        _layout("layout 8 rows x 9", 8, (9, 9), (100, 4000), 16),
        # a large mixed batch: 255 requests that draft beside one that prefills 8192 tokens
        _layout("layout 256 rows + prefill", 256, (1, 9), (1, 30000), 16, long_q=8192),
        # keys and values of that draft step
        _write("write 72 tokens", 72, 8, 128, 16),
        # keys and values of a prefill chunk, pages with the heads outermost
        _write("write 8192 tokens hnd", 8192, 8, 128, 64, order="hnd"),
        # one user, one token: latency
        _attend("decode 1 row", 1, (1, 1), (1000, 1000), 32, 8),
        # one token each of a full batch with ragged contexts: the cache's bytes count
        _attend("decode 64 rows ragged", 64, (1, 1), (500, 32000), 64, 8, page=64),
        # the target's check of 8 drafts for 8 requests
        _attend("verify chunk 8 rows x 9", 8, (9, 9), (1000, 16000), 64, 8),
        # a chunk of a long prompt
        _attend("prefill 4096 over 16384", 1, (4096, 4096), (12288, 12288), 32, 8, page=64),
        # prefill chunks and single tokens in one batch; 7 query heads to a key head
        _attend("mixed 16 rows, group 7", 16, (1, 500), (0, 8000), 28, 4, page=32, lens=3),
        # long contexts of which a window and the first tokens are kept in sight
        _attend("window 1000 + 4 sinks", 32, (9, 9), (2000, 100000), 64, 8, d=64, page=16,
                dtype="fp16", window=1000, sinks=4, order="hnd"),
        # acceptance for one request: latency
        _verify("accept 1 row x 8", 1, 8, 129280),
        # acceptance for the large batch, every eighth row padding
        _verify("accept 64 rows x 8", 64, 8, 129280, padding=8),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["layout", "write", "attend", "attend", "attend", "verify"])
    if op == "layout":
        hi = _log(rng, 16, 30000)
        c = _layout("", _log(rng, 1, 256), (1, rng.randint(1, 17)), (1, hi),
                    rng.choice([8, 16, 32, 64, 128]), long_q=rng.choice([0, _log(rng, 10, 8192)]),
                    lens=rng.randint(1, 10 ** 6))
    elif op == "write":
        c = _write("", _log(rng, 1, 8192), rng.randint(1, 8), rng.choice([64, 128]),
                   rng.choice([8, 16, 32, 64, 128]), rng.choice(["bf16", "fp16"]),
                   rng.choice(["nhd", "hnd"]))
    elif op == "attend":
        kind = rng.choice(["decode", "drafts", "chunks"])
        hkv, d = rng.randint(1, 8), rng.choice([64, 128])
        group = rng.randint(1, 8)
        window = rng.choice([0, 0, _log(rng, 16, 4000)])
        hi = _log(rng, 32, 32000)
        q = {"decode": (1, 1), "drafts": (2, rng.randint(2, 17)), "chunks": (1, _log(rng, 20, 2000))}[kind]
        rows = _log(rng, 1, {"decode": 64, "drafts": 32, "chunks": 4}[kind])
        c = _attend("", rows, q, (rng.choice([0, hi // 2]), hi), group * hkv, hkv, d,
                    rng.choice([8, 16, 32, 64, 128]), rng.choice(["bf16", "fp16"]), window,
                    rng.choice([0, 1, 4, 100]) if window else 0, rng.choice(["nhd", "hnd"]),
                    lens=rng.randint(1, 10 ** 6))
    else:
        c = _verify("", _log(rng, 1, 64), rng.randint(1, 12), 16 * _log(rng, 250, 8080),
                    rng.choice(["bf16", "fp32"]), rng.choice(["bf16", "fp32"]),
                    rng.choice([0, 3, 8]))
        # no more logits than the largest listed case reads
        c["rows"] = max(1, min(c["rows"], 64 * 17 // (2 * c["steps"] + 1) // 2))
    del c["name"]
    return c


def _lengths(case):
    """(new tokens, context before them) of each request: the case's own, whatever the seed."""
    r = np.random.RandomState(case["lens"])
    rows, lo, hi = case["rows"], case["ctx_lo"], case["ctx_hi"]
    q = r.randint(case["q_lo"], case["q_hi"] + 1, rows)
    if lo >= hi:
        c = np.full(rows, lo)
    else:
        a, b = math.log(lo + 1), math.log(hi + 1)
        c = np.clip(np.round(np.exp(r.uniform(a, b, rows)) - 1), lo, hi).astype(np.int64)
        c[r.randint(rows)] = hi                    # the longest is there
    if case.get("long_q"):
        q[r.randint(rows)] = case["long_q"]
    return q.astype(np.int64), c.astype(np.int64)


def _visible(case):
    """(query-key pairs, keys that some query of their request sees) over all requests."""
    pairs = keys = 0
    w, k = case["window"], case["sinks"]
    for n, c in zip(*_lengths(case)):
        p = np.arange(c, c + n)
        if w:
            first = np.maximum(0, p - w + 1)
            pairs += int((p + 1 - first + np.minimum(k, first)).sum())
            keys += int(c + n - first[0] + min(k, first[0]))
        else:
            pairs += int((p + 1).sum())
            keys += int(c + n)
    return pairs, keys


def work(case):
    op = case["op"]
    if op == "layout":
        q, c = _lengths(case)
        touched = int(sum(-(-int(a + b) // case["page"]) - int(b) // case["page"] for a, b in zip(q, c)))
        # lengths, states and held counts; the pages of new tokens in and out; positions and slots
        return {"bytes": 32 * case["rows"] + 8 * touched + 12 * int(q.sum()), "flops": 0}
    if op == "write":
        return {"bytes": case["tokens"] * (2 * 2 * case["hkv"] * case["d"] * 2 + 8), "flops": 0}
    if op == "attend":
        pairs, keys = _visible(case)
        q, c = _lengths(case)
        io = int(q.sum()) * case["hq"] * (2 * case["d"] * 2 + 4)
        return {"bytes": keys * case["hkv"] * case["d"] * 2 * 2 + io,
                "flops": 4 * case["d"] * case["hq"] * pairs}
    live = case["rows"] - (case["rows"] // case["padding"] if case["padding"] else 0)
    size = {"bf16": 2, "fp32": 4}
    n = case["steps"]
    # every logit once, and the noise of the token that each request draws itself
    return {"bytes": live * case["vocab"] * ((n + 1) * size[case["target"]] + n * size[case["draft"]] + 4),
            "flops": 0}


# ---------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 11)


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    x = torch.empty(shape, dtype=dtype, device="cuda")
    return x.normal_(0.0, std, generator=g)


def _cache(g, pages, case):
    """A paged cache [pages, page, heads, d], its storage in the case's order."""
    if case["order"] == "hnd":
        return _randn(g, pages, case["hkv"], case["page"], case["d"], dtype=DT[case["dtype"]]).transpose(1, 2)
    return _randn(g, pages, case["page"], case["hkv"], case["d"], dtype=DT[case["dtype"]])


def _int(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x)).to(device="cuda", dtype=dtype)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "layout":
        return _prepare_layout(case, seed, g)
    if op == "write":
        return _prepare_write(case, seed, g)
    if op == "attend":
        return _prepare_attend(case, seed, g)
    return _prepare_verify(case, seed, g)


def _prepare_layout(case, seed, g):
    q, c = _lengths(case)
    rows, ps = case["rows"], case["page"]
    r = np.random.RandomState(seed % (1 << 31))
    # pages held from the step before, whose drafts were not all accepted
    held = -(-(c + r.randint(0, 2 * case["q_hi"] + 1, rows)) // ps)
    most = -(-(c + q + 2 * case["q_hi"]) // ps)
    states, width, total = rows + 5, int(most.max()) + 3, int(2 * most.sum()) + 64
    perm = r.permutation(total)
    idx = r.permutation(states)[:rows]
    table = np.full((states, width), -1)
    at = 0
    for b in range(rows):
        table[idx[b], :held[b]] = perm[at:at + held[b]]
        at += held[b]
    head, count = int(r.randint(total)), total - at
    ring = np.full(total, -1)
    ring[(head + np.arange(count)) % total] = perm[at:]
    held_s = np.zeros(states)
    held_s[idx] = held
    T = int(q.sum()) + 3                           # room beyond the tokens, as a captured graph has
    st = {"op": "layout", "page": ps, "T": T, "context": _int(c), "query": _int(q),
          "idx": _int(idx, torch.int64), "table": _int(table), "held": _int(held_s),
          "held_out": _int(held_s), "ring": _int(ring), "free": _int([head, count], torch.int64),
          "free_out": _int([0, 0], torch.int64),
          "query_start": _int(np.zeros(rows + 1)), "seq_lens": _int(np.zeros(rows)),
          "positions": _int(np.zeros(T)), "slots": _int(np.zeros(T), torch.int64)}
    if own:
        from draft_token_markov_gb300 import api
        st["api"] = api
        st["plan"] = api.PagedPlan(8, 8, 64, ps, torch.bfloat16, max_rows=rows)
    return st


def _prepare_write(case, seed, g):
    T, ps = case["tokens"], case["page"]
    pages = -(-T // ps) + 7
    r = np.random.RandomState(seed % (1 << 31))
    # tokens of requests of about 100 tokens, each on pages of its own order
    page = r.permutation(pages)
    slots = page[np.arange(T) // ps] * ps + np.arange(T) % ps
    st = {"op": "write", "k_cache": _cache(g, pages, case), "v_cache": _cache(g, pages, case),
          "key": _randn(g, T, case["hkv"], case["d"], dtype=DT[case["dtype"]]),
          "value": _randn(g, T, case["hkv"], case["d"], dtype=DT[case["dtype"]]),
          "slots": _int(slots, torch.int64)}
    if own:
        from draft_token_markov_gb300 import api
        st["api"] = api
        st["plan"] = api.PagedPlan(case["hkv"], case["hkv"], case["d"], ps, DT[case["dtype"]], max_rows=1)
    return st


def _prepare_attend(case, seed, g):
    q, c = _lengths(case)
    rows, ps = case["rows"], case["page"]
    r = np.random.RandomState(seed % (1 << 31))
    need = -(-(c + q) // ps)
    pages = int(need.sum()) + 3
    perm, idx = r.permutation(pages), r.permutation(rows + 2)[:rows]
    table = np.full((rows + 2, int(need.max()) + 1), -1)
    at = 0
    for b in range(rows):
        table[idx[b], :need[b]] = perm[at:at + need[b]]
        at += need[b]
    start = np.concatenate([[0], np.cumsum(q)])
    T, dt = int(start[-1]), DT[case["dtype"]]
    st = {"op": "attend", "q_hi": int(q.max()), "len_hi": int((c + q).max()),
          "k_cache": _cache(g, pages, case), "v_cache": _cache(g, pages, case),
          # scores spread with a deviation of two, as trained heads' do
          "q": _randn(g, T, case["hq"], case["d"], dtype=dt, std=2.0),
          "scale": case["d"] ** -0.5, "window": case["window"], "sinks": case["sinks"],
          "table": _int(table), "idx": _int(idx, torch.int64), "query_start": _int(start),
          "seq_lens": _int(c + q), "out": torch.zeros((T, case["hq"], case["d"]), dtype=dt, device="cuda"),
          "lse": torch.zeros((T, case["hq"]), device="cuda")}
    if own:
        from draft_token_markov_gb300 import api
        st["api"] = api
        st["plan"] = api.PagedPlan(case["hq"], case["hkv"], case["d"], ps, dt, max_rows=rows)
    return st


def _prepare_verify(case, seed, g):
    R, N, V = case["rows"], case["steps"], case["vocab"]
    draft = _randn(g, R, N, V, std=3.0)
    # the target agrees with the draft model for the most part
    target = torch.cat([draft, _randn(g, R, 1, V, std=3.0)], 1)
    target += _randn(g, R, N + 1, V, std=0.7)
    draft, target = draft.to(DT[case["draft"]]), target.to(DT[case["target"]])
    temperature = torch.tensor([0.0, 0.6, 1.0], device="cuda")[torch.randint(0, 3, (R,), generator=g, device="cuda")]
    temperature[0] = 0.8
    # the drafts, drawn from the draft logits
    e = torch.empty((R, N, V), device="cuda").exponential_(generator=g).clamp_(min=1e-30)
    t = torch.where(temperature > 0, temperature, 1.0)[:, None, None]
    key = draft.float() / t - torch.where(temperature > 0, 1.0, 0.0)[:, None, None] * e.log_()
    tokens = key.argmax(-1)
    del e, key
    u = torch.empty((R, V), device="cuda").uniform_(generator=g).clamp_(1e-12, 1 - 6e-8)
    noise = -torch.log(-torch.log(u))
    del u
    idx = torch.arange(R, device="cuda")
    if case["padding"]:
        idx[case["padding"] - 1::case["padding"]] = -1
    st = {"op": "verify", "target": target, "draft": draft, "tokens": tokens, "temperature": temperature,
          "uniforms": torch.empty((R, N), device="cuda").uniform_(generator=g), "noise": noise, "idx": idx,
          "out_tokens": torch.full((R, N + 1), -7, dtype=torch.int64, device="cuda"),
          "accepted": torch.full((R,), -7, dtype=torch.int32, device="cuda"),
          "p": torch.zeros((R, N), device="cuda"), "q": torch.zeros((R, N), device="cuda")}
    if own:
        from draft_token_markov_gb300 import api
        st["api"] = api
        st["plan"] = api.Plan(V, 64, N, R)
    return st


# ---------------------------------------------------------------- the passes

def run(state):
    op = state["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_layout(s):
    s["api"].markov_paged_layout(s["plan"], s["context"], s["query"], s["idx"], s["table"], s["held"],
                                 s["ring"], s["free"], s["T"], query_start=s["query_start"],
                                 seq_lens=s["seq_lens"], positions=s["positions"], slots=s["slots"],
                                 pages_held_out=s["held_out"], free_state_out=s["free_out"])
    return {k: s[k] for k in ("query_start", "seq_lens", "positions", "slots", "table", "held_out",
                              "ring", "free_out")}


def _plain_layout(s):
    ps, T, idx = s["page"], s["T"], s["idx"]
    table, ring, C = s["table"], s["ring"], s["ring"].numel()
    c, q, held = s["context"], s["query"], s["held"][idx]
    need = (c + q + ps - 1) // ps
    grow, shrink = (need - held).clamp(min=0), (held - need).clamp(min=0)
    grown, shrunk = torch.cumsum(grow, 0), torch.cumsum(shrink, 0)
    head, count = s["free"][0], s["free"][1]
    start = torch.cat([torch.zeros_like(q[:1]), torch.cumsum(q, 0, dtype=torch.int32)])
    rows = table[idx]
    k = torch.arange(rows.shape[1], device="cuda")[None, :]
    take = (head + (grown - grow)[:, None] + k - held[:, None]) % C
    give = (head + count + (shrunk - shrink)[:, None] + k - need[:, None]) % C
    new = torch.where((k >= held[:, None]) & (k < need[:, None]), ring[take], rows)
    back = (k >= need[:, None]) & (k < held[:, None])
    pad = torch.cat([ring, ring[:1]])
    pad.scatter_(0, torch.where(back, give, C).reshape(-1), rows.reshape(-1))
    ring.copy_(pad[:C])
    table[idx] = new
    held_out = s["held"].clone()
    held_out[idx] = need
    free_out = torch.stack([(head + grown[-1]) % C, count - grown[-1] + shrunk[-1]])
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(start[1:], t, right=True).clamp(max=idx.numel() - 1)
    inside = t < start[-1]
    pos = torch.where(inside, c[b] + t - start[b], 0)
    slots = torch.where(inside, new[b, pos // ps].to(torch.int64) * ps + pos % ps, -1)
    return {"query_start": start, "seq_lens": c + q, "positions": pos, "slots": slots, "table": table,
            "held_out": held_out, "ring": ring, "free_out": free_out}


def _own_write(s):
    s["api"].markov_paged_write(s["plan"], s["key"], s["value"], s["k_cache"], s["v_cache"], s["slots"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_write(s):
    ps = s["k_cache"].shape[1]
    page, at = s["slots"] // ps, s["slots"] % ps
    s["k_cache"][page, at] = s["key"]
    s["v_cache"][page, at] = s["value"]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attend(s):
    s["api"].markov_paged_attention(s["plan"], s["q"], s["k_cache"], s["v_cache"], s["table"], s["idx"],
                                    s["query_start"], s["seq_lens"], scale=s["scale"], window=s["window"],
                                    sinks=s["sinks"], out=s["out"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_attend(s):
    q, kc, vc = s["q"], s["k_cache"], s["v_cache"]
    T, hq, d = q.shape
    ps, hkv = kc.shape[1], kc.shape[2]
    R, M, L = s["idx"].numel(), s["q_hi"], s["len_hi"]
    # every request padded to the longest: [R, hkv, M * group, L] scores
    i = torch.arange(L, device="cuda")
    page = s["table"][s["idx"]][:, i // ps].clamp(min=0)
    k = kc[page, i % ps].float().permute(0, 2, 3, 1)
    start, n = s["query_start"][:-1, None], (s["query_start"][1:] - s["query_start"][:-1])[:, None]
    j = torch.arange(M, device="cuda")[None, :]
    tok = (start + torch.minimum(j, n - 1)).clamp(0, T - 1)
    x = q[tok].float().reshape(R, M, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(R, hkv, -1, d)
    p = (x @ k).mul_(s["scale"]).view(R, hkv, M, hq // hkv, L)
    del k
    pos = (s["seq_lens"][:, None] - n + j)[:, :, None]
    seen = (i <= pos) & (i < s["seq_lens"][:, None, None])
    if s["window"]:
        seen &= (i > pos - s["window"]) | (i < s["sinks"])
    p.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = p.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    v = vc[page, i % ps].float().permute(0, 2, 1, 3)
    o = (p.view(R, hkv, -1, L) @ v).view(R, hkv, M, hq // hkv, d) / torch.where(z > 0, z, 1.0)
    lse = (m + torch.log(z)).squeeze(-1)
    # back to one row per token
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["query_start"][1:].contiguous(), t, right=True)
    at = t - s["query_start"][b]
    out = o.permute(0, 2, 1, 3, 4)[b, at].reshape(T, hq, d).to(q.dtype)
    return {"out": out, "lse": lse.permute(0, 2, 1, 3)[b, at].reshape(T, hq)}


def _own_verify(s):
    s["api"].markov_verify(s["plan"], s["target"], s["tokens"], s["draft"], s["temperature"], s["uniforms"],
                           s["noise"], s["idx"], tokens=s["out_tokens"], num_accepted=s["accepted"],
                           target_probs=s["p"], draft_probs=s["q"])
    return {k: s[k] for k in ("out_tokens", "accepted", "p", "q")}


def _first_max(x):
    at = torch.arange(x.shape[-1], device=x.device)
    return torch.where(x == x.amax(-1, keepdim=True), at, x.shape[-1]).amin(-1)


def _softmax(logits, temperature):
    samples = (temperature > 0)[:, None, None]
    x = logits.float() / torch.where(samples, temperature[:, None, None], 1.0)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    one = torch.arange(x.shape[-1], device=x.device) == _first_max(x)[..., None]
    return torch.where(samples, e / e.sum(-1, keepdim=True), one.float())


def _plain_verify(s):
    R, N = s["tokens"].shape
    p, q = _softmax(s["target"], s["temperature"]), _softmax(s["draft"], s["temperature"])
    px = p[:, :N].gather(-1, s["tokens"][..., None])[..., 0]
    qx = q.gather(-1, s["tokens"][..., None])[..., 0]
    n = torch.cumprod((s["uniforms"] * qx < px).to(torch.int32), 1).sum(1)
    r = torch.arange(R, device="cuda")
    last = p[r, n]
    rest = torch.where((n < N)[:, None], last - q[r, n.clamp(max=N - 1)], last).clamp(min=0)
    rest = torch.where(rest.amax(-1, keepdim=True) > 0, rest, last)
    key = torch.log(rest) + torch.where((s["temperature"] > 0)[:, None], s["noise"], 0.0)
    own_token = _first_max(key)
    j = torch.arange(N + 1, device="cuda")[None, :]
    drafts = torch.cat([s["tokens"], s["tokens"][:, :1]], 1)
    tokens = torch.where(j < n[:, None], drafts, torch.where(j == n[:, None], own_token[:, None], -1))
    live = s["idx"] >= 0
    return {"out_tokens": torch.where(live[:, None], tokens, s["out_tokens"]),
            "accepted": torch.where(live, n.to(torch.int32), s["accepted"]),
            "p": torch.where(live[:, None], px, s["p"]), "q": torch.where(live[:, None], qx, s["q"])}


_OWN = {"layout": _own_layout, "write": _own_write, "attend": _own_attend, "verify": _own_verify}
_PLAIN = {"layout": _plain_layout, "write": _plain_write, "attend": _plain_attend, "verify": _plain_verify}


# -------------------------------------------------------------- in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "attend":
        return _exact_attend(case, s)
    if case["op"] == "verify":
        return _exact_verify(case, s)
    if case["op"] == "write":
        return _exact_write(case, s)
    return None                                    # whole numbers only


def _exact_write(case, s):
    out = {}
    for cache, new in (("k_cache", "key"), ("v_cache", "value")):
        x = s[cache].double().contiguous()
        x.view(-1, case["hkv"], case["d"]).index_copy_(0, s["slots"], s[new].double())
        out[cache] = x
    return out


def _exact_attend(case, s):
    hq, hkv, d, ps = case["hq"], case["hkv"], case["d"], case["page"]
    group = hq // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    first = 0
    for b, (n, c) in enumerate(zip(*_lengths(case))):
        n, c = int(n), int(c)
        L = c + n
        pages = s["table"][s["idx"][b], :-(-L // ps)].long()
        pos = torch.arange(c, L, device="cuda")[:, None]
        key = torch.arange(L, device="cuda")[None, :]
        hide = key > pos
        if case["window"]:
            hide |= (key <= pos - case["window"]) & (key >= case["sinks"])
        for h in range(hkv):
            k = s["k_cache"][pages, :, h].reshape(-1, d)[:L].double()
            v = s["v_cache"][pages, :, h].reshape(-1, d)[:L].double()
            for a in range(h * group, (h + 1) * group):
                x = s["q"][first:first + n, a].double() @ k.T * s["scale"]
                x[hide] = -math.inf
                lse[first:first + n, a] = torch.logsumexp(x, -1)
                out[first:first + n, a] = torch.softmax(x, -1) @ v
        first += n
    return {"out": out, "lse": lse}


def _exact_verify(case, s):
    R, N = case["rows"], case["steps"]
    p = torch.zeros((R, N), dtype=torch.float64, device="cuda")
    q = torch.zeros_like(p)
    for b in range(R):
        t = float(s["temperature"][b])
        if int(s["idx"][b]) < 0:
            continue
        for logits, into in ((s["target"][b, :N], p), (s["draft"][b], q)):
            x = logits.double()
            at = s["tokens"][b][:, None]
            if t > 0:
                into[b] = torch.log_softmax(x / t, -1).gather(1, at)[:, 0].exp()
            else:
                into[b] = (x.argmax(-1) == s["tokens"][b]).double()
    return {"out_tokens": None, "accepted": None, "p": p, "q": q}
