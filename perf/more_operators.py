"""The cases that the operators around the verify step are timed on: rotary
positions of queries and keys (rotary), the store of keys and values in a paged
cache of 8 bits with a scale for each block of tokens and head (store), reading
such a cache back (fetch), attention over it (attend), and log probabilities of
given tokens with entropy and top alternatives (logprobs).

Where ``own`` is false ``run`` computes a case with elementary torch
operations in 32 bits (64 for the angles of far positions); where it is true it
calls the library."""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3 = torch.float8_e4m3fn


# ----------------------------------------------------------------- the cases

def _rotary(name, tokens, hq, hk, d, rot, dtype="bf16", interleaved=False, scaling="none", far=4000):
    return {"name": name, "op": "rotary", "tokens": tokens, "hq": hq, "hk": hk, "d": d, "rot": rot,
            "dtype": dtype, "interleaved": interleaved, "scaling": scaling, "far": far}


def _store(name, rows, per, hkv, d, page, block, dtype="bf16", order="nhd"):
    return {"name": name, "op": "store", "rows": rows, "per": per, "hkv": hkv, "d": d, "page": page,
            "block": block, "dtype": dtype, "order": order}


def _paged(name, op, rows, q, ctx, hq, hkv, d=128, page=16, block=16, dtype="bf16", window=0, sinks=0,
           order="nhd", lens=1):
    return {"name": name, "op": op, "rows": rows, "q_lo": q[0], "q_hi": q[1], "ctx_lo": ctx[0],
            "ctx_hi": ctx[1], "hq": hq, "hkv": hkv, "d": d, "page": page, "block": block, "dtype": dtype,
            "window": window, "sinks": sinks, "order": order, "lens": lens}


def _logprobs(name, rows, vocab, top, dtype="bf16", padding=0, masked=0.0):
    return {"name": name, "op": "logprobs", "rows": rows, "vocab": vocab, "top": top, "dtype": dtype,
            "padding": padding, "masked": masked}


def listed():
    return [
        # the target's check of 8 drafts for 8 requests: latency
        _rotary("rotary 8 x 9 tokens", 72, 64, 8, 128, 128),
        # an odd chunk of a long prompt, half of every head turned, far positions
        _rotary("rotary 8191 tokens, part", 8191, 32, 8, 128, 64, "fp16", True, "parts", 10 ** 6),
        # keys and values of the draft step, in the middle of their blocks
        _store("store 8 x 9 tokens", 8, 9, 8, 128, 16, 16),
        # keys and values of a prefill chunk, pages with the heads outermost
        _store("store 8192 tokens hnd", 1, 8192, 8, 128, 64, 64, order="hnd"),
        # one short request handed to a draft model without a cache of its own kind
        _paged("fetch 1 x 500", "fetch", 1, (500, 500), (0, 0), 32, 8),
        # requests moved out of the cache, ragged
        _paged("fetch 16 rows", "fetch", 16, (100, 8000), (0, 0), 64, 8, page=64, block=32, lens=2),
        # one user, one token: latency
        _paged("decode 1 row", "attend", 1, (1, 1), (1000, 1000), 32, 8),
        # one token each of a full batch with ragged contexts: the cache's bytes count
        _paged("decode 64 rows ragged", "attend", 64, (1, 1), (500, 32000), 64, 8, page=64, block=64),
        # the target's check of 8 drafts for 8 requests
        _paged("verify chunk 8 rows x 9", "attend", 8, (9, 9), (1000, 16000), 64, 8),
        # a chunk of a long prompt
        _paged("prefill 4096 over 16384", "attend", 1, (4096, 4096), (12288, 12288), 32, 8, page=64, block=32),
        # the tokens of one request's step, with eight alternatives each: latency
        _logprobs("logprobs 9, top 8", 9, 129280, 8),
        # a large batch's step, every eighth position past the accepted tokens
        _logprobs("logprobs 576, top 20", 576, 129280, 20, padding=8),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rotary", "rotary", "store", "store", "fetch", "attend", "attend", "attend", "attend",
                     "logprobs", "logprobs"])
    page = rng.choice([16, 32, 64, 128])
    block = rng.choice([b for b in (16, 32, 64, 128) if b <= page])
    dtype, order, d = rng.choice(["bf16", "fp16"]), rng.choice(["nhd", "hnd"]), rng.choice([64, 128])
    if op == "rotary":
        hk = rng.randint(1, 8)
        c = _rotary("", _log(rng, 1, 8192), hk * rng.randint(1, 6), hk, d, rng.choice([d, d // 2, d // 4]),
                    rng.choice(["bf16", "fp16", "fp32"]), rng.random() < 0.5,
                    rng.choice(["none", "linear", "base", "parts", "wavelength"]), _log(rng, 100, 10 ** 7))
    elif op == "store":
        rows = _log(rng, 1, 64)
        c = _store("", rows, _log(rng, 1, max(1, 8192 // rows)), rng.randint(1, 8), d, page, block, dtype, order)
    elif op == "fetch":
        c = _paged("", op, _log(rng, 1, 16), (1, _log(rng, 2, 8000)), (0, 0), 8, rng.randint(1, 8), d, page, block,
                   dtype, order=order, lens=rng.randint(1, 10 ** 6))
        c["hq"] = c["hkv"]
    elif op == "attend":
        kind = rng.choice(["decode", "drafts", "chunks"])
        hkv, group = rng.randint(1, 8), rng.randint(1, 8)
        window = rng.choice([0, 0, _log(rng, 16, 4000)])
        hi = _log(rng, 32, 32000)
        q = {"decode": (1, 1), "drafts": (2, rng.randint(2, 17)), "chunks": (1, _log(rng, 20, 2000))}[kind]
        rows = _log(rng, 1, {"decode": 64, "drafts": 32, "chunks": 4}[kind])
        c = _paged("", op, rows, q, (rng.choice([0, hi // 2]), hi), group * hkv, hkv, d, page, block, dtype, window,
                   rng.choice([0, 1, 4, 100]) if window else 0, order, rng.randint(1, 10 ** 6))
    else:
        c = _logprobs("", _log(rng, 1, 576), 16 * _log(rng, 250, 8080) + rng.choice([0, 0, 1, 7]),
                      rng.choice([0, 1, 5, 20, 32]), rng.choice(["bf16", "fp32"]), rng.choice([0, 3, 8]),
                      rng.choice([0.0, 0.0, 0.9]))
    # no more work than the largest listed case of its kind
    most = [work(x) for x in listed() if x["op"] == op]
    size = "tokens" if op == "rotary" else "rows"
    while any(work(c)[k] > max(w[k] for w in most) for k in ("bytes", "flops")):
        c[size] = 3 * c[size] // 4
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


SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def work(case):
    op = case["op"]
    if op == "rotary":
        x = case["tokens"] * (case["hq"] + case["hk"])
        return {"bytes": x * case["d"] * 2 * SIZE[case["dtype"]] + 4 * case["tokens"], "flops": x * case["rot"] * 3}
    if op == "store":
        T = case["rows"] * case["per"]
        return {"bytes": T * (2 * case["hkv"] * case["d"] * 3 + 8) + 8 * case["hkv"] * (T // case["block"] + 1),
                "flops": 0}
    if op == "fetch":
        T = int(_lengths(case)[0].sum())
        return {"bytes": T * 2 * case["hkv"] * case["d"] * 3 + 8 * case["hkv"] * (T // case["block"] + 1), "flops": 0}
    if op == "attend":
        pairs, keys = _visible(case)
        io = int(_lengths(case)[0].sum()) * case["hq"] * (2 * case["d"] * 2 + 4)
        return {"bytes": keys * case["hkv"] * case["d"] * 2 + 8 * case["hkv"] * keys // case["block"] + io,
                "flops": 4 * case["d"] * case["hq"] * pairs}
    live = case["rows"] - (case["rows"] // case["padding"] if case["padding"] else 0)
    return {"bytes": live * (case["vocab"] * SIZE[case["dtype"]] + 12 * case["top"] + 20), "flops": 0}


# ---------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 11)


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    x = torch.empty(shape, dtype=dtype, device="cuda")
    return x.normal_(0.0, std, generator=g)


def _int(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x)).to(device="cuda", dtype=dtype)


def _cache(g, pages, case):
    """A paged cache [pages, page, heads, d] in e4m3, its storage in the case's order, and its
    scales [pages, blocks of a page, heads]."""
    n = case["page"] // case["block"]
    if case["order"] == "hnd":
        shape = (pages, case["hkv"], case["page"], case["d"])
        values = _randn(g, *shape, dtype=torch.float16, std=100.0).clamp_(-440, 440).to(E4M3).transpose(1, 2)
    else:
        shape = (pages, case["page"], case["hkv"], case["d"])
        values = _randn(g, *shape, dtype=torch.float16, std=100.0).clamp_(-440, 440).to(E4M3)
    # blocks whose largest values differ by a factor of four
    k = torch.randint(-8, -5, (pages, n, case["hkv"]), generator=g, device="cuda")
    return values, torch.exp2(k.float())


def _frequencies(case):
    """The angle that a step of one position turns each pair by, in 64 bits."""
    rot, theta, factor, length, low, high = case["rot"], 10000.0, 8.0, 8192, 1.0, 32.0
    i = np.arange(rot // 2, dtype=np.float64)
    if case["scaling"] == "base":
        theta *= factor ** (rot / (rot - 2))
    f = theta ** (-2 * i / rot)
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] == "parts":
        # pairs that turn more than `high` times in the original length stay, below `low` they are stretched
        at = [rot * math.log(length / (2 * math.pi * r)) / (2 * math.log(theta)) for r in (high, low)]
        a, b = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = np.clip((i - a) / max(b - a, 0.001), 0, 1)
        f = f / factor * ramp + f * (1 - ramp)
    if case["scaling"] == "wavelength":
        s = np.clip((length * f / (2 * math.pi) - low) / (high - low), 0, 1)
        f = f / factor * (1 - s) + f * s
    return f


def _amplitude(case):
    return 0.1 * math.log(8.0) + 1 if case["scaling"] == "parts" else 1.0


def prepare(case, seed):
    return _PREPARE[case["op"]](case, seed, _gen(seed))


def _prepare_rotary(case, seed, g):
    T, dt = case["tokens"], DT[case["dtype"]]
    # the layout's positions: requests of up to 100 tokens, each from a position of its own
    first = torch.randint(0, case["far"], (T // 100 + 1,), generator=g, device="cuda")
    t = torch.arange(T, device="cuda")
    s = {"op": "rotary", "q": _randn(g, T, case["hq"], case["d"], dtype=dt),
         "k": _randn(g, T, case["hk"], case["d"], dtype=dt), "positions": (first[t // 100] + t % 100).int(),
         "f": torch.as_tensor(_frequencies(case)).cuda(), "amp": _amplitude(case), "interleaved": case["interleaved"]}
    s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
    if own:
        from draft_token_markov_gb300 import api
        s["api"] = api
        s["plan"] = api.RotaryPlan(case["d"], case["rot"], theta=10000.0, interleaved=case["interleaved"],
                                   scaling=case["scaling"], factor=8.0, original_len=8192, low=1.0, high=32.0)
    return s


def _prepare_store(case, seed, g):
    rows, per, ps = case["rows"], case["per"], case["page"]
    r = np.random.RandomState(seed % (1 << 31))
    # each request continues where its context ended, on pages of its own order
    c = r.randint(0, 3 * ps, rows)
    need = -(-(c + per) // ps)
    pages = rows * (3 + -(-per // ps)) + 3
    perm, first = r.permutation(pages), np.concatenate([[0], np.cumsum(need)])
    pos = c[:, None] + np.arange(per)
    slots = perm[first[:-1, None] + pos // ps] * ps + pos % ps
    T, dt = rows * per, DT[case["dtype"]]
    s = {"op": "store", "block": case["block"], "slots": _int(slots.reshape(-1), torch.int64),
         # some keys are much larger than what their blocks held so far
         "key": _randn(g, T, case["hkv"], case["d"], dtype=dt) * (1 + 7 * (torch.arange(T, device="cuda") % 5 == 0)).to(dt)[:, None, None],
         "value": _randn(g, T, case["hkv"], case["d"], dtype=dt)}
    for x in "kv":
        s[x + "_cache"], s[x + "_scales"] = _cache(g, pages, case)
    if own:
        from draft_token_markov_gb300 import api
        s["api"] = api
        s["plan"] = api.PagedPlan(case["hkv"], case["hkv"], case["d"], ps, dt, max_rows=1)
    return s


def _prepare_paged(case, seed, g):
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
    s = {"op": case["op"], "table": _int(table), "idx": _int(idx, torch.int64), "query_start": _int(start),
         "seq_lens": _int(c + q), "block": case["block"], "T": T}
    for x in "kv":
        s[x + "_cache"], s[x + "_scales"] = _cache(g, pages, case)
    if case["op"] == "fetch":
        s["key"], s["value"] = (torch.zeros((T, case["hkv"], case["d"]), dtype=dt, device="cuda") for _ in "kv")
    else:
        s |= {"q_hi": int(q.max()), "len_hi": int((c + q).max()), "scale": case["d"] ** -0.5,
              "window": case["window"], "sinks": case["sinks"],
              # scores spread with a deviation of two, as trained heads' do
              "q": _randn(g, T, case["hq"], case["d"], dtype=dt, std=1.5),
              "out": torch.zeros((T, case["hq"], case["d"]), dtype=dt, device="cuda"),
              "lse": torch.zeros((T, case["hq"]), device="cuda")}
    if own:
        from draft_token_markov_gb300 import api
        s["api"] = api
        s["plan"] = api.PagedPlan(case["hq"], case["hkv"], case["d"], ps, dt, max_rows=rows)
    return s


def _prepare_logprobs(case, seed, g):
    R, V, k = case["rows"], case["vocab"], case["top"]
    logits = _randn(g, R, V, std=3.0)
    if case["masked"]:
        # a grammar allows few ids
        off = torch.empty((R, V), device="cuda").uniform_(generator=g) < case["masked"]
        logits.masked_fill_(off, -math.inf)
        del off
    logits = logits.to(DT[case["dtype"]])
    temperature = torch.tensor([0.6, 1.0, 1.3], device="cuda")[torch.randint(0, 3, (R,), generator=g, device="cuda")]
    # tokens drawn from them
    e = torch.empty((R, V), device="cuda").exponential_(generator=g).clamp_(min=1e-30)
    tokens = (logits.float() / temperature[:, None] - e.log_()).argmax(-1)
    del e
    if case["padding"]:
        tokens[case["padding"] - 1::case["padding"]] = -1
    s = {"op": "logprobs", "logits": logits, "tokens": tokens, "temperature": temperature, "top": k,
         "logprobs": torch.full((R,), -7.0, device="cuda"), "entropy": torch.full((R,), -7.0, device="cuda"),
         "ranks": torch.full((R,), -7, dtype=torch.int32, device="cuda"),
         "top_ids": torch.full((R, k), -7, dtype=torch.int32, device="cuda"),
         "top_logprobs": torch.full((R, k), -7.0, device="cuda")}
    if own:
        from draft_token_markov_gb300 import api
        s["api"] = api
    return s


_PREPARE = {"rotary": _prepare_rotary, "store": _prepare_store, "fetch": _prepare_paged, "attend": _prepare_paged,
            "logprobs": _prepare_logprobs}


# ---------------------------------------------------------------- the passes

def run(state):
    if own:
        return _OWN[state["op"]](state)
    return _PLAIN[state["op"]](state)


def _own_rotary(s):
    s["api"].markov_rotary(s["plan"], s["q"], s["k"], s["positions"], q_out=s["q_out"], k_out=s["k_out"])
    return {"q": s["q_out"], "k": s["k_out"]}


def _plain_rotary(s):
    angle = s["positions"].double()[:, None] * s["f"]
    cos, sin = ((x * s["amp"]).float()[:, None] for x in (torch.cos(angle), torch.sin(angle)))
    n = s["f"].numel()
    out = {}
    for name in "qk":
        x = s[name].float()
        turned, rest = x[..., :2 * n], x[..., 2 * n:]
        a, b = (turned[..., 0::2], turned[..., 1::2]) if s["interleaved"] else (turned[..., :n], turned[..., n:])
        a, b = a * cos - b * sin, b * cos + a * sin
        both = torch.stack([a, b], -1).flatten(-2) if s["interleaved"] else torch.cat([a, b], -1)
        out[name] = torch.cat([both, rest], -1).to(s[name].dtype)
    return out


def _own_store(s):
    s["api"].markov_paged_write_e4m3(s["plan"], s["key"], s["value"], s["k_cache"], s["v_cache"], s["k_scales"],
                                     s["v_scales"], s["slots"])
    return {x: s[x] for x in ("k_cache", "v_cache", "k_scales", "v_scales")}


def _plain_store(s):
    B, out = s["block"], {}
    slots = s["slots"]
    block = slots // B
    for x, new in (("k", s["key"].float()), ("v", s["value"].float())):
        cache, scales = s[x + "_cache"], s[x + "_scales"]
        pages, ps, h, d = cache.shape
        n = pages * ps // B
        old = scales.reshape(n, h)
        top = torch.full((n, h), -1.0, device="cuda")
        top.scatter_reduce_(0, block[:, None].expand(-1, h), new.abs().amax(-1), "amax")
        anew = torch.zeros(n, device="cuda").scatter_reduce_(0, block, (slots % B == 0).float(), "amax") > 0
        # the least power of two that top / 448 is not above: 448 is 0.875 * 2^9
        mantissa, exponent = torch.frexp(top.clamp(min=0))
        need = torch.exp2((exponent - 9 + (mantissa > 0.875).int()).float()).clamp(min=2.0 ** -40)
        now = torch.where(anew[:, None], need, torch.maximum(old, need))
        now = torch.where(top >= 0, now, old)
        keep = torch.where(anew[:, None], 1.0, old / now)
        values = cache.float().reshape(n, B, h, d) * keep[:, None, :, None]
        values = values.reshape(n * B, h, d)
        values[slots] = new / now[block][..., None]
        cache.copy_(values.view(pages, ps, h, d).to(E4M3))
        scales.copy_(now.view(scales.shape))
        out[x + "_cache"], out[x + "_scales"] = cache, scales
    return out


def _own_fetch(s):
    s["api"].markov_paged_read_e4m3(s["plan"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["table"],
                                    s["idx"], s["query_start"], s["seq_lens"], s["T"], key=s["key"], value=s["value"])
    return {"key": s["key"], "value": s["value"]}


def _plain_fetch(s):
    ps, B = s["k_cache"].shape[1], s["block"]
    t = torch.arange(s["T"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["query_start"][1:].contiguous(), t, right=True)
    pos = s["seq_lens"][b] - s["query_start"][b + 1] + t
    page = s["table"][s["idx"][b], pos // ps]
    at = pos % ps
    out = {}
    for x, name in (("k", "key"), ("v", "value")):
        out[name] = (s[x + "_cache"][page, at].float() * s[x + "_scales"][page, at // B][..., None]).to(s[name].dtype)
    return out


def _own_attend(s):
    s["api"].markov_paged_attention_e4m3(s["plan"], s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"],
                                         s["table"], s["idx"], s["query_start"], s["seq_lens"], scale=s["scale"],
                                         window=s["window"], sinks=s["sinks"], out=s["out"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_attend(s):
    q = s["q"]
    T, hq, d = q.shape
    ps, hkv, B = s["k_cache"].shape[1], s["k_cache"].shape[2], s["block"]
    R, M, L = s["idx"].numel(), s["q_hi"], s["len_hi"]
    # every request padded to the longest: [R, hkv, M * group, L] scores
    i = torch.arange(L, device="cuda")
    page, at = s["table"][s["idx"]][:, i // ps].clamp(min=0), i % ps

    def values(x):
        return s[x + "_cache"][page, at].float() * s[x + "_scales"][page, at // B][..., None]

    k = values("k").permute(0, 2, 3, 1)
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
    v = values("v").permute(0, 2, 1, 3)
    o = (p.view(R, hkv, -1, L) @ v).view(R, hkv, M, hq // hkv, d) / torch.where(z > 0, z, 1.0)
    lse = (m + torch.log(z)).squeeze(-1)
    # back to one row per token
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["query_start"][1:].contiguous(), t, right=True)
    at = t - s["query_start"][b]
    out = o.permute(0, 2, 1, 3, 4)[b, at].reshape(T, hq, d).to(q.dtype)
    return {"out": out, "lse": lse.permute(0, 2, 1, 3)[b, at].reshape(T, hq)}


def _own_logprobs(s):
    s["api"].markov_logprobs(s["logits"], s["tokens"], s["temperature"], s["top"], logprobs=s["logprobs"],
                             ranks=s["ranks"], entropy=s["entropy"], top_ids=s["top_ids"],
                             top_logprobs=s["top_logprobs"])
    return {x: s[x] for x in ("logprobs", "ranks", "entropy", "top_ids", "top_logprobs")}


def _plain_logprobs(s):
    x, t = s["logits"].float(), s["tokens"].clamp(min=0)[:, None]
    at = torch.arange(x.shape[1], device="cuda")
    d = (x - x.amax(-1, keepdim=True)) / s["temperature"][:, None]
    e = torch.exp(d)
    z = e.sum(-1, keepdim=True)
    log_z = torch.log(z)
    own_logit = x.gather(1, t)
    out = {"logprobs": (d.gather(1, t) - log_z)[:, 0],
           "ranks": ((x > own_logit) | ((x == own_logit) & (at < t))).sum(-1, dtype=torch.int32),
           "entropy": (log_z - torch.where(e > 0, e * d, 0.0).sum(-1, keepdim=True) / z)[:, 0]}
    ids = torch.sort(x, dim=-1, descending=True, stable=True)[1][:, :s["top"]]
    out["top_ids"], out["top_logprobs"] = ids.int(), d.gather(1, ids) - log_z
    live = s["tokens"] >= 0
    return {n: torch.where(live if y.dim() == 1 else live[:, None], y, s[n]) for n, y in out.items()}


_OWN = {"rotary": _own_rotary, "store": _own_store, "fetch": _own_fetch, "attend": _own_attend,
        "logprobs": _own_logprobs}
_PLAIN = {"rotary": _plain_rotary, "store": _plain_store, "fetch": _plain_fetch, "attend": _plain_attend,
          "logprobs": _plain_logprobs}


# -------------------------------------------------------------- in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return _EXACT[case["op"]](case, s)


def _exact_rotary(case, s):
    f, n = _frequencies(case), case["rot"] // 2
    z = torch.polar(torch.full((case["tokens"], n), _amplitude(case), dtype=torch.float64, device="cuda"),
                    s["positions"].double()[:, None] * torch.as_tensor(f, device="cuda"))
    out = {}
    for name in "qk":
        x = s[name].double()
        a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if case["interleaved"] else (slice(0, n), slice(n, 2 * n))
        w = torch.complex(x[..., a], x[..., b]) * z[:, None]
        x[..., a], x[..., b] = w.real, w.imag
        out[name] = x
    return out


def _round_e4m3(x):
    """The nearest value of e4m3, ties to even, of |x| <= 448 in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_store(case, s):
    B, out, slots = case["block"], {}, s["slots"]
    first, blocks = torch.unique(slots // B, return_inverse=True)
    for x, new in (("k", s["key"].double()), ("v", s["value"].double())):
        values = s[x + "_cache"].double().reshape(-1, B, case["hkv"], case["d"])
        scales = s[x + "_scales"].double().reshape(-1, case["hkv"])
        top = torch.zeros((len(first), case["hkv"]), dtype=torch.float64, device="cuda")
        top = top.index_reduce(0, blocks, new.abs().amax(-1), "amax")
        mantissa, exponent = torch.frexp((top / 448).clamp(min=2.0 ** -40))
        need = torch.exp2(exponent.double() - (mantissa == 0.5).double())
        anew = torch.isin(first * B, slots)
        had = torch.where(anew[:, None], 0.0, scales[first])
        now = torch.maximum(had, need)
        moved = _round_e4m3(values[first] * (had / now)[:, None, :, None])
        values[first] = torch.where(anew[:, None, None, None], values[first], moved)
        values = values.reshape(-1, case["hkv"], case["d"])
        values[slots] = _round_e4m3(new / now[blocks][..., None])
        scales[first] = now
        out[x + "_cache"] = values.reshape(s[x + "_cache"].shape)
        out[x + "_scales"] = scales.reshape(s[x + "_scales"].shape)
    return out


def _gathered(s, b, L):
    """Keys and values [L, heads, d] of a request in 64 bits."""
    ps, B = s["k_cache"].shape[1], s["block"]
    pages = s["table"][s["idx"][b], :-(-L // ps)].long()
    out = []
    for x in "kv":
        y = s[x + "_cache"][pages].double() * s[x + "_scales"][pages].double().repeat_interleave(B, 1)[..., None]
        out.append(y.flatten(0, 1)[:L])
    return out


def _exact_fetch(case, s):
    parts = [_gathered(s, b, int(n)) for b, n in enumerate(_lengths(case)[0])]
    return {"key": torch.cat([k for k, _ in parts]), "value": torch.cat([v for _, v in parts])}


def _exact_attend(case, s):
    hq, hkv = case["hq"], case["hkv"]
    group = hq // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    first = 0
    for b, (n, c) in enumerate(zip(*_lengths(case))):
        n, c = int(n), int(c)
        L = c + n
        keys, values = _gathered(s, b, L)
        pos = torch.arange(c, L, device="cuda")[:, None]
        key = torch.arange(L, device="cuda")[None, :]
        hide = key > pos
        if case["window"]:
            hide |= (key <= pos - case["window"]) & (key >= case["sinks"])
        for a in range(hq):
            x = s["q"][first:first + n, a].double() @ keys[:, a // group].T * s["scale"]
            x[hide] = -math.inf
            lse[first:first + n, a] = torch.logsumexp(x, -1)
            out[first:first + n, a] = torch.softmax(x, -1) @ values[:, a // group]
        first += n
    return {"out": out, "lse": lse}


def _exact_logprobs(case, s):
    R = case["rows"]
    out = {"logprobs": s["logprobs"].double(), "entropy": s["entropy"].double(),
           "top_logprobs": s["top_logprobs"].double(), "ranks": None, "top_ids": None}
    for b in range(R):
        t = int(s["tokens"][b])
        if t < 0:
            continue
        p = torch.log_softmax(s["logits"][b].double() / float(s["temperature"][b].double()), -1)
        out["logprobs"][b] = p[t]
        some = p[p > -math.inf]
        out["entropy"][b] = -(some.exp() * some).sum()
        out["top_logprobs"][b] = torch.sort(p, descending=True)[0][:case["top"]]
    return out


_EXACT = {"rotary": _exact_rotary, "store": _exact_store, "fetch": _exact_fetch, "attend": _exact_attend,
          "logprobs": _exact_logprobs}
