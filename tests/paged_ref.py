"""Plain 64-bit forms of the verify step's operators, on the CPU, one request
and one token after the other, for the tests to compare with."""
from __future__ import annotations

import math

import numpy as np
import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half an ulp of 1


# ------------------------------------------------------------------ layout

def layout(page, context, query, idx, table, held, ring, free, T):
    """The layout call's outputs and updated state, as python integers."""
    table, held, ring = table.copy(), held.copy(), ring.copy()
    old = held.copy()
    head, count = free
    C, width, states = len(ring), table.shape[1], len(held)
    start, lens, pos, slots = [0], [], [], []
    taken = returned = demand = 0
    for c, q, s in zip(context, query, idx):
        c, q, s = int(c), int(q), int(s)
        ok = 0 <= s < states and c >= 0 and q >= 0 and c + q <= width * page
        if ok:
            n, h = -(-(c + q) // page), int(old[s])
            demand += max(0, n - h)
            if n > h and demand > count:
                ok = False
        if ok:
            for k in range(h, n):
                table[s, k] = ring[(head + taken) % C]
                taken += 1
            for k in range(n, h):
                ring[(head + count + returned) % C] = table[s, k]
                returned += 1
            held[s] = n
        for j in range(max(q, 0)):
            pos.append(c + j if ok else 0)
            slots.append(int(table[s, (c + j) // page]) * page + (c + j) % page if ok else -1)
        start.append(start[-1] + max(q, 0))
        lens.append(c + q if ok else 0)
    pos, slots = (pos + [0] * T)[:T], (slots + [-1] * T)[:T]
    return dict(query_start=start, seq_lens=lens, positions=pos, slots=slots, page_table=table,
                pages_held=held, free_pages=ring,
                free_state=[(head + taken) % C, count - taken + returned])


# --------------------------------------------------------------- attention

def visible(n_seen, pos, window, sinks):
    """Key indices that a token at `pos` sees of n_seen keys."""
    i = np.arange(max(0, min(pos + 1, n_seen)))
    if window:
        i = i[(i > pos - window) | (i < sinks)]
    return i


def attention(q, k_cache, v_cache, table, idx, start, lens, scale, window, sinks, page):
    """(out, lse, bound on out's error, bound on lse's error) in fp64; tokens
    of padding rows are NaN in all four.

    The bounds: scores are sums of head_dim products whose terms are exact, so
    their error is at most head_dim roundings of 2^-23 (an addition that may
    truncate) of sum |q k|; the weights are off by that exponent's error and
    one rounding to the type, the output by one more.  fp16 weights below the
    normal range are off by half the smallest step, 2^-25, of a sum that is at
    least 1.  fp32 exponentials, sums and divisions are within 1e-5."""
    T, hq, d = q.shape
    hkv = k_cache.shape[2]
    unit = UNIT[q.dtype]
    q, kc, vc = q.double(), k_cache.double(), v_cache.double()
    out = torch.full((T, hq, d), math.nan, dtype=torch.float64)
    lse = torch.full((T, hq), math.nan, dtype=torch.float64)
    tol, tol_lse = out.clone(), lse.clone()
    for b in range(len(idx)):
        s, n, L = int(idx[b]), int(start[b + 1] - start[b]), int(lens[b])
        if s < 0:
            continue
        for j in range(n):
            t = int(start[b]) + j
            if t >= T:
                continue
            i = visible(table.shape[1] * page, L - n + j, window, sinks)
            if len(i) == 0:
                out[t], lse[t], tol[t], tol_lse[t] = 0, -math.inf, 0, 0
                continue
            pages = table[s, i // page].long()
            bad = (pages < 0) | (pages >= kc.shape[0])
            pages = pages.clamp(0, kc.shape[0] - 1)
            at = torch.as_tensor(i % page)
            k, v = kc[pages, at], vc[pages, at]
            k[bad], v[bad] = 0, 0
            k = k.repeat_interleave(hq // hkv, 1)
            v = v.repeat_interleave(hq // hkv, 1)
            x = torch.einsum("hd,ihd->hi", q[t], k) * scale
            e = d * 2.0 ** -23 * abs(scale) * torch.einsum("hd,ihd->hi", q[t].abs(), k.abs()).amax(1)
            lse[t] = torch.logsumexp(x, 1)
            w = torch.softmax(x, 1)
            out[t] = torch.einsum("hi,ihd->hd", w, v)
            mass = torch.einsum("hi,ihd->hd", w, v.abs())
            tol[t] = (unit + 2 * e[:, None] + 1e-5) * mass + unit * out[t].abs()
            if unit < 2.0 ** -10:
                tol[t] += 2.0 ** -25 * v.abs().sum(0) + 2.0 ** -25
            tol_lse[t] = e + 1e-5 * (1 + lse[t].abs())
    return out, lse, tol * 1.01, tol_lse


# ------------------------------------------------------------------ verify

def distribution(l, T):
    """softmax(l / T) in fp64, or the one-hot of the argmax order."""
    nan = np.isnan(l)
    top = -np.inf if nan.all() else np.max(l[~nan])
    if nan.any() or not np.isfinite(top) or not T > 0:
        p = np.zeros(len(l))
        p[np.argmax(nan) if nan.any() else np.argmax(l == top)] = 1.0
        return p, True
    e = np.exp((l - top) / np.float64(T))
    return e / e.sum(), False


def verify_row(target, tokens, draft, T, uniforms, noise):
    """One row: (tokens out, accepted, p, q, near) in fp64.  near: the
    smallest relative distance by which a decision was taken (a test keeps
    rows whose decisions fp32 cannot turn)."""
    N, V = draft.shape
    P = [distribution(target[i].astype(np.float64), T) for i in range(N + 1)]
    Q = [distribution(draft[i].astype(np.float64), T) for i in range(N)]
    p = np.array([P[i][0][tokens[i]] if 0 <= tokens[i] < V else 0.0 for i in range(N)])
    q = np.array([Q[i][0][tokens[i]] if 0 <= tokens[i] < V else 0.0 for i in range(N)])
    n, near = 0, np.inf
    for i in range(N):
        a, b = float(uniforms[i]) * q[i], p[i]
        if max(a, b) > 0 and not (P[i][1] and Q[i][1]):
            near = min(near, abs(a - b) / max(a, b))
        if not a < b:
            break
        n += 1
    r, one = P[n]
    if n < N and not one:
        rest = np.maximum(r - Q[n][0], 0)
        r = rest if rest.max() > 0 else r
    if one:
        own = int(np.argmax(r))
    else:
        with np.errstate(divide="ignore"):
            key = np.log(r) + noise.astype(np.float64)
        own = int(np.argmax(key))
        two = np.sort(key)[-2:]
        near = min(near, two[1] - two[0])
    out = [int(x) for x in tokens[:n]] + [own] + [-1] * (N - n)
    return out, n, p, q, near
