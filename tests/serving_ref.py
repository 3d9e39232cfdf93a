"""Plain 64-bit forms of the operators around the verify step (rotary positions,
e4m3 caches, log probabilities) for the tests to compare with."""
from __future__ import annotations

import math

import numpy as np
import torch

from tests.paged_ref import UNIT, visible

E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ rotary

def frequencies(rot, theta=10000.0, scaling="none", factor=1.0, length=0.0, low=1.0, high=32.0):
    """Radians per position of each pair."""
    out = []
    for i in range(rot // 2):
        base = theta * factor ** (rot / (rot - 2)) if scaling == "base" else theta
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= factor
        elif scaling == "parts":
            def dim(r):
                return rot * math.log(length / (2 * math.pi * r)) / (2 * math.log(theta))
            a, b = max(math.floor(dim(high)), 0), min(math.ceil(dim(low)), rot - 1)
            t = min(max((i - a) / max(b - a, 0.001), 0.0), 1.0)
            f = f / factor * t + f * (1 - t)
        elif scaling == "wavelength":
            t = min(max((length * f / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
            f = f * t + f / factor * (1 - t)
        out.append(f)
    return np.array(out)


def rotary(x, positions, f, interleaved, amplitude=1.0):
    """(turned, bound on the error) of x [T, H, D] in fp64: sines and cosines are off
    by at most 2^-22 (their angle and themselves in fp32), times the amplitude, rounded
    (2^-24); two products and their sum are rounded, then the result."""
    n = len(f)
    y = x.double().clone()
    t = positions.double()[:, None] * torch.as_tensor(f, dtype=torch.float64, device=x.device)
    cos, sin = torch.cos(t)[:, None] * amplitude, torch.sin(t)[:, None] * amplitude
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    xa, xb = x.double()[..., a], x.double()[..., b]
    y[..., a], y[..., b] = xa * cos - xb * sin, xb * cos + xa * sin
    tol = torch.zeros_like(y)
    both = (xa.abs() + xb.abs()) * (2.0 ** -22 + 3 * 2.0 ** -24) * amplitude
    tol[..., a], tol[..., b] = both, both
    unit = UNIT.get(x.dtype, 2.0 ** -24)
    tol[..., :2 * n] += unit * y[..., :2 * n].abs()
    if unit == 2.0 ** -11:
        tol[..., :2 * n] += 2.0 ** -25
    return y, tol


# ------------------------------------------------------------- e4m3 caches

def scale_of(top):
    """The least power of two that top / 448 is not above, 2^-40 at least."""
    s = 2.0 ** -40
    while s * 448 < top:
        s *= 2
    return s


def round_e4m3(x):
    """fp64 values as the nearest of e4m3, ties to even, beyond +-448 that."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(2.0 ** -6, 448))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def store(new, cache, scales, slots, keep):
    """The cache [pages, page, heads, d] (values in fp64) and its scales after
    a store, one cache block after the other."""
    pages, page, heads, d = cache.shape
    B = page // scales.shape[1]
    out, s_out = cache.double().clone(), scales.double().clone()
    new = new.double()
    by_block = {}
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pages * page:
            by_block.setdefault(s // B, []).append((s, t))
    for b, tokens in by_block.items():
        p, k = b * B // page, b * B % page // B
        for h in range(heads):
            x = torch.stack([new[t, h] for _, t in tokens])
            old = float(s_out[p, k, h])
            s = old
            if not keep:
                finite = x[torch.isfinite(x)].abs()
                s = scale_of(float(finite.max()) if len(finite) else 0.0)
                anew = any(slot % B == 0 for slot, _ in tokens)
                if not anew and old > 0 and math.isfinite(old):
                    if s > old:
                        block = out[p, k * B:(k + 1) * B, h]
                        out[p, k * B:(k + 1) * B, h] = round_e4m3((block.float() * (np.float32(old) / np.float32(s))).double())
                    else:
                        s = old
                s_out[p, k, h] = s
            for (slot, _), row in zip(tokens, x):
                q = (row.float() / np.float32(s)).double()
                out[p, slot % page, h] = round_e4m3(q)
    return out, s_out


def values_of(cache, scales):
    """What the elements stand for, fp64 [pages, page, heads, d]."""
    return cache.double() * scales.double().repeat_interleave(cache.shape[1] // scales.shape[1], 1)[..., None]


def attention(q, k_cache, v_cache, k_scales, v_scales, table, idx, start, lens, scale, window, sinks):
    """(out, lse, bound on out's error, bound on lse's error) in fp64; tokens of
    padding rows are NaN in all four.

    The bounds: scores are sums of head_dim products of exact terms, so their error is
    at most head_dim roundings of 2^-23 (an addition that may truncate) of sum |q k|;
    the factors after that (scale, log2 e, a block's scale) add a few 2^-24 of the
    score, which that covers.  The weights are off by that exponent's error and one
    rounding to fp16, 2^-11; below fp16's normal range by half its smallest step,
    2^-25, where the largest weight is 2^7 at least (times the ratio of two blocks' value
    scales).  The output is rounded once.  fp32 exponentials, sums and divisions are
    within 1e-5."""
    T, hq, d = q.shape
    page, hkv = k_cache.shape[1:3]
    kc, vc = values_of(k_cache, k_scales), values_of(v_cache, v_scales)
    q64 = q.double()
    unit = UNIT[q.dtype]
    out = torch.full((T, hq, d), math.nan, dtype=torch.float64, device=q.device)
    lse = torch.full((T, hq), math.nan, dtype=torch.float64, device=q.device)
    tol, tol_lse = out.clone(), lse.clone()
    raw_v = v_cache.double().abs()
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
            i = torch.as_tensor(i, device=q.device)
            pages = table[s, i // page].long() if s < table.shape[0] else torch.full_like(i, -1)
            bad = (pages < 0) | (pages >= kc.shape[0])
            pages = pages.clamp(0, kc.shape[0] - 1)
            at = i % page
            k, v, raw = kc[pages, at], vc[pages, at], raw_v[pages, at]
            k[bad], v[bad], raw[bad] = 0, 0, 0
            used = v_scales[pages, at // (page // v_scales.shape[1])].clone()
            used[bad] = 1.0
            top_scale = float(used.amax())
            k, v, raw = (x.repeat_interleave(hq // hkv, 1) for x in (k, v, raw))
            x = torch.einsum("hd,ihd->hi", q64[t], k) * scale
            e = d * 2.0 ** -23 * abs(scale) * torch.einsum("hd,ihd->hi", q64[t].abs(), k.abs()).amax(1)
            lse[t] = torch.logsumexp(x, 1)
            w = torch.softmax(x, 1)
            out[t] = torch.einsum("hi,ihd->hd", w, v)
            mass = torch.einsum("hi,ihd->hd", w, v.abs())
            tol[t] = (2.0 ** -11 + 2 * e[:, None] + 1e-5) * mass + unit * out[t].abs()
            tol[t] += 2.0 ** -32 * top_scale * raw.sum(0)
            if unit == 2.0 ** -11:
                tol[t] += 2.0 ** -25
            tol_lse[t] = e + 1e-5 * (1 + lse[t].abs())
    return out, lse, tol * 1.01, tol_lse


# ------------------------------------------------------- log probabilities

def logprobs(l, token, T, top):
    """(logprob, rank, entropy, ids, their logprobs) of one row of fp64 logits."""
    V = len(l)
    nan = np.isnan(l)
    if not T > 0:
        T = 1.0
    # NaN above all, then by falling logit, the lowest id first
    order = np.lexsort((np.arange(V), -np.where(nan, np.inf, l), ~nan))
    first = order[0]
    if nan.any() or not np.isfinite(l[first]):
        p = np.full(V, -np.inf)
        p[first] = 0.0
        entropy = 0.0
    else:
        with np.errstate(invalid="ignore", over="ignore"):
            d = np.where(np.isneginf(l), -np.inf, 0.0) if np.isinf(T) else (l - l[first]) / T
        p = d - math.log(np.exp(d).sum())
        some = p > -np.inf
        entropy = float(-(np.exp(p[some]) * p[some]).sum())
    rank = int(np.nonzero(order == token)[0][0]) if 0 <= token < V else None
    ids = order[:top]
    return (p[token] if rank is not None else None), rank, entropy, ids, p[ids]
