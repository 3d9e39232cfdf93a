"""The verify step's entry points without a device: argument errors come back
as status codes, nothing is launched; the plain forms agree with themselves."""
import ctypes
import math

import numpy as np
import pytest
import torch

from tests import paged_ref as ref
from tests.conftest import has_gpu


@pytest.fixture(scope="module")
def L():
    from draft_token_markov_gb300 import api
    return api.lib()


def test_null_plans_are_refused(L):
    assert L.markov_paged_plan_status(None) == 1
    assert L.markov_paged_plan_inject_status(None, 4, 0) == 1
    assert L.markov_paged_layout(*([None] * 4), 1, None, 1, 1, 1, None, None, 1, *([None] * 7), 1, None) == 1
    assert L.markov_paged_write(None, None, 0, 0, None, 0, 0, None, None, None, 1, None) == 1
    assert L.markov_paged_attention(None, None, 0, 0, None, None, None, 1, 1, 1, None, None, None, 1, 1, 1.0, 0, 0,
                                    None, 0, 0, None, None) == 1
    assert L.markov_verify(None, None, 0, 0, 0, None, 0, None, 0, 0, 0, None, None, 0, None, 0, None, 1, None, 0,
                           None, None, None, None) == 1
    L.markov_paged_plan_destroy(None)


@pytest.mark.parametrize("bad", [dict(q_heads=5), dict(q_heads=1), dict(q_heads=258), dict(q_heads=256, kv_heads=1), dict(kv_heads=0),
                                 dict(head_dim=96), dict(page_size=24), dict(page_size=4), dict(page_size=512),
                                 dict(max_rows=0), dict(max_rows=1025), dict(dtype=1), dict(dtype=3),
                                 dict(timeout_ms=-1)])
def test_paged_desc_validation(L, bad):
    from draft_token_markov_gb300.api import _PagedDesc
    a = dict(q_heads=4, kv_heads=2, head_dim=64, page_size=16, max_rows=4, dtype=0, device=0, timeout_ms=0)
    h = ctypes.c_void_p()
    d = _PagedDesc(**dict(a, **bad))
    assert L.markov_paged_plan_create(ctypes.byref(d), ctypes.byref(h)) == 1 and not h.value
    assert L.markov_paged_plan_create(ctypes.byref(d), None) == 1
    assert L.markov_paged_plan_create(None, ctypes.byref(h)) == 1


@pytest.mark.skipif(has_gpu(), reason="checks the no-device answer")
def test_paged_plan_without_device(L):
    from draft_token_markov_gb300.api import _PagedDesc
    h = ctypes.c_void_p()
    d = _PagedDesc(4, 2, 64, 16, 4, 0, 0, 0)
    assert L.markov_paged_plan_create(ctypes.byref(d), ctypes.byref(h)) == 6


# --------------------------------------------------- the plain forms themselves

def test_plain_layout_keeps_every_page_once():
    rng = np.random.default_rng(0)
    S, W, page, C = 6, 9, 8, 40
    table, held, ring, free = np.full((S, W), -1), np.zeros(S, int), rng.permutation(C), [0, C]
    ctx = np.zeros(S, int)
    for _ in range(60):
        q = rng.integers(0, 20, S)
        ctx = np.where(rng.random(S) < 0.2, 0, ctx)
        r = ref.layout(page, ctx, q, np.arange(S), table, held, ring, tuple(free), int(q.sum()))
        table, held, ring, free = r["page_table"], r["pages_held"], r["free_pages"], r["free_state"]
        owned = [int(p) for s in range(S) for p in table[s, :held[s]]]
        left = [int(ring[(free[0] + k) % C]) for k in range(free[1])]
        assert sorted(owned + left) == list(range(C))
        ctx = np.where(np.array(r["seq_lens"]) > 0, r["seq_lens"], ctx)


def test_plain_attention_against_a_dense_softmax():
    g = torch.Generator().manual_seed(0)
    L, d = 21, 64
    kc, vc = torch.randn((4, 8, 1, d), generator=g).bfloat16(), torch.randn((4, 8, 1, d), generator=g).bfloat16()
    q = torch.randn((3, 2, d), generator=g).bfloat16()
    table = torch.tensor([[2, 0, 3]])
    out, lse, _, _ = ref.attention(q, kc, vc, table, [0], [0, 3], [L], 0.2, 5, 2, 8)
    k, v = (c[table[0]].reshape(-1, d)[:L].double() for c in (kc, vc))
    for j in range(3):
        p = L - 3 + j
        mask = torch.full((L,), -math.inf)
        mask[:2], mask[p - 4:p + 1] = 0, 0
        x = q[j].double() @ k.T * 0.2 + mask
        assert torch.allclose(out[j], torch.softmax(x, -1) @ v) and torch.allclose(lse[j], torch.logsumexp(x, -1))


def test_plain_verify_draws_from_the_target():
    rng = np.random.default_rng(1)
    V, n = 5, 4000
    t, d = rng.normal(size=(2, V)), rng.normal(size=(1, V))
    p, q = ref.distribution(t[0], 1.0)[0], ref.distribution(d[0], 1.0)[0]
    seen = np.zeros(V)
    for _ in range(n):
        x = rng.choice(V, p=q)
        out, _, _, _, _ = ref.verify_row(t, np.array([x]), d, 1.0, rng.random(1), rng.gumbel(size=V))
        seen[out[0]] += 1
    assert (np.abs(seen - n * p) <= 5 * np.sqrt(n * p * (1 - p)) + 1).all()
