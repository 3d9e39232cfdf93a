"""The entry points around the verify step without a device: argument errors come
back as status codes, nothing is launched; the plain forms agree with themselves."""
import ctypes
import math

import numpy as np
import pytest
import torch

from tests import serving_ref as ref
from tests.conftest import has_gpu


@pytest.fixture(scope="module")
def L():
    from draft_token_markov_gb300 import api
    return api.lib()


def test_null_plans_are_refused(L):
    assert L.markov_rotary(None, None, 0, 0, 1, None, 0, 0, 0, 0, None, 1, None, 0, 0, None, 0, 0, None) == 1
    assert L.markov_paged_write_e4m3(None, None, 0, 0, None, 0, 0, None, None, None, 1, 0, None) == 1
    assert L.markov_paged_read_e4m3(None, None, None, None, 1, 1, 1, None, None, None, 1, 1, None, 0, 0, None, 0, 0, None) == 1
    assert L.markov_paged_attention_e4m3(None, None, 0, 0, None, None, None, 1, 1, 1, None, None, None, 1, 1, 1.0, 0, 0, None,
                                         0, 0, None, None) == 1
    L.markov_rotary_plan_destroy(None)


def _desc(**kw):
    from draft_token_markov_gb300.api import _RotaryDesc
    a = dict(head_dim=64, rot_dim=32, interleaved=0, scaling=0, device=0, theta=1e4, factor=2.0, original_len=4096.0, low=1.0,
             high=32.0, amplitude=0.0, frequencies=None)
    return _RotaryDesc(**dict(a, **kw))


@pytest.mark.parametrize("bad", [dict(head_dim=8), dict(head_dim=72), dict(head_dim=528), dict(rot_dim=0), dict(rot_dim=24),
                                 dict(rot_dim=80), dict(interleaved=2), dict(scaling=-1), dict(scaling=6), dict(theta=1.0),
                                 dict(theta=math.nan), dict(theta=math.inf), dict(amplitude=-1.0), dict(amplitude=math.nan),
                                 dict(scaling=1, factor=0.0), dict(scaling=1, factor=0.1), dict(scaling=2, factor=math.inf),
                                 dict(scaling=3, original_len=0.0), dict(scaling=3, low=0.0), dict(scaling=4, low=32.0),
                                 dict(scaling=4, high=math.nan), dict(scaling=5)])
def test_rotary_desc_validation(L, bad):
    h = ctypes.c_void_p()
    assert L.markov_rotary_plan_create(ctypes.byref(_desc(**bad)), ctypes.byref(h)) == 1 and not h.value
    assert L.markov_rotary_plan_create(ctypes.byref(_desc()), None) == 1
    assert L.markov_rotary_plan_create(None, ctypes.byref(h)) == 1


def test_given_frequencies_are_checked(L):
    h = ctypes.c_void_p()
    for bad in (math.nan, math.inf, 6.3, -7.0):
        f = (ctypes.c_double * 16)(*([0.5] * 15 + [bad]))
        assert L.markov_rotary_plan_create(ctypes.byref(_desc(scaling=5, frequencies=f)), ctypes.byref(h)) == 1


@pytest.mark.skipif(has_gpu(), reason="checks the no-device answer")
def test_rotary_plan_without_device(L):
    h = ctypes.c_void_p()
    assert L.markov_rotary_plan_create(ctypes.byref(_desc()), ctypes.byref(h)) == 6


def test_logprobs_refusals(L):
    x = (ctypes.c_float * 64)()
    t = (ctypes.c_int64 * 4)()
    p, q = ctypes.addressof(x), ctypes.addressof(t)

    def call(logits=p, dtype=1, s0=8, rows=4, vocab=8, tokens=q, top=2, logprobs=p, ranks=p, entropy=p, ids=p, top_p=p):
        return L.markov_logprobs(logits, dtype, s0, rows, vocab, tokens, None, top, logprobs, ranks, entropy, ids, top_p, None)

    for bad in (dict(dtype=2), dict(dtype=3), dict(s0=7), dict(rows=-1), dict(vocab=0), dict(vocab=262145), dict(top=-1), dict(top=33),
                dict(top=9), dict(tokens=None), dict(ids=None), dict(top_p=None), dict(logits=None), dict(logits=p + 2)):
        assert call(**bad) == 1, bad
    assert call(rows=0) == 0
    assert call(logprobs=None, ranks=None, entropy=None, ids=None, top_p=None) == 0
    if not has_gpu():
        assert call() == 6                                    # host memory


# --------------------------------------------------- the plain forms themselves

def test_plain_rounding_is_the_types_own():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(20000, generator=g) * torch.exp2(torch.randint(-12, 9, (20000,), generator=g).float())
    x = x.clamp(-448, 448)
    assert torch.equal(ref.round_e4m3(x.double()).float(), x.to(torch.float8_e4m3fn).float())


def test_plain_store_keeps_values_within_a_rounding():
    g = torch.Generator().manual_seed(1)
    x = torch.randn((40, 2, 8), generator=g)
    c, s = ref.store(x, torch.zeros((3, 16, 2, 8)), torch.zeros((3, 1, 2)), torch.arange(3, 43), False)
    got = ref.values_of(c, s).reshape(48, 2, 8)[3:43]
    assert bool(((got - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -10 * s.max()).all())
    assert float(c.abs().max()) <= 448 and bool((torch.log2(s) % 1 == 0).all())


def test_plain_attention_is_the_paged_one_on_read_back_values():
    from tests import paged_ref
    g = torch.Generator().manual_seed(2)
    kc, vc = (torch.randn((4, 16, 2, 64), generator=g).to(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.exp2(torch.randint(-3, 3, (4, 1, 2), generator=g).float()) for _ in range(2))
    q = torch.randn((3, 4, 64), generator=g).bfloat16()
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32)
    a = ref.attention(q, kc, vc, ks, vs, table, [0], [0, 3], [37], 0.2, 9, 2)
    b = paged_ref.attention(q, ref.values_of(kc, ks).bfloat16(), ref.values_of(vc, vs).bfloat16(), table, [0], [0, 3], [37], 0.2, 9, 2, 16)
    assert torch.allclose(a[0], b[0]) and torch.allclose(a[1], b[1])


def test_plain_rotary_keeps_lengths_and_differences():
    f = ref.frequencies(64, scaling="parts", factor=4.0, length=4096.0)
    g = torch.Generator().manual_seed(3)
    q, k = (torch.randn((1, 1, 64), generator=g).double() for _ in range(2))
    at = lambda x, p, i: ref.rotary(x, torch.tensor([p]), f, i)[0]  # noqa: E731
    for i in (False, True):
        assert abs(float((at(q, 1000, i) ** 2).sum() - (q ** 2).sum())) < 1e-9
        assert abs(float((at(q, 1007, i) * at(k, 1000, i)).sum() - (at(q, 7, i) * k).sum())) < 1e-9


def test_plain_logprobs_against_a_dense_softmax():
    rng = np.random.default_rng(4)
    l = rng.normal(size=200) * 3
    p, rank, entropy, ids, top = ref.logprobs(l, 17, 0.7, 5)
    dense = torch.log_softmax(torch.as_tensor(l / 0.7), 0)
    assert abs(p - float(dense[17])) < 1e-12 and abs(entropy + float((dense.exp() * dense).sum())) < 1e-12
    assert rank == int((dense > dense[17]).sum()) and ids.tolist() == torch.topk(dense, 5)[1].tolist()
    l[3] = math.nan
    p, rank, entropy, ids, top = ref.logprobs(l, 17, 0.7, 2)
    assert p == -math.inf and entropy == 0 and ids[0] == 3 and top.tolist() == [0, -math.inf]
