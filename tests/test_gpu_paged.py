"""The paged calls on the GPU against their plain 64-bit forms: page tables
and slots from request lengths, cache writes, and attention of new tokens
over the paged cache (chunks, single tokens, windows, first tokens kept,
ragged and empty rows, strides, streams, graphs)."""
import math

import numpy as np
import pytest
import torch

from tests import paged_ref as ref

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ layout

def _layout_state(rng, states, width, page, held, extra=8, head=None):
    total = int(sum(held)) + extra
    perm = rng.permutation(total)
    table = np.full((states, width), -1, np.int32)
    at = 0
    for s in range(states):
        table[s, :held[s]] = perm[at:at + held[s]]
        at += held[s]
    head = int(rng.integers(total)) if head is None else head
    ring = np.full(total, -1, np.int32)
    ring[(head + np.arange(extra)) % total] = perm[at:]
    return table, np.array(held, np.int32), ring, np.array([head, extra], np.int64)


def _layout_both(api, page, context, query, idx, table, held, ring, free, T, in_place=True):
    plan = api.PagedPlan(4, 4, 64, page, max_rows=len(context))
    d = lambda x, t: torch.as_tensor(np.asarray(x)).to(device="cuda", dtype=t)  # noqa: E731
    i32, i64 = torch.int32, torch.int64
    st = [d(table, i32), d(held, i32), d(ring, i32), d(free, i64)]
    more = {} if in_place else {"pages_held_out": st[1].clone(), "free_state_out": torch.zeros_like(st[3])}
    got = api.markov_paged_layout(plan, d(context, i32), d(query, i32), d(idx, i64), *st, T, **more)
    assert api.markov_paged_plan_status(plan) == 0
    plan.close()
    if not in_place:
        assert st[1].tolist() == list(held) and st[3].tolist() == list(free)
        st[1], st[3] = more["pages_held_out"], more["free_state_out"]
    want = ref.layout(page, context, query, idx, table, held, ring, tuple(int(x) for x in free), T)
    have = dict(zip(("query_start", "seq_lens", "positions", "slots"), got))
    have.update(zip(("page_table", "pages_held", "free_pages", "free_state"), st))
    for k, w in want.items():
        assert np.array_equal(have[k].cpu().numpy(), np.asarray(w)), k


@pytest.mark.parametrize("rows,page,T_extra", [(1, 8, 0), (8, 16, 3), (33, 32, 0), (256, 16, 5),
                                               (257, 64, 1), (1000, 8, 0)])
@pytest.mark.parametrize("in_place", [True, False])
def test_layout_ragged(gpu_lib, rows, page, T_extra, in_place):
    rng = np.random.default_rng(rows + page)
    context, query = rng.integers(0, 300, rows), rng.integers(0, 12, rows)
    states = rows + 3
    idx = rng.permutation(states)[:rows].astype(np.int64)
    idx[rng.random(rows) < 0.1] = -1
    held = np.zeros(states, np.int64)
    for b in range(rows):
        if idx[b] >= 0:
            held[idx[b]] = max(0, -(-context[b] // page) + rng.integers(-1, 3))
    table, held, ring, free = _layout_state(rng, states, 60, page, held, extra=4 * rows)
    _layout_both(gpu_lib, page, context, query, idx, table, held, ring, free,
                 int(query.sum()) + T_extra, in_place)


@pytest.mark.parametrize("rows,long_row", [(5, 2), (300, 150)])
def test_layout_one_long_prompt_among_short_rows(gpu_lib, rows, long_row):
    rng = np.random.default_rng(9)
    query = rng.integers(1, 9, rows)
    query[long_row] = 20000                                   # several blocks
    context = rng.integers(0, 200, rows)
    held = [-(-int(c) // 16) for c in context]
    table, held, ring, free = _layout_state(rng, rows, 1400, 16, held, extra=2000 + 2 * rows)
    _layout_both(gpu_lib, 16, context, query, np.arange(rows), table, held, ring, free, int(query.sum()))


def test_layout_refusals_leave_rows_alone(gpu_lib):
    rng = np.random.default_rng(3)
    #          fits  neg  too long  bad state  padding  needs 3 of the 4 left  short  needs none
    context = [10, -1, 70, 5, 5, 0, 0, 9]
    query = [8, 3, 20, 2, 2, 20, 30, 5]
    idx = [0, 1, 2, 99, -1, 3, 4, 5]
    held = [2, 1, 9, 0, 0, 2]
    table, held, ring, free = _layout_state(rng, 6, 10, 8, held, extra=5)
    _layout_both(gpu_lib, 8, context, query, idx, table, held, ring, free, sum(max(q, 0) for q in query) + 2)


def test_layout_release_then_reuse(gpu_lib):
    """Released pages are taken by the next call, in the order they came."""
    api = gpu_lib
    rng = np.random.default_rng(4)
    table, held, ring, free = _layout_state(rng, 3, 8, 16, [3, 4, 0], extra=1, head=7)
    _layout_both(api, 16, [0, 64], [0, 0], [0, 1], table, held, ring, free, 0)
    want = ref.layout(16, [0, 64], [0, 0], [0, 1], table, held, ring, (7, 1), 0)
    _layout_both(api, 16, [0], [64], [2], want["page_table"], want["pages_held"], want["free_pages"],
                 want["free_state"], 64)


def test_layout_empty_and_all_padding(gpu_lib):
    rng = np.random.default_rng(5)
    table, held, ring, free = _layout_state(rng, 2, 4, 8, [1, 0], extra=3)
    _layout_both(gpu_lib, 8, [3, 0], [0, 0], [0, 1], table, held, ring, free, 0)
    _layout_both(gpu_lib, 8, [3, 5], [4, 2], [-1, -1], table, held, ring, free, 9)


# ------------------------------------------------------------------- cache

def _cache(pages, page, heads, d, dtype, order, fill=math.nan):
    shape = (pages, heads, page, d) if order == "hnd" else (pages, page, heads, d)
    c = torch.full(shape, fill, dtype=dtype, device="cuda")
    return c.transpose(1, 2) if order == "hnd" else c


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,heads,d,page,order", [(1, 1, 64, 8, "nhd"), (7, 3, 128, 16, "hnd"),
                                                  (130, 8, 64, 256, "nhd"), (2100, 5, 128, 32, "hnd")])
def test_write(gpu_lib, dtype, T, heads, d, page, order):
    api = gpu_lib
    g = torch.Generator(device="cuda").manual_seed(T)
    pages = T // page + 4
    kc, vc = (_cache(pages, page, heads, d, dtype, order, fill=3.0) for _ in range(2))
    # strided inputs: a slice of a wider projection's output
    wide = torch.randn((T, 2 * heads + 1, d), generator=g, device="cuda").to(dtype)
    key, value = wide[:, :heads], wide[:, heads:2 * heads]
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T]
    slots[::5] = -1
    if T > 3:
        slots[3] = pages * page                               # past the cache: skipped
    want_k, want_v = kc.clone(), vc.clone()
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pages * page:
            want_k[s // page, s % page], want_v[s // page, s % page] = key[t], value[t]
    plan = api.PagedPlan(heads, heads, d, page, dtype, max_rows=1)
    api.markov_paged_write(plan, key, value, kc, vc, slots)
    assert api.markov_paged_plan_status(plan) == 0
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)
    plan.close()


# --------------------------------------------------------------- attention

class Case:
    """Requests of the given (context, new tokens), their keys and values in
    scattered pages of a cache that holds NaN everywhere else."""

    def __init__(self, reqs, hq, hkv, d, page, dtype=torch.bfloat16, order="nhd", seed=0, padding=(),
                 width_extra=1, std=2.0, mean=0.0):
        g = torch.Generator().manual_seed(seed)
        self.page, self.dtype, self.hq, self.hkv, self.d = page, dtype, hq, hkv, d
        n = [q for _, q in reqs]
        lens = [c + q for c, q in reqs]
        need = [-(-max(L, 0) // page) for L in lens]
        pages = sum(need) + 5
        perm = torch.randperm(pages, generator=g)
        states = len(reqs) + 2
        idx = torch.randperm(states, generator=g)[:len(reqs)]
        self.table = torch.full((states, max(need) + width_extra), -7, dtype=torch.int32)
        self.kc, self.vc = (_cache(pages, page, hkv, d, dtype, order).cpu() for _ in range(2))
        at = 0
        for b, L in enumerate(lens):
            mine = perm[at:at + need[b]]
            at += need[b]
            self.table[idx[b], :need[b]] = mine.int()
            i = torch.arange(max(L, 0))
            for c in (self.kc, self.vc):
                c[mine[i // page], i % page] = (torch.randn((max(L, 0), hkv, d), generator=g) + mean).to(dtype)
        self.T = sum(n)
        self.q = (torch.randn((self.T, hq, d), generator=g) * std).to(dtype)
        self.start = torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32)
        self.lens = torch.tensor(lens, dtype=torch.int32)
        self.idx = idx.clone()
        for b in padding:
            self.idx[b] = -1

    def dev(self):
        keys = ("q", "kc", "vc", "table", "idx", "start", "lens")
        d = {k: getattr(self, k).cuda() for k in keys}
        for k in ("kc", "vc"):                       # .cuda() of a permuted view keeps its strides
            assert d[k].stride() == getattr(self, k).stride()
        return d

    def plan(self, api):
        return api.PagedPlan(self.hq, self.hkv, self.d, self.page, self.dtype, max_rows=len(self.idx))


SENT = 123.0


def run(api, case, scale=None, window=0, sinks=0, d=None, plan=None, **kw):
    d = d or case.dev()
    own = plan is None
    plan = plan or case.plan(api)
    out = torch.full((case.T, case.hq, case.d), SENT, dtype=case.dtype, device="cuda")
    lse = torch.full((case.T, case.hq), SENT, device="cuda")
    api.markov_paged_attention(plan, d["q"], d["kc"], d["vc"], d["table"], d["idx"], d["start"], d["lens"],
                               scale=scale, window=window, sinks=sinks, out=out, lse=lse, **kw)
    assert api.markov_paged_plan_status(plan) == 0
    if own:
        plan.close()
    return out, lse


def check(case, out, lse, scale=None, window=0, sinks=0):
    want, wl, tol, tl = ref.attention(case.q, case.kc, case.vc, case.table, case.idx, case.start, case.lens,
                                      case.d ** -0.5 if scale is None else scale, window, sinks, case.page)
    out, lse = out.cpu().double(), lse.cpu().double()
    dead = wl.isnan()
    assert torch.equal(out[dead], torch.full_like(out[dead], SENT)) and bool((lse[dead] == SENT).all())
    empty = wl == -math.inf
    assert bool((lse[empty] == -math.inf).all()) and bool((out[empty] == 0).all())
    live = ~dead & ~empty
    assert bool(torch.isfinite(out[live]).all()) and bool(torch.isfinite(lse[live]).all())
    over = ((out - want).abs() - tol)[live]
    assert over.numel() == 0 or float(over.max()) <= 0, float((((out - want).abs() / tol)[live]).max())
    over = ((lse - wl).abs() - tl)[live]
    assert over.numel() == 0 or float(over.max()) <= 0, float(over.max())


def both(api, case, **kw):
    out, lse = run(api, case, **kw)
    check(case, out, lse, **kw)


DT = [torch.bfloat16, torch.float16]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 1), (8, 2), (6, 2), (21, 3), (40, 1), (5, 5)])
def test_single_tokens(gpu_lib, dtype, d, hq, hkv):
    reqs = [(0, 1), (1, 1), (126, 1), (127, 1), (128, 1), (300, 1), (1000, 1)]
    both(gpu_lib, Case(reqs, hq, hkv, d, 16, dtype, seed=hq))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
def test_draft_chunks_every_page_size(gpu_lib, dtype, d, page):
    reqs = [(0, 9), (3, 9), (page - 1, 2), (2 * page - 9, 9), (517, 9), (5, 17)]
    both(gpu_lib, Case(reqs, 8, 2, d, page, dtype, order="hnd" if page % 32 else "nhd", seed=page))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 257])
def test_chunk_lengths_around_tile_edges(gpu_lib, d, n):
    both(gpu_lib, Case([(0, n), (70, n)], 4, 2, d, 16, seed=n))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 128), (7, 1, 64), (12, 4, 128)])
def test_long_chunks(gpu_lib, dtype, hq, hkv, d):
    both(gpu_lib, Case([(0, 400), (333, 150)], hq, hkv, d, 32, dtype, seed=7))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 0), (7, 3), (64, 4), (128, 0), (128, 130),
                                          (200, 1), (5, 300), (10 ** 9, 4), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_windows_and_first_tokens(gpu_lib, window, sinks):
    reqs = [(0, 1), (0, 5), (6, 1), (250, 9), (600, 1), (500, 140), (129, 128)]
    both(gpu_lib, Case(reqs, 8, 2, 64, 16, seed=window % 1000), window=window, sinks=sinks)
    both(gpu_lib, Case(reqs[2:5], 4, 4, 128, 32, torch.float16, seed=sinks % 1000), window=window, sinks=sinks)


def test_pages_before_the_window_are_not_read(gpu_lib):
    """Freed pages before the window: table entries gone, their keys NaN."""
    c = Case([(700, 1), (650, 9)], 8, 2, 128, 16, seed=3)
    window, sinks = 100, 20
    for b, n in enumerate((1, 9)):
        L = int(c.lens[b])
        first = (L - n - window + 1) // 16                    # the window's first page
        gone = c.table[c.idx[b], 2:first].long()
        c.kc[gone], c.vc[gone] = math.nan, math.nan
        c.table[c.idx[b], 2:first] = -1
        # and in the pages at both edges, what nobody sees
        for cache in (c.kc, c.vc):
            cache[c.table[c.idx[b], 1].long(), 4:] = math.nan
            edge = L - n - window + 1
            if edge % 16:
                cache[c.table[c.idx[b], first].long(), :edge % 16] = math.nan
    d = c.dev()
    out, lse = run(gpu_lib, c, window=window, sinks=sinks, d=d)
    c.kc, c.vc = c.kc.nan_to_num(0.0), c.vc.nan_to_num(0.0)
    check(c, out, lse, window=window, sinks=sinks)


def test_keys_hidden_from_one_token_may_be_anything(gpu_lib):
    """A chunk's later keys are not finite: the tokens before do not see them."""
    c = Case([(40, 3)], 4, 2, 64, 16, seed=5)
    page = int(c.table[c.idx[0], 42 // 16])
    for bad in (math.nan, math.inf, -math.inf):
        d = c.dev()
        d["kc"][page, 42 % 16] = bad
        out, lse = run(gpu_lib, c, d=d)
        clean, clean_lse = run(gpu_lib, c)
        assert torch.equal(out[:2], clean[:2]) and torch.equal(lse[:2], clean_lse[:2])


def test_rows_that_see_nothing(gpu_lib):
    """Refused rows (length 0), lengths below the chunk's, padding rows, rows without tokens."""
    c = Case([(10, 4), (0, 9), (20, 0), (3, 3), (50, 6)], 8, 4, 128, 16, seed=6, padding=(3,))
    c.lens[0] = 0                                             # refused
    c.lens[1] = 5                                             # four of nine before the start
    both(gpu_lib, c)
    both(gpu_lib, c, window=3, sinks=1)


def test_tokens_outside_every_row_are_left_alone(gpu_lib):
    c = Case([(10, 4), (0, 3)], 4, 4, 64, 16, seed=8)
    d = c.dev()
    d["q"] = torch.cat([d["q"], d["q"][:5]])
    plan = c.plan(gpu_lib)
    out = torch.full((c.T + 5, c.hq, c.d), SENT, dtype=c.dtype, device="cuda")
    gpu_lib.markov_paged_attention(plan, d["q"], d["kc"], d["vc"], d["table"], d["idx"], d["start"], d["lens"], out=out)
    want, _ = run(gpu_lib, c)
    assert torch.equal(out[:c.T], want) and bool((out[c.T:] == SENT).all())
    # and rows past the tokens that there are
    out = torch.full((5, c.hq, c.d), SENT, dtype=c.dtype, device="cuda")
    gpu_lib.markov_paged_attention(plan, d["q"][:5].clone(), d["kc"], d["vc"], d["table"], d["idx"], d["start"], d["lens"], out=out)
    assert torch.equal(out, want[:5])
    plan.close()


def test_length_past_the_table(gpu_lib):
    """A length beyond the table's keys sees the table's keys only."""
    c = Case([(60, 4)], 4, 2, 64, 16, seed=9, width_extra=0)
    c.lens[0] = 200
    both(gpu_lib, c)


def test_page_ids_outside_the_cache_read_as_zeros(gpu_lib):
    c = Case([(200, 2)], 4, 2, 128, 16, seed=10)
    c.table[c.idx[0], 3], c.table[c.idx[0], 7] = -5, c.kc.shape[0] + 3
    both(gpu_lib, c)


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 5.0])
def test_scales(gpu_lib, scale):
    both(gpu_lib, Case([(300, 3), (5, 40)], 4, 2, 64, 16, seed=11), scale=scale)


def test_rising_scores(gpu_lib):
    """Keys whose scores rise all the way, by far more than a weight's range."""
    c = Case([(900, 2), (400, 130)], 4, 2, 128, 16, seed=12, std=1.0)
    for b in range(2):
        i = torch.arange(int(c.lens[b]))
        pages = c.table[c.idx[b], i // 16].long()
        c.kc[pages, i % 16, :, 0] = (i.float() / 8).to(c.dtype)[:, None]
    c.q[..., 0] = 20.0
    both(gpu_lib, c)


@pytest.mark.parametrize("mean", [0.0, 5.0])
def test_many_ragged_rows(gpu_lib, mean):
    """More rows than blocks, of every length, split between blocks."""
    rng = np.random.default_rng(1)
    reqs = [(int(c), int(q)) for c, q in zip(rng.integers(0, 260, 200), rng.integers(1, 4, 200))]
    both(gpu_lib, Case(reqs, 4, 2, 64, 8, torch.float16 if mean else torch.bfloat16, seed=13, mean=mean))


@pytest.mark.parametrize("hq,hkv,d", [(128, 1, 64), (100, 1, 128), (129 * 1, 3, 64), (256, 2, 64)])
def test_large_groups(gpu_lib, hq, hkv, d):
    """Groups that fill a row tile, leave some of it, or all but one row."""
    both(gpu_lib, Case([(50, 3), (200, 1), (0, 2)], hq, hkv, d, 16, seed=hq))


def test_a_thousand_rows(gpu_lib):
    rng = np.random.default_rng(2)
    reqs = [(int(c), 1) for c in rng.integers(0, 40, 1000)]
    reqs[700] = (5000, 3)
    both(gpu_lib, Case(reqs, 2, 1, 64, 8, seed=19, padding=(0, 31, 32, 999)))


def test_window_and_first_tokens_far_apart(gpu_lib):
    """Key tiles of the first tokens and of the window, with many between."""
    c = Case([(3000, 9), (5000, 1), (2500, 300)], 4, 2, 128, 32, seed=20)
    both(gpu_lib, c, window=130, sinks=200)
    both(gpu_lib, c, window=1, sinks=129)


def test_more_key_tiles_than_are_counted(gpu_lib):
    """2^31 key tiles of work: refused on the device, nothing is written."""
    api = gpu_lib
    plan = api.PagedPlan(256, 256, 64, 256, torch.bfloat16, max_rows=1)
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = torch.zeros((1, 256, 256, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((1, 256, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, SENT)
    api.markov_paged_attention(plan, q, cache, cache.clone(), torch.full((1, 1 << 22), -1, **i32),
                               torch.zeros(1, dtype=torch.int64, device="cuda"), torch.tensor([0, 1], **i32),
                               torch.tensor([1 << 30], **i32), out=out)
    assert api.markov_paged_plan_status(plan) == 2 and bool((out == SENT).all())
    assert api.markov_paged_plan_status(plan) == 0
    plan.close()


def test_one_long_row_is_split(gpu_lib):
    """One token over a long cache, where blocks share the row."""
    for dtype, d, reqs in ((torch.bfloat16, 128, [(20000, 1)]), (torch.float16, 64, [(9000, 9), (17, 1)])):
        both(gpu_lib, Case(reqs, 2, 1, d, 64, dtype, seed=14))


def test_strided_queries_and_outputs(gpu_lib):
    """Queries out of a fused projection, outputs into a wider buffer."""
    c = Case([(30, 5), (200, 2)], 6, 2, 64, 16, seed=15)
    d = c.dev()
    wide = torch.full((c.T, 10, 64), math.nan, dtype=c.dtype, device="cuda")
    wide[:, 2:8] = d["q"]
    d["q"] = wide[:, 2:8]
    plan = c.plan(gpu_lib)
    buf = torch.full((c.T, 12, 64), SENT, dtype=c.dtype, device="cuda")
    out = buf[:, ::2]
    gpu_lib.markov_paged_attention(plan, d["q"], d["kc"], d["vc"], d["table"], d["idx"], d["start"], d["lens"], out=out)
    want, _ = run(gpu_lib, c)
    assert torch.equal(out, want) and bool((buf[:, 1::2] == SENT).all())
    plan.close()


def test_same_bits_every_time_and_on_another_stream(gpu_lib):
    c = Case([(3000, 1), (700, 9), (100, 200)], 8, 2, 128, 16, seed=16)
    d = c.dev()
    plan = c.plan(gpu_lib)
    want, wl = run(gpu_lib, c, d=d, plan=plan)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        out, lse = gpu_lib.markov_paged_attention(plan, d["q"], d["kc"], d["vc"], d["table"], d["idx"], d["start"],
                                                  d["lens"], lse=True, stream=s)
        s.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)
    plan.close()


def test_row_of_the_batch_does_not_change_its_bits_alone(gpu_lib):
    """A row's result is within the bound whatever shares the call."""
    big = Case([(500, 9)] + [(i * 37 % 900, 1 + i % 9) for i in range(60)], 8, 2, 64, 16, seed=17)
    both(gpu_lib, big)


def test_offsets_past_32_bits(gpu_lib):
    """Pages whose elements lie more than 2^32 bytes and 2^31 elements in."""
    c = Case([(150, 3)], 4, 2, 128, 16, seed=18)
    small = run(gpu_lib, c)
    d = c.dev()
    pages = (1 << 31) // (16 * 2 * 128) + 4 * c.kc.shape[0]
    far = pages - c.kc.shape[0]
    for k in ("kc", "vc"):
        x = torch.empty((pages, 16, 2, 128), dtype=c.dtype, device="cuda")
        x[far:] = d[k]
        d[k] = x
    d["table"] = torch.where(d["table"] >= 0, d["table"] + far, d["table"])
    out, lse = run(gpu_lib, c, d=d)
    assert torch.equal(out, small[0]) and torch.equal(lse, small[1])
    # a write there
    plan = gpu_lib.PagedPlan(2, 2, 128, 16, c.dtype, max_rows=1)
    new = torch.randn((1, 2, 128), device="cuda").to(c.dtype)
    slot = torch.tensor([pages * 16 - 1], device="cuda")
    gpu_lib.markov_paged_write(plan, new, new, d["kc"], d["vc"], slot)
    assert torch.equal(d["kc"][-1, -1], new[0]) and torch.equal(d["vc"][-1, -1], new[0])
    plan.close()


def test_layout_write_attention_in_one_graph(gpu_lib):
    """The calls captured once, replayed as the requests grow."""
    api = gpu_lib
    R, hq, hkv, dd, page, n, width = 5, 8, 2, 64, 16, 3, 12
    plan = api.PagedPlan(hq, hkv, dd, page, torch.bfloat16, max_rows=R)
    g = torch.Generator(device="cuda").manual_seed(1)
    pages = R * width
    kc, vc = (torch.full((pages, page, hkv, dd), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
    held = torch.zeros(R, dtype=torch.int32, device="cuda")
    ring = torch.randperm(pages, generator=g, device="cuda").int()
    free = torch.tensor([0, pages], device="cuda")
    ctx = torch.zeros(R, dtype=torch.int32, device="cuda")
    ql = torch.full((R,), n, dtype=torch.int32, device="cuda")
    idx = torch.arange(R, device="cuda").flip(0)
    T = R * n
    key, val = (torch.zeros((T, hkv, dd), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros((T, hq, dd), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    lse = torch.zeros((T, hq), device="cuda")

    def step(s):
        start, lens, _, slots = api.markov_paged_layout(plan, ctx, ql, idx, table, held, ring, free, T, *bufs, stream=s)
        api.markov_paged_write(plan, key, val, kc, vc, slots, stream=s)
        api.markov_paged_attention(plan, q, kc, vc, table, idx, start, lens, out=out, lse=lse, stream=s)

    bufs = (torch.zeros(R + 1, dtype=torch.int32, device="cuda"), torch.zeros(R, dtype=torch.int32, device="cuda"),
            torch.zeros(T, dtype=torch.int32, device="cuda"), torch.zeros(T, dtype=torch.int64, device="cuda"))
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            step(s)
    hist_k = [[] for _ in range(R)]
    hist_v = [[] for _ in range(R)]
    for k in range(20):
        for t in (key, val, q):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert api.markov_paged_plan_status(plan) == 0
        for b in range(R):
            hist_k[b].append(key[b * n:(b + 1) * n].clone())
            hist_v[b].append(val[b * n:(b + 1) * n].clone())
        if k % 6 == 5:
            c = Case([(0, 1)], hq, hkv, dd, page)             # the same check on the graph's tensors
            c.T, c.q, c.kc, c.vc, c.table = T, q.cpu(), kc.cpu(), vc.cpu(), table.cpu()
            c.idx, c.start, c.lens = idx.cpu(), bufs[0].cpu(), bufs[1].cpu()
            for b in range(R):
                L = int(c.lens[b])
                i = torch.arange(L)
                pg = c.table[c.idx[b], i // page].long()
                assert torch.equal(c.kc[pg, i % page], torch.cat(hist_k[b]).cpu())
                assert torch.equal(c.vc[pg, i % page], torch.cat(hist_v[b]).cpu())
            check(c, out, lse)
        ctx += n
    assert int(free[1]) == pages - R * -(-60 // page)
    plan.close()


# ---------------------------------------------------------------- refusals

def test_refusals(gpu_lib):
    api = gpu_lib
    c = Case([(10, 2)], 4, 2, 64, 16)
    d = c.dev()
    plan = c.plan(api)

    def attend(**kw):
        a = dict(d, out=torch.full((2, 4, 64), SENT, dtype=c.dtype, device="cuda"), lse=None, window=0, sinks=0,
                 scale=None)
        a.update(kw)
        try:
            api.markov_paged_attention(plan, a["q"], a["kc"], a["vc"], a["table"], a["idx"], a["start"], a["lens"],
                                       scale=a["scale"], window=a["window"], sinks=a["sinks"], out=a["out"], lse=a["lse"])
        finally:
            torch.cuda.synchronize()
            assert a["out"] is a["q"] or bool((a["out"] == SENT).all())

    for kw, err in [(dict(q=d["q"].half()), TypeError), (dict(q=d["q"][:, :2]), ValueError),
                    (dict(q=d["q"].cpu()), TypeError), (dict(kc=d["kc"][:, :8]), ValueError),
                    (dict(kc=d["kc"][:-1]), api.MarkovError), (dict(idx=d["idx"].int()), TypeError),
                    (dict(start=d["start"][:1]), ValueError), (dict(lens=d["lens"].long()), TypeError),
                    (dict(table=d["table"][0]), ValueError), (dict(window=-1), api.MarkovError),
                    (dict(sinks=-2), api.MarkovError), (dict(scale=math.nan), api.MarkovError),
                    (dict(scale=math.inf), api.MarkovError), (dict(out=d["q"]), api.MarkovError),
                    (dict(lse=torch.zeros((2, 3), device="cuda")), ValueError),
                    (dict(idx=d["idx"].repeat(2), start=torch.zeros(3, dtype=torch.int32, device="cuda"),
                          lens=d["lens"].repeat(2)), api.MarkovError)]:
        with pytest.raises(err):
            attend(**kw)
    # a head stride that is no multiple of 16 bytes, and a base that is off
    odd = torch.zeros((2, 4, 68), dtype=c.dtype, device="cuda")[:, :, :64]
    with pytest.raises(api.MarkovError):
        attend(q=odd)
    off = torch.zeros(2 * 4 * 64 + 1, dtype=c.dtype, device="cuda")[1:].view(2, 4, 64)
    with pytest.raises(api.MarkovError):
        attend(q=off)
    with pytest.raises(ValueError):
        api.markov_paged_write(plan, d["kc"][0, :2], d["kc"][0, :3], d["kc"], d["vc"],
                               torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        api.markov_paged_layout(plan, d["lens"], d["lens"], d["idx"], d["table"], d["lens"].repeat(9), d["lens"],
                                torch.zeros(2, dtype=torch.int64, device="cuda"), 4)
    assert api.markov_paged_plan_status(plan) == 0
    plan.close()


@pytest.mark.parametrize("bad", [dict(q_heads=5), dict(q_heads=1), dict(q_heads=258), dict(q_heads=256, kv_heads=1), dict(kv_heads=0),
                                 dict(head_dim=96), dict(page_size=24), dict(page_size=4), dict(page_size=512),
                                 dict(max_rows=0), dict(max_rows=1025), dict(timeout_ms=-1)])
def test_plan_refusals(gpu_lib, bad):
    args = dict(q_heads=4, kv_heads=2, head_dim=64, page_size=16, max_rows=4)
    with pytest.raises(gpu_lib.MarkovError) as e:
        gpu_lib.PagedPlan(**dict(args, **bad))
    assert e.value.code == 1
    with pytest.raises(TypeError):
        gpu_lib.PagedPlan(**args, dtype=torch.float32)


def test_a_pending_status_stops_the_calls(gpu_lib):
    api = gpu_lib
    c = Case([(10, 2)], 4, 2, 64, 16)
    d = c.dev()
    plan = c.plan(api)
    api.markov_paged_plan_inject_status(plan, 4, 9)
    out = torch.full((2, 4, 64), SENT, dtype=c.dtype, device="cuda")
    api.markov_paged_attention(plan, d["q"], d["kc"], d["vc"], d["table"], d["idx"], d["start"], d["lens"], out=out)
    slots = torch.zeros(2, dtype=torch.int64, device="cuda")
    before = d["kc"].clone()
    api.markov_paged_write(plan, d["q"][:, :2], d["q"][:, :2], d["kc"], d["vc"], slots)
    torch.cuda.synchronize()
    assert bool((out == SENT).all()) and torch.equal(d["kc"].view(torch.int16), before.view(torch.int16))
    assert api.markov_paged_plan_status(plan) == 4
    assert api.markov_paged_plan_status(plan) == 0
    both(api, c)
    plan.close()
