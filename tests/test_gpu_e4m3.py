"""The e4m3 cache on the GPU against its plain 64-bit forms: stores that quantise,
reading back, attention over it."""
import math

import numpy as np
import pytest
import torch

from tests import serving_ref as ref

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
DT = [torch.bfloat16, torch.float16]
SENT = 123.0


def _bytes(shape, order, g, std=60.0):
    """A cache [pages, page, heads, d] of e4m3 in the given order."""
    pages, page, heads, d = shape
    x = torch.randn((pages, heads, page, d) if order == "hnd" else shape, generator=g) * std
    x = x.clamp(-448, 448).to(E4M3)
    return x.transpose(1, 2) if order == "hnd" else x


def _scales(pages, blocks, heads, g, lo=-9, hi=-4):
    return torch.exp2(torch.randint(lo, hi, (pages, blocks, heads), generator=g).float())


def _same(got, want):
    """Equal values of e4m3, NaN where NaN."""
    got, want = got.cpu().double(), want.double()
    assert torch.equal(got.isnan(), want.isnan())
    differ = (got != want) & ~got.isnan()
    assert not bool(differ.any()), (int(differ.sum()), differ.nonzero()[:5].tolist())


# ------------------------------------------------------------------- store

def _store(api, new, value, kc, vc, ks, vs, slots, keep=False, page=None, **kw):
    T, heads, d = new.shape
    dev = [x.cuda() for x in (kc, vc, ks, vs)]
    for x, y in zip(dev, (kc, vc, ks, vs)):
        assert x.stride() == y.stride()
    plan = api.PagedPlan(heads, heads, d, kc.shape[1], new.dtype, max_rows=1)
    api.markov_paged_write_e4m3(plan, new.cuda(), value.cuda(), *dev, slots.cuda(), keep_scales=keep, **kw)
    assert api.markov_paged_plan_status(plan) == 0
    plan.close()
    for x, cache, scales, c0, s0 in ((new, dev[0], dev[2], kc, ks), (value, dev[1], dev[3], vc, vs)):
        want, want_s = ref.store(x, c0, s0, slots, keep)
        _same(cache, want)
        got_s = scales.cpu().double()
        assert torch.equal(got_s[~want_s.isnan()], want_s[~want_s.isnan()])
    return dev


def _runs(page, pages, rng, rows, most):
    """Slots of `rows` requests that go on where their pages are filled so far."""
    perm, at, out = rng.permutation(pages), 0, []
    for _ in range(rows):
        c, n = int(rng.integers(0, 2 * page)), int(rng.integers(1, most + 1))
        need = -(-(c + n) // page)
        if at + need > pages:
            break
        mine = perm[at:at + need]
        at += need
        pos = np.arange(c, c + n)
        out.append(mine[pos // page] * page + pos % page)
    return torch.as_tensor(np.concatenate(out))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("heads,d,page,blocks,order,rows,most", [
    (1, 64, 16, 1, "nhd", 1, 1), (3, 128, 16, 1, "hnd", 8, 9), (8, 64, 64, 4, "nhd", 5, 40),
    (2, 128, 256, 1, "nhd", 2, 300), (5, 128, 32, 2, "hnd", 60, 100), (8, 128, 64, 1, "nhd", 4, 700),
    (2, 64, 256, 16, "hnd", 3, 500), (4, 128, 64, 1, "nhd", 700, 1), (8, 64, 32, 2, "hnd", 300, 9), (2, 128, 128, 1, "nhd", 1500, 3)])
def test_store(gpu_lib, dtype, heads, d, page, blocks, order, rows, most):
    rng = np.random.default_rng(page + rows)
    g = torch.Generator().manual_seed(page * rows)
    pages = rows * (most // page + 3) + 2
    slots = _runs(page, pages, rng, rows, most)
    T = len(slots)
    new, value = torch.randn((T, heads, d), generator=g) * 2, torch.randn((T, heads, d), generator=g)
    new[::3] *= torch.exp2(torch.randint(-6, 7, (len(new[::3]), heads, 1), generator=g).float())
    caches = [_bytes((pages, page, heads, d), order, g) for _ in range(2)]
    scales = [_scales(pages, blocks, heads, g) for _ in range(2)]
    _store(gpu_lib, new.to(dtype), value.to(dtype), *caches, *scales, slots)
    _store(gpu_lib, new.to(dtype), value.to(dtype), *caches, *scales, slots, keep=True)


@pytest.mark.parametrize("rows,most", [(3, 9), (300, 1), (2, 700)])
def test_store_blocks_of_keys_and_values_differ(gpu_lib, rows, most):
    rng = np.random.default_rng(rows)
    g = torch.Generator().manual_seed(rows)
    page, heads, d = 128, 8, 128
    pages = rows * (most // page + 3) + 2
    slots = _runs(page, pages, rng, rows, most)
    new, value = (torch.randn((len(slots), heads, d), generator=g).bfloat16() for _ in range(2))
    caches = [_bytes((pages, page, heads, d), "nhd", g) for _ in range(2)]
    for k, v in ((1, 8), (8, 1), (2, 4)):
        _store(gpu_lib, new, value, *caches, _scales(pages, k, heads, g), _scales(pages, v, heads, g), slots)


def test_store_skips_and_strides(gpu_lib):
    g = torch.Generator().manual_seed(2)
    heads, d, page, pages = 3, 64, 32, 6
    # requests of four tokens each, then skipped ones between them
    slots = torch.tensor([5, 6, 7, 8, -1, 64, 65, 66, 67, -1, -3, pages * page, 96 + 30, 96 + 31, 10 ** 12, 129, 130])
    wide = torch.randn((len(slots), 2 * heads + 1, d), generator=g).bfloat16()
    caches = [_bytes((pages, page, heads, d), "nhd", g) for _ in range(2)]
    # scales with the heads outermost
    scales = [_scales(pages, 2, heads, g).permute(2, 0, 1).contiguous().permute(1, 2, 0) for _ in range(2)]
    _store(gpu_lib, wide[:, :heads], wide[:, heads:2 * heads], *caches, *scales, slots)


@pytest.mark.parametrize("dtype", DT)
def test_store_growth_and_scales_that_are_none(gpu_lib, dtype):
    """A block's scale grows with its entries; zeros, NaN, infinities and the smallest values."""
    g = torch.Generator().manual_seed(3)
    heads, d, page, pages = 9, 64, 16, 4
    old = torch.tensor([2.0 ** -9, 2.0 ** -20, 2.0 ** -40, 0.0, math.nan, math.inf, -1.0, 0.003, 7.0])
    caches = [_bytes((pages, page, heads, d), "nhd", g) for _ in range(2)]
    caches[0].view(torch.uint8)[0, 3, :, 5] = 0x7F                         # NaN in the cache stays
    scales = [old.expand(pages, 1, heads).contiguous() for _ in range(2)]
    for slots in (torch.tensor([16, 17, 18]), torch.tensor([18, 19]), torch.tensor([31]), torch.tensor([15, 16])):
        T = len(slots)
        new, value = torch.randn((T, heads, d), generator=g).to(dtype), torch.randn((T, heads, d), generator=g).to(dtype)
        _store(gpu_lib, new, value, *caches, *scales, slots)
        value[:, 0], value[:, 1] = 0, torch.finfo(dtype).tiny
        value[0, 2, 3], value[0, 3, 4] = math.inf, -math.inf
        value[0, 4, 5], value[:, 5] = math.nan, math.nan
        value[:, 6], value[:, 7] = torch.finfo(dtype).max, math.inf
        _store(gpu_lib, new, value, *caches, *scales, slots)


def test_store_rounds_to_even_and_at_powers(gpu_lib):
    """Halves between two values of e4m3, and largest values at 448 times a power of two."""
    d, page = 64, 16
    x = torch.zeros((9, 1, d))
    grid = torch.arange(0, 0x7F, dtype=torch.uint8).view(E4M3).float()     # every value from 0 to 448
    mid = (grid[:-1] + grid[1:]) / 2
    x[0, 0], x[1, 0, :d - 2] = mid[:64], mid[64:]
    x[0, 0, -1] = 448
    x[1, 0, -2:] = -mid[100:102]
    x[2, 0, 0], x[3, 0, 0], x[4, 0, 0], x[5, 0, 0] = 7.0, 7.03125, 3.5, 448 * 2.0 ** -41
    x[6, 0, 0], x[7, 0, 0], x[8, 0, 0] = 28672.0, 2.0 ** -14, 6.96875
    caches = [torch.zeros((9, page, 1, d)).to(E4M3) for _ in range(2)]
    scales = [torch.ones((9, 1, 1)) for _ in range(2)]
    for dtype in DT:
        _store(gpu_lib, x.to(dtype), -x.to(dtype), *caches, *scales, torch.arange(9) * page)


def test_store_with_shared_scales(gpu_lib):
    """Calibrated scales, one for everything or one a head, not a power of two; values beyond them saturate."""
    api = gpu_lib
    g = torch.Generator().manual_seed(4)
    heads, d, page, pages = 4, 128, 64, 5
    new, value = torch.randn((150, heads, d), generator=g).half(), torch.randn((150, heads, d), generator=g).half() * 100
    slots = torch.randperm(pages * page, generator=g)[:150]                # any order
    caches = [_bytes((pages, page, heads, d), "nhd", g) for _ in range(2)]
    dev = [c.cuda() for c in caches]
    one, by_head = torch.tensor([0.01234], device="cuda"), torch.rand(heads, generator=g).cuda() * 0.01 + 0.001
    ks, vs = one.expand(pages, 1, heads), by_head.expand(pages, 4, heads)
    plan = api.PagedPlan(heads, heads, d, page, torch.float16, max_rows=1)
    api.markov_paged_write_e4m3(plan, new.cuda(), value.cuda(), *dev, ks, vs, slots.cuda(), keep_scales=True)
    for x, c, s, c0 in ((new, dev[0], ks, caches[0]), (value, dev[1], vs, caches[1])):
        _same(c, ref.store(x, c0, s.cpu(), slots, True)[0])
    with pytest.raises(api.MarkovError):                                   # nothing of their own to write
        api.markov_paged_write_e4m3(plan, new.cuda(), value.cuda(), *dev, ks, vs, slots.cuda())
    api.markov_paged_write_e4m3(plan, new.cuda()[:0], value.cuda()[:0], *dev, ks, vs, slots.cuda()[:0], keep_scales=True)
    plan.close()


def test_store_step_by_step_is_near_one_store(gpu_lib):
    """Token after token, as decoding stores, the values stay within a rounding of what they are."""
    api = gpu_lib
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((64, 2, 64), generator=g, device="cuda").bfloat16()
    plan = api.PagedPlan(2, 2, 64, 32, max_rows=1)
    caches = [torch.zeros((2, 32, 2, 64), dtype=E4M3, device="cuda") for _ in range(2)]
    scales = [torch.zeros((2, 2, 2), device="cuda") for _ in range(2)]
    slots = torch.arange(64, device="cuda")
    for t in range(64):
        api.markov_paged_write_e4m3(plan, x[t:t + 1], x[t:t + 1], *caches, *scales, slots[t:t + 1])
    got = ref.values_of(caches[0].cpu(), scales[0].cpu()).reshape(64, 2, 64)
    # scales are powers of two: a rescaled value is a rounding of 2^-4, and one of half the least
    # step of its block, 2^-10 of the scale, for each growth (four at most here: 2^-4 to 2^-8 of it)
    s = scales[0].cpu().double().repeat_interleave(16, 1).reshape(64, 2, 1)
    assert bool(((got - x.cpu().double()).abs() <= 2.0 ** -4 * x.cpu().double().abs() + 4 * 2.0 ** -10 * s).all())
    plan.close()


# ------------------------------------------------------------------ requests

class Case:
    """Requests of the given (context, new tokens), their keys and values in
    scattered pages of a cache that holds NaN, scales too, everywhere else."""

    def __init__(self, reqs, hq, hkv, d, page, block=16, dtype=torch.bfloat16, order="nhd", seed=0, padding=(),
                 width_extra=1, std=1.5, spread=(-9, -4)):
        g = torch.Generator().manual_seed(seed)
        self.page, self.block, self.dtype, self.hq, self.hkv, self.d = page, block, dtype, hq, hkv, d
        n, lens = [q for _, q in reqs], [c + q for c, q in reqs]
        need = [-(-max(L, 0) // page) for L in lens]
        pages, states = sum(need) + 5, len(reqs) + 2
        perm, idx = torch.randperm(pages, generator=g), torch.randperm(states, generator=g)[:len(reqs)]
        self.table = torch.full((states, max(need) + width_extra), -7, dtype=torch.int32)
        self.kc, self.vc = (_bytes((pages, page, hkv, d), order, g) for _ in range(2))
        seen = torch.zeros((pages, page), dtype=torch.bool)
        at = 0
        for b, L in enumerate(lens):
            mine = perm[at:at + need[b]]
            at += need[b]
            self.table[idx[b], :need[b]] = mine.int()
            i = torch.arange(max(L, 0))
            seen[mine[i // page], i % page] = True
        for c in (self.kc, self.vc):
            c.view(torch.uint8)[~seen] = 0x7F
        held = seen.view(pages, page // block, block).any(-1)
        self.ks, self.vs = (_scales(pages, page // block, hkv, g, *spread) for _ in range(2))
        for s in (self.ks, self.vs):
            s[~held] = math.nan
        self.T = sum(n)
        self.q = (torch.randn((self.T, hq, d), generator=g) * std).to(dtype)
        self.start = torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32)
        self.lens, self.idx = torch.tensor(lens, dtype=torch.int32), idx.clone()
        for b in padding:
            self.idx[b] = -1

    def dev(self):
        return {k: getattr(self, k).cuda() for k in ("q", "kc", "vc", "ks", "vs", "table", "idx", "start", "lens")}

    def plan(self, api):
        return api.PagedPlan(self.hq, self.hkv, self.d, self.page, self.dtype, max_rows=len(self.idx))


def run(api, case, scale=None, window=0, sinks=0, d=None, plan=None, **kw):
    d = d or case.dev()
    own = plan is None
    plan = plan or case.plan(api)
    out = torch.full((case.T, case.hq, case.d), SENT, dtype=case.dtype, device="cuda")
    lse = torch.full((case.T, case.hq), SENT, device="cuda")
    api.markov_paged_attention_e4m3(plan, d["q"], d["kc"], d["vc"], d["ks"], d["vs"], d["table"], d["idx"], d["start"],
                                    d["lens"], scale=scale, window=window, sinks=sinks, out=out, lse=lse, **kw)
    assert api.markov_paged_plan_status(plan) == 0
    if own:
        plan.close()
    return out, lse


def check(case, out, lse, scale=None, window=0, sinks=0):
    want, wl, tol, tl = ref.attention(case.q, case.kc, case.vc, case.ks, case.vs, case.table, case.idx, case.start,
                                      case.lens, case.d ** -0.5 if scale is None else scale, window, sinks)
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


# requests of one and of several row tiles, around an average of 128 query rows a request
_ROW_TILES = {
    "one tile each": [(3000, 16), (0, 1), (700, 9), (64, 16), (5000, 11)],
    "many rows, some alone": [(300, 100), (10, 1), (2000, 1), (0, 1), (129, 3), (127, 1), (40, 2), (900, 1)],
    "above the average": [(3000, 17), (100, 40), (1500, 33)],
    "a lone request of two tiles": [(9000, 32)],
    "a lone request of one tile": [(9000, 16)],
    "short ones": [(0, 16), (0, 5), (1, 12), (15, 16)],
}


@pytest.mark.parametrize("d,dtype,scale", [(128, torch.bfloat16, None), (128, torch.float16, -0.1), (64, torch.bfloat16, -0.2),
                                           (64, torch.float16, None)])
@pytest.mark.parametrize("reqs", list(_ROW_TILES.values()), ids=list(_ROW_TILES))
def test_row_tiles_of_an_item(gpu_lib, reqs, d, dtype, scale):
    both(gpu_lib, Case(reqs, 16, 2, d, 32, 16, dtype=dtype, seed=len(reqs)), scale=scale)


def test_padding_rows_change_the_row_tiles_of_an_item(gpu_lib):
    """40 tokens of 8 heads a request, alone and among rows of padding (no tokens)."""
    for pad in (0, 1, 5):
        reqs = [(500, 40), (2500, 40)] + [(0, 0)] * pad
        both(gpu_lib, Case(reqs, 16, 2, 128, 64, 32, seed=3, padding=tuple(range(2, 2 + pad))), window=700, sinks=5)


# ------------------------------------------------------------------- fetch

def _fetch(api, case, T=None, key=None, value=None):
    d = case.dev()
    T = case.T if T is None else T
    plan = case.plan(api)
    shape = (T, case.hkv, case.d)
    key = torch.full(shape, SENT, dtype=case.dtype, device="cuda") if key is None else key
    value = torch.full(shape, SENT, dtype=case.dtype, device="cuda") if value is None else value
    api.markov_paged_read_e4m3(plan, d["kc"], d["vc"], d["ks"], d["vs"], d["table"], d["idx"], d["start"], d["lens"], T,
                               key=key, value=value)
    assert api.markov_paged_plan_status(plan) == 0
    plan.close()
    pages = case.kc.shape[0]
    for got, cache, scales in ((key, case.kc, case.ks), (value, case.vc, case.vs)):
        v = ref.values_of(cache, scales)
        want = torch.full(shape, SENT, dtype=torch.float64)
        for b in range(len(case.idx)):
            n, L, s = int(case.start[b + 1] - case.start[b]), int(case.lens[b]), int(case.idx[b])
            for j in range(n):
                t, p = int(case.start[b]) + j, L - n + j
                if s < 0 or t >= T:
                    continue
                want[t] = 0
                if 0 <= p < case.table.shape[1] * case.page and s < case.table.shape[0]:
                    pid = int(case.table[s, p // case.page])
                    if 0 <= pid < pages:
                        want[t] = v[pid, p % case.page]
        # the product is exact in fp32 for a scale that is a power of two: one rounding
        assert torch.equal(got.cpu(), want.to(case.dtype))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("hkv,d,page,block,order,reqs", [
    (1, 64, 16, 16, "nhd", [(0, 1)]), (8, 128, 64, 32, "hnd", [(0, 100), (13, 7), (5, 0), (0, 250)]),
    (3, 64, 256, 128, "nhd", [(0, 1)] * 40), (5, 128, 128, 16, "hnd", [(3, 900), (0, 1500)])])
def test_fetch(gpu_lib, dtype, hkv, d, page, block, order, reqs):
    _fetch(gpu_lib, Case(reqs, hkv, hkv, d, page, block, dtype, order, seed=page))


def test_fetch_rows_that_are_not_there(gpu_lib):
    c = Case([(10, 4), (0, 9), (20, 0), (3, 3), (50, 6), (0, 0), (7, 2)], 4, 4, 64, 16, seed=6, padding=(3,), width_extra=0)
    c.lens[1] = 5                                             # four of nine before the start
    c.table[c.idx[0], 0] = c.kc.shape[0]                      # pages that are none
    c.table[c.idx[6], 0] = -1
    c.lens[4] += 100                                          # past the table
    _fetch(gpu_lib, c)
    _fetch(gpu_lib, c, T=c.T + 7)                             # tokens outside every row
    _fetch(gpu_lib, c, T=5)
    wide = torch.full((c.T, 9, 64), SENT, dtype=c.dtype, device="cuda")
    _fetch(gpu_lib, c, key=wide[:, :4], value=wide[:, 4:8])
    assert bool((wide[:, 8] == SENT).all())


def test_store_then_fetch(gpu_lib):
    """What was stored comes back, rounded to e4m3."""
    api = gpu_lib
    g = torch.Generator(device="cuda").manual_seed(8)
    plan = api.PagedPlan(4, 4, 128, 32, max_rows=2)
    x, y = (torch.randn((70, 4, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    caches = [torch.zeros((5, 32, 4, 128), dtype=E4M3, device="cuda") for _ in range(2)]
    scales = [torch.ones((5, 1, 4), device="cuda") for _ in range(2)]
    table = torch.tensor([[4, 0], [3, 1]], dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(40), torch.arange(30)]).cuda()
    row = torch.tensor([0] * 40 + [1] * 30, device="cuda")
    slots = table[row, pos // 32] * 32 + pos % 32
    api.markov_paged_write_e4m3(plan, x, y, *caches, *scales, slots.long())
    start, lens = torch.tensor([0, 40, 70], dtype=torch.int32, device="cuda"), torch.tensor([40, 30], dtype=torch.int32, device="cuda")
    k, v = api.markov_paged_read_e4m3(plan, *caches, *scales, table, torch.arange(2, device="cuda"), start, lens, 70)
    for got, want in ((k, x), (v, y)):
        # half a step of e4m3; below its normal range half the least step of a scale that is at most 2^-6 here
        assert bool(((got - want).abs().float() <= 2.0 ** -4 * want.abs().float() * 1.01 + 2.0 ** -16).all())
    plan.close()


# --------------------------------------------------------------- attention

@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 1), (8, 2), (6, 2), (21, 3), (40, 1), (16, 1), (5, 5), (128, 1)])
def test_single_tokens(gpu_lib, dtype, d, hq, hkv):
    reqs = [(0, 1), (1, 1), (14, 1), (15, 1), (16, 1), (126, 1), (127, 1), (128, 1), (300, 1), (1000, 1)]
    both(gpu_lib, Case(reqs, hq, hkv, d, 16, 16, dtype, seed=hq))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,block", [(16, 16), (32, 16), (32, 32), (64, 16), (64, 64), (128, 32), (128, 128), (256, 16), (256, 256)])
def test_draft_chunks_every_page_and_block(gpu_lib, dtype, d, page, block):
    reqs = [(0, 9), (3, 9), (page - 1, 2), (2 * page - 9, 9), (517, 9), (5, 17)]
    both(gpu_lib, Case(reqs, 8, 2, d, page, block, dtype, order="hnd" if block % 32 else "nhd", seed=page + block))
    # one token each, the same pages
    both(gpu_lib, Case([(c, 1) for c, _ in reqs], 8, 2, d, page, block, dtype, order="nhd" if block % 32 else "hnd", seed=page))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 257])
def test_chunk_lengths_around_tile_edges(gpu_lib, d, n):
    both(gpu_lib, Case([(0, n), (70, n)], 4, 2, d, 32, 16, seed=n))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 128), (7, 1, 64), (12, 4, 128)])
def test_long_chunks(gpu_lib, dtype, hq, hkv, d):
    both(gpu_lib, Case([(0, 400), (333, 150)], hq, hkv, d, 32, 32, dtype, seed=7))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 0), (7, 3), (64, 4), (128, 0), (128, 130),
                                          (200, 1), (5, 300), (10 ** 9, 4), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_windows_and_first_tokens(gpu_lib, window, sinks):
    reqs = [(0, 1), (0, 5), (6, 1), (250, 9), (600, 1), (500, 140), (129, 128)]
    both(gpu_lib, Case(reqs, 8, 2, 64, 16, seed=window % 1000), window=window, sinks=sinks)
    both(gpu_lib, Case(reqs[2:5], 4, 4, 128, 32, 16, torch.float16, seed=sinks % 1000), window=window, sinks=sinks)
    both(gpu_lib, Case([(c, 1) for c, _ in reqs], 8, 2, 128, 32, 32, seed=sinks % 1000), window=window, sinks=sinks)


def test_pages_before_the_window_are_not_read(gpu_lib):
    """Freed pages before the window: table entries gone, their keys and scales NaN."""
    for reqs in ([(700, 1), (650, 9)], [(700, 1), (658, 1)]):
        c = Case(reqs, 8, 2, 128, 16, seed=3)
        window, sinks = 100, 20
        for b, (_, n) in enumerate(reqs):
            L = int(c.lens[b])
            first = (L - n - window + 1) // 16                # the window's first page
            gone = c.table[c.idx[b], 2:first].long()
            for cache, scales in ((c.kc, c.ks), (c.vc, c.vs)):
                cache.view(torch.uint8)[gone] = 0x7F
                scales[gone] = math.nan
                # and in the pages at both edges, what nobody sees
                cache.view(torch.uint8)[c.table[c.idx[b], 1].long(), 4:] = 0x7F
                edge = L - n - window + 1
                if edge % 16:
                    cache.view(torch.uint8)[c.table[c.idx[b], first].long(), :edge % 16] = 0x7F
            c.table[c.idx[b], 2:first] = -1
        out, lse = run(gpu_lib, c, window=window, sinks=sinks)
        for x in (c.kc, c.vc):
            x.view(torch.uint8)[x.float().isnan()] = 0
        c.ks, c.vs = c.ks.nan_to_num(1.0), c.vs.nan_to_num(1.0)
        check(c, out, lse, window=window, sinks=sinks)


def test_keys_hidden_from_one_token_may_be_anything(gpu_lib):
    for n in (3, 40):
        c = Case([(40, n)], 4, 2, 64, 16, seed=5)
        page = int(c.table[c.idx[0], (40 + n - 1) // 16])
        d = c.dev()
        d["kc"].view(torch.uint8)[page, (40 + n - 1) % 16] = 0x7F
        out, lse = run(gpu_lib, c, d=d)
        clean, clean_lse = run(gpu_lib, c)
        assert torch.equal(out[:n - 1], clean[:n - 1]) and torch.equal(lse[:n - 1], clean_lse[:n - 1])


def test_rows_that_see_nothing(gpu_lib):
    """Refused rows (length 0), lengths below the chunk's, padding rows, rows without tokens."""
    for reqs in ([(10, 4), (0, 9), (20, 0), (3, 3), (50, 6)], [(10, 1), (0, 9), (20, 0), (3, 1), (50, 1)]):
        c = Case(reqs, 8, 4, 128, 16, seed=6, padding=(3,))
        c.lens[0] = 0                                         # refused
        c.lens[1] = 5                                         # four of nine before the start
        both(gpu_lib, c)
        both(gpu_lib, c, window=3, sinks=1)
    c = Case([(4, 1), (9, 1)], 8, 4, 128, 16, seed=6)
    c.idx[0] = c.table.shape[0] + 3                           # a state that there is not
    out, lse = run(gpu_lib, c)
    assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all())


def test_tokens_outside_every_row_are_left_alone(gpu_lib):
    for reqs in ([(10, 4), (0, 3)], [(10, 1), (0, 1), (3, 1), (40, 1), (70, 1), (2, 1), (9, 1)]):
        c = Case(reqs, 4, 4, 64, 16, seed=8)
        d = c.dev()
        d["q"] = torch.cat([d["q"], d["q"][:5]])
        plan = c.plan(gpu_lib)
        out = torch.full((c.T + 5, c.hq, c.d), SENT, dtype=c.dtype, device="cuda")
        args = (d["kc"], d["vc"], d["ks"], d["vs"], d["table"], d["idx"], d["start"], d["lens"])
        gpu_lib.markov_paged_attention_e4m3(plan, d["q"], *args, out=out)
        want, _ = run(gpu_lib, c)
        assert torch.equal(out[:c.T], want) and bool((out[c.T:] == SENT).all())
        plan.close()
        c.T, c.q = 5, c.q[:5]                                 # rows past the tokens that there are
        both(gpu_lib, c)


def test_length_past_the_table_and_pages_that_are_none(gpu_lib):
    for n in (4, 1):
        c = Case([(64 - n, n), (40, n)], 4, 2, 64, 16, seed=9, width_extra=0)
        c.lens[0] = 200
        c.table[c.idx[1], 1] = c.kc.shape[0] + 4              # zeros
        c.table[c.idx[1], 0] = -1
        both(gpu_lib, c)


def test_scales_of_any_kind(gpu_lib):
    """Scales that are no powers of two, far apart, 0 for a block of zeros, negative query scales."""
    for reqs in ([(200, 9), (77, 30)], [(200, 1), (777, 1)]):
        for dtype in DT:
            c = Case(reqs, 8, 2, 128, 64, 16, dtype, seed=11, spread=(-20, -3))
            both(gpu_lib, c)
            both(gpu_lib, c, scale=-0.05)
            both(gpu_lib, c, scale=0.0)
            g = torch.Generator().manual_seed(3)
            for s in (c.ks, c.vs):
                s *= torch.rand(s.shape, generator=g) + 0.5
            both(gpu_lib, c)
            # a block of zeros whose scale is 0, as max / 448 gives
            p = int(c.table[c.idx[0], 1])
            c.vc.view(torch.uint8)[p, 16:32], c.kc.view(torch.uint8)[p, :16] = 0, 0
            c.vs[p, 1], c.ks[p, 0] = 0.0, 0.0
            both(gpu_lib, c)


def test_large_and_small_queries(gpu_lib):
    """Rows of queries whose sizes differ by many powers of two, scores that fill the range."""
    for reqs in ([(150, 20)], [(150, 1), (30, 1)]):
        c = Case(reqs, 8, 2, 64, 32, 32, seed=12)
        f = torch.exp2(torch.linspace(-120, 10, c.T * 8)).view(c.T, 8, 1)
        c.q = (c.q.float() * f).to(torch.bfloat16)
        both(gpu_lib, c)
        both(gpu_lib, c, scale=1.0)


def test_one_key_is_its_value(gpu_lib):
    """A token that sees one key returns the value, exactly."""
    c = Case([(0, 1), (0, 1)], 8, 2, 128, 16, seed=13)
    out, lse = run(gpu_lib, c)
    v = ref.values_of(c.vc, c.vs)
    for b in range(2):
        want = v[int(c.table[c.idx[b], 0]), 0].repeat_interleave(4, 0)
        assert torch.equal(out[b].cpu(), want.to(torch.bfloat16))


def test_shared_scales_strides_streams_and_graphs(gpu_lib):
    api = gpu_lib
    for reqs in ([(300, 5), (9, 5), (1000, 5)], [(300, 1), (9, 1), (1000, 1)]):
        c = Case(reqs, 8, 2, 128, 64, 64, seed=14)
        d = c.dev()
        pages = c.kc.shape[0]
        d["ks"], d["vs"] = torch.tensor([0.0123], device="cuda").expand(pages, 4, 2), torch.tensor([0.3, 0.02], device="cuda").expand(pages, 1, 2)
        c.ks, c.vs = d["ks"].cpu().contiguous(), d["vs"].cpu().contiguous()
        out, lse = run(api, c, d=d)
        check(c, out, lse)
        # queries as a slice of a projection, outputs with the heads outermost
        wide = torch.zeros((c.T, 12, 128), dtype=c.dtype, device="cuda")
        wide[:, :8] = d["q"]
        plan = c.plan(api)
        heads_first = torch.zeros((8, c.T, 128), dtype=c.dtype, device="cuda").transpose(0, 1)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        args = (d["kc"], d["vc"], d["ks"], d["vs"], d["table"], d["idx"], d["start"], d["lens"])
        api.markov_paged_attention_e4m3(plan, wide[:, :8], *args, out=heads_first, stream=side)
        got, _ = api.markov_paged_attention_e4m3(plan, wide[:, :8], *args, stream=side)
        side.synchronize()
        assert torch.equal(heads_first, out) and torch.equal(got, out)
        graph = torch.cuda.CUDAGraph()
        y = torch.zeros_like(out)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            api.markov_paged_attention_e4m3(plan, d["q"], *args, out=y)
        d["lens"].sub_(1)                                      # a captured call follows the lengths
        c.lens -= 1
        graph.replay()
        torch.cuda.synchronize()
        want, _ = run(api, c, d=d)
        assert torch.equal(y, want)
        plan.close()


@pytest.mark.parametrize("hq,hkv,rows,hi", [(8, 8, 300, 400), (64, 8, 40, 3000), (4, 1, 1000, 60), (8, 1, 2, 60000)])
def test_many_rows_and_long_ones(gpu_lib, hq, hkv, rows, hi):
    """Work that is cut between many workers; the plain form on the GPU."""
    rng = np.random.default_rng(rows)
    for n in (1, 7):
        reqs = [(int(x), n if b % 3 else 1) for b, x in enumerate(np.exp(rng.uniform(0, np.log(hi), rows)))]
        reqs[0] = (hi, n)
        c = Case(reqs, hq, hkv, 64, 32, 32, seed=rows)
        d = c.dev()
        out, lse = run(gpu_lib, c, d=d)
        sample = rng.permutation(rows)[:12].tolist() + [0]
        keep = torch.zeros(rows, dtype=torch.bool)
        keep[sample] = True
        idx = torch.where(keep, c.idx, -1)
        want, wl, tol, tl = ref.attention(d["q"], d["kc"], d["vc"], d["ks"], d["vs"], d["table"], idx, c.start, c.lens, 64 ** -0.5, 0, 0)
        live = ~wl.isnan()
        assert int(live.sum()) >= min(12, rows) * hq
        assert float(((out.double() - want).abs() - tol)[live].max()) <= 0
        assert float(((lse.double() - wl).abs() - tl)[live].max()) <= 0


def test_two_plans_at_once(gpu_lib):
    """Calls that may overlap, each on a plan and a stream of its own."""
    api = gpu_lib
    for reqs in ([(3000, 1)] * 20, [(700, 60)] * 5):
        cases = [Case(reqs, 8, 2, 128, 64, 32, seed=s) for s in (21, 22)]
        want = [run(api, c) for c in cases]
        plans, devs = [c.plan(api) for c in cases], [c.dev() for c in cases]
        streams = [torch.cuda.Stream() for _ in cases]
        torch.cuda.synchronize()
        got = []
        for _ in range(5):
            for plan, d, s in zip(plans, devs, streams):
                got.append(api.markov_paged_attention_e4m3(plan, d["q"], d["kc"], d["vc"], d["ks"], d["vs"], d["table"], d["idx"],
                                                           d["start"], d["lens"], lse=True, stream=s))
        torch.cuda.synchronize()
        for i, (out, lse) in enumerate(got):
            assert torch.equal(out, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])
        for p in plans:
            assert api.markov_paged_plan_status(p) == 0
            p.close()


def test_a_pending_status_computes_nothing(gpu_lib):
    api = gpu_lib
    c = Case([(30, 1), (40, 1)], 4, 2, 64, 16, seed=15)
    d, plan = c.dev(), c.plan(api)
    api.markov_paged_plan_inject_status(plan, 4)
    out = torch.full((c.T, c.hq, c.d), SENT, dtype=c.dtype, device="cuda")
    args = (d["kc"], d["vc"], d["ks"], d["vs"], d["table"], d["idx"], d["start"], d["lens"])
    api.markov_paged_attention_e4m3(plan, d["q"], *args, out=out)
    key, value = api.markov_paged_read_e4m3(plan, *args, 2, key=torch.full((2, 2, 64), SENT, dtype=c.dtype, device="cuda"),
                                            value=torch.full((2, 2, 64), SENT, dtype=c.dtype, device="cuda"))
    before = d["kc"].clone().view(torch.uint8)
    api.markov_paged_write_e4m3(plan, key, value, *args[:4], torch.arange(2, device="cuda"))
    assert api.markov_paged_plan_status(plan) == 4
    for x in (out, key, value):
        assert bool((x == SENT).all())
    assert torch.equal(d["kc"].view(torch.uint8), before)
    assert torch.equal(run(api, c, d=d, plan=plan)[0], run(api, c, d=d)[0])
    plan.close()


def test_refusals(gpu_lib):
    api = gpu_lib
    c = Case([(30, 2)], 4, 2, 64, 32, 16, seed=16)
    d, plan = c.dev(), c.plan(api)
    rest = (d["table"], d["idx"], d["start"], d["lens"])
    call = lambda q=d["q"], kc=d["kc"], ks=d["ks"], **kw: api.markov_paged_attention_e4m3(  # noqa: E731
        plan, q, kc, d["vc"], ks, d["vs"], *rest, **kw)
    call()
    for bad in (dict(q=d["q"].float()), dict(kc=d["kc"].view(torch.uint8)), dict(ks=d["ks"].half())):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in (dict(q=d["q"][:, :3]), dict(kc=d["kc"][:, :16]), dict(ks=d["ks"][:, :, :1]), dict(ks=d["ks"][:-1]),
                dict(ks=torch.ones((c.kc.shape[0], 3, 2), device="cuda"))):
        with pytest.raises(ValueError):
            call(**bad)
    # blocks of 8 tokens, windows below 0, scales that are not finite, queries as the output
    for bad in (dict(ks=torch.ones((c.kc.shape[0], 4, 2), device="cuda")), dict(window=-1), dict(sinks=-1),
                dict(scale=math.inf), dict(out=d["q"])):
        with pytest.raises(api.MarkovError):
            call(**bad)
    small = api.PagedPlan(4, 2, 64, 8, max_rows=1)               # pages of 8 slots have no block of 16
    with pytest.raises(api.MarkovError):
        api.markov_paged_attention_e4m3(small, d["q"], d["kc"].view(-1, 8, 2, 64), d["vc"].view(-1, 8, 2, 64),
                                        d["ks"][:, :1].repeat_interleave(4, 0), d["vs"][:, :1].repeat_interleave(4, 0), *rest)
    small.close()
    with pytest.raises(ValueError):
        api.markov_paged_read_e4m3(plan, d["kc"], d["vc"], d["ks"], d["vs"], *rest, 3, key=d["q"][:, :2])
    plan.close()


@pytest.mark.parametrize("reqs,hq,hkv", [([(16000, 1)], 8, 1), ([(9000, 2)], 8, 8), ([(7000, 1), (30, 1), (0, 1)], 16, 2)])
def test_long_items_of_few_rows_are_cut_into_few_parts(gpu_lib, reqs, hq, hkv):
    """An item's parts are fewer than the warps there are: by the root of its length."""
    for d in (64, 128):
        both(gpu_lib, Case(reqs, hq, hkv, d, 64, 64, seed=hq))
