"""Shared prefixes, chosen pages and eviction over the paged cache against their plain
64-bit forms (GPU)."""
import math
import os
import sys

import pytest
import torch

import mixture_experts_gb300 as moe

sys.path.insert(0, os.path.dirname(__file__))
import attn_ref  # noqa: E402
import context_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    moe.build()
    assert torch.cuda.is_available()


@pytest.fixture(autouse=True)
def clean_status():
    assert moe.coli_device_status() == moe.COLI_OK
    yield
    assert moe.coli_device_status() == moe.COLI_OK


def queries(g, B, hq, D, fmt):
    """Queries as a slice of a wider row."""
    wide = torch.randn(B, (hq + 2) * D, generator=g).to(ref.act(fmt)).cuda()
    return wide[:, :hq * D].unflatten(-1, (hq, D))


def out_step(fmt):
    return 2.0 ** -24 if fmt == "f32" else 2.0 ** -8


# ---- shared prefix -------------------------------------------------------------------------
SHARED = [  # fmt, B, hq, hk, D, page, prefix, own
    ("bf16", 1, 4, 4, 64, 16, 1, [1]),
    ("bf16", 3, 8, 2, 128, 16, 100, [0, 1, 40]),
    ("bf16", 5, 20, 4, 80, 48, 777, [3, 0, 99, 48, 17]),
    ("bf16", 40, 8, 1, 128, 64, 1500, [7 * b % 61 for b in range(40)]),
    ("bf16", 33, 16, 2, 64, 32, 2049, [1] * 33),
    ("bf16", 70, 10, 2, 256, 16, 700, [b % 5 for b in range(70)]),
    ("bf16", 17, 16, 2, 8, 16, 129, [0] * 17),
    ("bf16", 130, 4, 4, 96, 16, 1027, [b % 40 for b in range(130)]),
    ("f32", 5, 20, 4, 80, 48, 777, [0, 99, 3, 20, 50]),
    ("f32", 24, 8, 2, 128, 16, 333, [b for b in range(24)]),
    ("mxfp8", 4, 16, 2, 128, 32, 500, [0, 1, 33, 90]),
    ("mxfp8", 64, 8, 2, 128, 64, 1999, [b % 50 for b in range(64)]),
    ("mxfp8", 50, 8, 2, 96, 16, 801, [b % 7 for b in range(50)]),
    ("mxfp8", 33, 8, 1, 256, 16, 401, [b % 9 for b in range(33)]),
    ("mxfp4", 6, 32, 2, 64, 16, 320, [5, 0, 16, 17, 1, 31]),
    ("mxfp4", 48, 16, 2, 128, 32, 1300, [b for b in range(48)]),
    ("mxfp4", 30, 12, 2, 32, 128, 901, [b for b in range(30)]),
    # several tiles a block, blocks that end one key head's tiles and begin the next one's
    ("bf16", 20, 32, 16, 64, 16, 3100, [b % 4 for b in range(20)]),
    ("bf16", 160, 32, 16, 32, 48, 1400, [1] * 160),
    ("mxfp8", 80, 32, 8, 64, 16, 3050, [b % 3 for b in range(80)]),
    ("mxfp4", 33, 32, 32, 64, 64, 2000, [b % 3 for b in range(33)]),
    # heads above 128, whose values two segments share
    ("bf16", 20, 16, 8, 160, 16, 3100, [b % 4 for b in range(20)]),
    ("bf16", 160, 16, 8, 256, 48, 1400, [1] * 160),
    ("bf16", 33, 6, 6, 136, 64, 1999, [b % 3 for b in range(33)]),
    ("bf16", 20, 100, 100, 192, 16, 140, [0] * 20),
    # more segments than blocks
    ("bf16", 20, 200, 200, 16, 16, 100, [0] * 20),
    ("mxfp8", 150, 200, 200, 32, 16, 130, [b % 2 for b in range(150)]),
]


@pytest.mark.parametrize("fmt,B,hq,hk,D,page,prefix,own", SHARED)
def test_shared_prefix(fmt, B, hq, hk, D, page, prefix, own):
    g = ref.gen(B, hq, D, prefix)
    n_pre = -(-prefix // page)
    n_pages = n_pre + sum(-(-n // page) for n in own) + 2
    cache, k, v = ref.pool(g, fmt, n_pages, page, hk, D)
    pre = torch.randperm(n_pages, generator=g)[:n_pre].int()
    table = ref.tables(g, own, page, n_pages, pre.tolist())
    q = queries(g, B, hq, D, fmt)
    lens = torch.tensor(own, dtype=torch.int32)
    scale = 1.3 * D ** -0.5

    def both(rows):
        return lambda b, h: torch.cat([ref.context(rows, pre.tolist(), h, prefix),
                                       ref.context(rows, table[b].tolist(), h, own[b])])

    want, want_lse, tol, tol_lse = attn_ref.attend(q, both(k), both(v), [prefix + n for n in own],
                                                   hk, scale)
    out, lse = cache.attend_shared(q, pre.cuda(), prefix, table.cuda(), lens.cuda(), scale=scale,
                                   return_lse=True)
    assert out.dtype == q.dtype
    tol = tol * (1 + out_step(fmt)) + out_step(fmt) * want.abs()
    assert ((out.cpu().double() - want).abs() <= tol).all()
    assert ((lse.cpu().double() - want_lse).abs() <= tol_lse).all()
    again, lse2 = cache.attend_shared(q, pre.cuda(), prefix, table.cuda(), lens.cuda(),
                                      scale=scale, return_lse=True)
    assert torch.equal(again, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "f32"])
def test_shared_without_prefix_is_attend(fmt):
    g = ref.gen(5)
    own = [0, 3, 200, 64]
    cache, k, v = ref.pool(g, fmt, 24, 16, 2, 64)
    table = ref.tables(g, own, 16, 24).cuda()
    q = queries(g, 4, 8, 64, fmt)
    lens = torch.tensor(own, dtype=torch.int32).cuda()
    a, la = cache.attend(q, table, lens, return_lse=True)
    b, lb = cache.attend_shared(q, None, 0, table, lens, return_lse=True)
    # the same means, rounded once each; an empty sequence: zeros, -inf
    assert torch.equal(a, b) and torch.equal(la, lb)
    assert not b[0].any() and (lb[0] == -math.inf).all()


def test_shared_prefix_of_left_out_pages():
    g = ref.gen(6)
    cache, k, v = ref.pool(g, "bf16", 40, 16, 1, 64)
    q = queries(g, 30, 4, 64, "bf16")
    pre = torch.tensor([3, -1, 7, 40, 9], dtype=torch.int32)
    table = torch.full((30, 1), -1, dtype=torch.int32)
    lens = torch.zeros(30, dtype=torch.int32)
    out, lse = cache.attend_shared(q, pre.cuda(), 75, table.cuda(), lens.cuda(), return_lse=True)
    assert moe.coli_device_status() == moe.COLI_EDEVICE
    rows = [torch.cat([x[3, 0], x[7, 0], x[9, 0, :11]]) for x in (k, v)]
    want, wl, tol, tl = attn_ref.attend(q, lambda b, h: rows[0], lambda b, h: rows[1], [43] * 30, 1,
                                        64 ** -0.5)
    assert ((out.cpu().double() - want).abs() <= tol + 2.0 ** -8 * want.abs()).all()
    assert ((lse.cpu().double() - wl).abs() <= tl).all()
    # nothing in sight at all
    bad = torch.full((5,), -1, dtype=torch.int32).cuda()
    out, lse = cache.attend_shared(q, bad, 75, table.cuda(), lens.cuda(), return_lse=True)
    assert moe.coli_device_status() == moe.COLI_EDEVICE
    assert not out.any() and (lse == -math.inf).all()


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_shared_prefix_ends_inside_a_page(fmt):
    # what lies behind the prefix in its last page, NaN included, has no influence
    g = ref.gen(8)
    cache, k, v = ref.pool(g, fmt, 60, 32, 2, 128)
    q = queries(g, 32, 8, 128, fmt)
    pre = torch.arange(50, dtype=torch.int32).cuda()
    table = torch.full((32, 1), -1, dtype=torch.int32).cuda()
    lens = torch.zeros(32, dtype=torch.int32).cuda()
    n = 49 * 32 + 5
    a = cache.attend_shared(q, pre, n, table, lens)
    if fmt == "bf16":
        cache.k[49, :, 5:], cache.v[49, :, 5:] = math.nan, math.inf
    else:
        cache.k[49, :, 5:], cache.v[49, :, 5:] = 127, 255
        cache.k_scale[49, :, 5:], cache.v_scale[49, :, 5:] = 255, 254
    assert torch.equal(cache.attend_shared(q, pre, n, table, lens), a)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_shared_prefix_of_large_scores_and_values(fmt):
    # scores up to thousands apart; values whose plain sums stay finite
    g = ref.gen(9)
    cache, k, v = ref.pool(g, fmt, 40, 32, 1, 128)
    q = queries(g, 40, 4, 128, fmt)
    pre = torch.arange(40, dtype=torch.int32).cuda()
    table = torch.full((40, 1), -1, dtype=torch.int32).cuda()
    lens = torch.zeros(40, dtype=torch.int32).cuda()
    for scale in (50.0, -50.0, 0.0):
        out, lse = cache.attend_shared(q, pre, 1280, table, lens, scale=scale, return_lse=True)
        rows = [ref.context(x, list(range(40)), 0, 1280) for x in (k, v)]
        want, wl, tol, tl = attn_ref.attend(q, lambda b, h: rows[0], lambda b, h: rows[1],
                                            [1280] * 40, 1, scale)
        # a weight below 2^-126, the least normal fp32 number, may count as 0: the 1280 of them
        # are worth 2^-126 sum |v| at most (e^-126 here is 2^-181, an output of 1e-57)
        tol = tol + 2.0 ** -126 * rows[1].abs().sum(0)
        assert ((out.cpu().double() - want).abs() <= tol + 2.0 ** -8 * want.abs()).all()
        assert ((lse.cpu().double() - wl).abs() <= tl).all()
    if fmt == "bf16":
        cache.v.copy_(cache.v.sign() * 2e35)
        out = cache.attend_shared(q, pre, 1280, table, lens)
        assert torch.isfinite(out).all()


# ---- bounds and choice of pages ------------------------------------------------------------
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-45])
@pytest.mark.parametrize("fmt,B,D", [("bf16", 40, 128), ("bf16", 80, 128), ("bf16", 40, 192),
                                     ("bf16", 1, 64), ("mxfp8", 80, 64), ("f32", 40, 64)])
def test_shared_prefix_without_scale(fmt, B, D, scale):
    # every token in sight weighs the same, what is behind the prefix in its last tile nothing
    g = ref.gen(B, D)
    cache, k, v = ref.pool(g, fmt, 40, 16, 1, D)
    q = queries(g, B, 4, D, fmt)
    pre = torch.arange(40, dtype=torch.int32)
    table = torch.full((B, 1), -1, dtype=torch.int32).cuda()
    lens = torch.zeros(B, dtype=torch.int32).cuda()
    for n in (601, 130, 7):
        rows = [ref.context(x, pre.tolist(), 0, n) for x in (k, v)]
        want, wl, tol, tl = attn_ref.attend(q, lambda b, h: rows[0], lambda b, h: rows[1], [n] * B,
                                            1, scale)
        out, lse = cache.attend_shared(q, pre.cuda(), n, table, lens, scale=scale, return_lse=True)
        tol = tol * (1 + out_step(fmt)) + out_step(fmt) * want.abs()
        assert ((out.cpu().double() - want).abs() <= tol).all()
        assert ((lse.cpu().double() - wl).abs() <= tl).all()


@pytest.mark.parametrize("fmt", list(ref.FMT))
@pytest.mark.parametrize("page,hk,D", [(16, 1, 8), (16, 2, 64), (48, 3, 80), (64, 2, 128),
                                       (32, 1, 256), (128, 2, 96), (16, 4, 32)])
def test_page_bounds(fmt, page, hk, D):
    if fmt in attn_ref.EMAX and D % 32:
        pytest.skip("MX heads are multiples of 32")
    g = ref.gen(page, hk, D)
    cache, k, _ = ref.pool(g, fmt, 9, page, hk, D)
    pages = torch.tensor([4, 0, 8, -1, 2, 7], dtype=torch.int32)
    fills = torch.tensor([page, 1, page - 1, 5, page // 2 + 1, 2], dtype=torch.int32)
    box = cache.new_bounds().fill_(7)
    cache.page_bounds(box, pages.cuda(), fills.cuda())
    want = torch.full(box.shape, 7.0, dtype=torch.float64)
    for p, f in zip(pages.tolist(), fills.tolist()):
        for h in range(hk):
            if p >= 0:
                want[p, h] = ref.bounds(k, p, h, f)
    assert torch.equal(box.cpu().double(), want)     # they are stored numbers: exact


def test_page_bounds_of_nan_and_bad_pages():
    g = ref.gen(1)
    cache, k, _ = ref.pool(g, "bf16", 4, 16, 2, 64)
    cache.k[1, 0, 3, 5] = math.nan
    cache.k[1, 1, 3, 5] = math.inf
    cache.k[2, 0, 9, 1] = math.nan                   # behind the page's fill
    box = cache.new_bounds()
    cache.page_bounds(box, torch.tensor([1, 2], dtype=torch.int32).cuda(),
                      torch.tensor([16, 9], dtype=torch.int32).cuda())
    assert torch.isnan(box[1, 0, :, 5]).all() and torch.isnan(box).sum() == 2
    assert box[1, 1, 1, 5] == math.inf and torch.isfinite(box[1, 1, 0, 5])
    assert moe.coli_device_status() == moe.COLI_OK
    for page, fill in ((4, 3), (-2, 3), (0, 0), (0, 17)):
        was = box.clone()
        cache.page_bounds(box, torch.tensor([page], dtype=torch.int32).cuda(),
                          torch.tensor([fill], dtype=torch.int32).cuda())
        assert moe.coli_device_status() == moe.COLI_EDEVICE
        assert torch.equal(box.nan_to_num(), was.nan_to_num())


SELECT = [  # fmt, B, hq, hk, D, page, lens, keep, first, last
    ("bf16", 1, 4, 4, 64, 16, [700], 5, 1, 2),
    ("bf16", 4, 16, 2, 128, 16, [0, 1, 900, 3000], 8, 1, 1),
    ("bf16", 3, 20, 4, 80, 48, [4000, 47, 480], 7, 0, 3),
    ("bf16", 2, 40, 2, 256, 16, [900, 640], 12, 2, 4),
    ("f32", 3, 6, 2, 80, 16, [1000, 333, 16], 9, 1, 1),
    ("f32", 1, 12, 1, 256, 16, [555], 3, 0, 1),
    ("mxfp8", 3, 8, 2, 128, 32, [2000, 64, 3001], 11, 1, 2),
    ("mxfp8", 1, 9, 1, 96, 64, [6400], 20, 3, 1),
    ("mxfp4", 2, 32, 2, 64, 16, [1600, 100], 6, 1, 1),
    ("bf16", 2, 8, 1, 128, 16, [40000, 33000], 40, 1, 2),
    ("bf16", 2, 8, 1, 64, 16, [500, 300], 3, 1, 2),      # nothing left to choose
]


@pytest.mark.parametrize("fmt,B,hq,hk,D,page,lens,keep,first,last", SELECT)
def test_select_and_attend(fmt, B, hq, hk, D, page, lens, keep, first, last):
    g = ref.gen(B, hq, D, keep)
    n_pages = sum(-(-n // page) for n in lens) + 2
    cache, k, v = ref.pool(g, fmt, n_pages, page, hk, D)
    table = ref.tables(g, lens, page, n_pages)
    q = queries(g, B, hq, D, fmt)
    box = torch.zeros(n_pages, hk, 2, D, dtype=torch.float64)
    fills = {}
    for b, n in enumerate(lens):
        for i in range(-(-n // page)):
            fills[int(table[b, i])] = min(page, n - i * page)
    bounds = cache.new_bounds()
    cache.page_bounds(bounds, torch.tensor(list(fills), dtype=torch.int32).cuda(),
                      torch.tensor(list(fills.values()), dtype=torch.int32).cuda())
    pages, held = cache.select_pages(q, bounds, table.cuda(), torch.tensor(
        lens, dtype=torch.int32).cuda(), keep, first=first, last=last)
    G = hq // hk
    qd, box = q.double().cpu(), bounds.double().cpu()
    want = torch.full((B, hk, keep), -1, dtype=torch.int32)
    seen = []
    for b, n in enumerate(lens):
        count = -(-n // page)
        seen.append(n - max(0, count - keep) * page)
        for h in range(hk):
            s = [ref.score(qd[b, h * G:(h + 1) * G], box[int(p), h]) for p in table[b, :count]]
            for r, j in enumerate(ref.largest(s, keep, first, last)):
                want[b, h, r] = table[b, j]
    assert torch.equal(pages.cpu(), want) and held.tolist() == seen
    out, lse = cache.attend_selected(q, pages, held, return_lse=True)

    def of(rows):
        return lambda b, h: ref.context(rows, want[b, h].tolist(), h, seen[b])

    o, l, tol, tol_l = attn_ref.attend(q, of(k), of(v), seen, hk, D ** -0.5)
    assert ((out.cpu().double() - o).abs() <= tol * (1 + out_step(fmt)) +
            out_step(fmt) * o.abs()).all()
    assert ((lse.cpu().double() - l).abs() <= tol_l)[torch.isfinite(l)].all()
    assert torch.equal(torch.isfinite(lse.cpu()), torch.isfinite(l))


@pytest.mark.parametrize("fmt", ["bf16", "f32"])
def test_select_near_ties_by_exact_scores(fmt):
    # pages whose bounds differ in one channel by the last place: fp32 sums cannot rank
    # them, exact ones can; and a run of equal pages, of which the earlier are taken
    g = ref.gen(77)
    page, D, n = 16, 128, 300
    cache, _, _ = ref.pool(g, fmt, n, page, 1, D)
    q = (torch.randn(1, 2, D, generator=g) * 100).to(ref.act(fmt)).cuda()
    q[0, 0, 0], q[0, 1, 0] = 2.0 ** -12, 2.0 ** -12
    bounds = cache.new_bounds()
    base = torch.randn(2, D, generator=g).sort(0).values.to(ref.act(fmt)).cuda()
    bounds[:, 0] = base
    pick = torch.randperm(n - 1, generator=g)[:150]
    step = torch.arange(1, 151, device="cuda")
    bounds[pick.cuda(), 0, 1, 0] = (1 + step / 256).to(bounds.dtype) * 4
    bounds[pick.cuda(), 0, 0, 0] = -1
    table = torch.randperm(n, generator=g).int().cuda()[None]
    lens = torch.tensor([n * page], dtype=torch.int32).cuda()
    for keep in (2, 40, 151, 220, 299):
        got, _ = cache.select_pages(q, bounds, table, lens, keep, first=0, last=1)
        box, qd = bounds.double().cpu(), q.double().cpu()
        s = [math.fsum(x) for x in ([float(a) * float(hi if a > 0 else lo) for a, lo, hi in zip(
            qd[0, 0], box[p, 0, 0], box[p, 0, 1])] for p in table[0].tolist())]
        t = [math.fsum(x) for x in ([float(a) * float(hi if a > 0 else lo) for a, lo, hi in zip(
            qd[0, 1], box[p, 0, 0], box[p, 0, 1])] for p in table[0].tolist())]
        want = [int(table[0, j]) for j in ref.largest([max(a, b) for a, b in zip(s, t)], keep, 0,
                                                      1)]
        assert got[0, 0].tolist() == want


def test_select_of_zero_queries_and_odd_bounds():
    g = ref.gen(78)
    cache, _, _ = ref.pool(g, "bf16", 64, 16, 2, 64)
    bounds = cache.new_bounds().normal_(generator=torch.Generator("cuda").manual_seed(3))
    table = torch.randperm(64, generator=g).int().cuda()[None]
    lens = torch.tensor([1000], dtype=torch.int32).cuda()          # 63 pages
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    got, held = cache.select_pages(q, bounds, table, lens, 10, first=1, last=2)
    want = table[0, :8].tolist() + table[0, 61:63].tolist()         # all equal: the earlier
    assert got[0, 0].tolist() == want and got[0, 1].tolist() == want and held.item() == 152
    # infinite bounds come first; NaN scores last, and latch
    q = torch.randn(1, 4, 64, generator=g).bfloat16().abs().cuda()
    bounds[int(table[0, 20]), 0, 1, 3] = math.inf
    bounds[int(table[0, 30]), 1, :, 3] = math.nan
    got, _ = cache.select_pages(q, bounds, table, lens, 4, first=1, last=2)
    assert moe.coli_device_status() == moe.COLI_EDEVICE
    assert got[0, 0].tolist() == [int(table[0, j]) for j in (0, 20, 61, 62)]
    got, _ = cache.select_pages(q, bounds, table, lens, 62, first=0, last=1)
    assert moe.coli_device_status() == moe.COLI_EDEVICE
    assert got[0, 1].tolist() == [int(table[0, j]) for j in range(63) if j != 30]
    # a page outside the pool counts as -inf
    table[0, 40] = 64
    bounds.nan_to_num_(0, 0, 0)
    got, _ = cache.select_pages(q, bounds, table, lens, 62, first=0, last=1)
    assert moe.coli_device_status() == moe.COLI_EDEVICE
    assert got[0, 0].tolist() == [int(table[0, j]) for j in range(63) if j != 40]


# ---- attention mass --------------------------------------------------------------------------
MASS = [  # fmt, B, hq, hk, D, page, lens, window
    ("bf16", 1, 2, 2, 64, 16, [1], 0), ("bf16", 4, 16, 2, 128, 16, [0, 17, 500, 1203], 0),
    ("bf16", 3, 20, 4, 80, 48, [100, 47, 480], 60), ("bf16", 2, 40, 2, 256, 16, [90, 333], 0),
    ("bf16", 2, 3, 1, 8, 16, [90, 33], 17), ("f32", 3, 6, 2, 80, 16, [300, 33, 16], 0),
    ("f32", 2, 24, 2, 128, 32, [200, 64], 5), ("mxfp8", 3, 8, 2, 128, 32, [700, 64, 301], 0),
    ("mxfp8", 2, 9, 1, 96, 64, [640, 5], 100), ("mxfp8", 1, 4, 2, 256, 16, [77], 0),
    ("mxfp4", 2, 32, 2, 64, 16, [400, 100], 0), ("mxfp4", 2, 34, 2, 128, 16, [1, 260], 33)]


@pytest.mark.parametrize("fmt,B,hq,hk,D,page,lens,window", MASS)
def test_attention_mass(fmt, B, hq, hk, D, page, lens, window):
    g = ref.gen(B, hq, D, lens[0])
    n_pages = sum(-(-n // page) for n in lens) + 2
    cache, k, _ = ref.pool(g, fmt, n_pages, page, hk, D)
    table = ref.tables(g, lens, page, n_pages)
    q = queries(g, B, hq, D, fmt)
    tl = torch.tensor(lens, dtype=torch.int32).cuda()
    _, lse = cache.attend(q, table.cuda(), tl, window=window, return_lse=True)
    before = torch.rand(n_pages, hk, page, generator=g)
    known = [max(0, n - 1 - b) for b, n in enumerate(lens)]
    got = cache.accumulate(before.cuda(), q, table.cuda(), tl, lse, window=window,
                           known=torch.tensor(known, dtype=torch.int32).cuda())
    want, tol = before.double(), torch.zeros(before.shape, dtype=torch.float64)
    G = hq // hk
    for b, n in enumerate(lens):
        lo = max(0, n - window) if window else 0
        for h in range(hk):
            w, t = ref.mass(q[b, h * G:(h + 1) * G].double().cpu(),
                            ref.context(k, table[b].tolist(), h, n)[lo:],
                            lse[b, h * G:(h + 1) * G].double().cpu(), D ** -0.5)
            for j in range(lo, n):
                at = (int(table[b, j // page]), h, j % page)
                old = 0.0 if j >= known[b] else float(before[at])
                want[at] = old + w[j - lo]
                # groups above 16 heads are added 16 (f32: 16) at a time
                tol[at] = t[j - lo] + (1 + G // 8) * 2.0 ** -24 * want[at]
    assert ((got.cpu().double() - want).abs() <= tol).all()
    # without `known` all are added to, and unseen places keep their bits
    got = cache.accumulate(before.cuda(), q, table.cuda(), tl, lse, window=window)
    for b, n in enumerate(lens):
        for j in range(known[b], n):
            at = (int(table[b, j // page]), slice(None), j % page)
            want[at] += before[at]
            tol[at] += 2.0 ** -23 * want[at]
    assert ((got.cpu().double() - want).abs() <= tol).all()
    if not window:                                   # the weights of a row sum to 1
        total = cache.accumulate(cache.new_mass(), q, table.cuda(), tl, lse).sum()
        assert abs(float(total) - hq * sum(n > 0 for n in lens)) < 1e-3 * hq * B


def test_attention_mass_of_empty_rows_masked_nans_and_bad_pages():
    g = ref.gen(31)
    cache, k, _ = ref.pool(g, "bf16", 8, 16, 1, 64)
    q = queries(g, 2, 4, 64, "bf16")
    table = torch.tensor([[0, 1], [2, 9]], dtype=torch.int32).cuda()
    lens = torch.tensor([20, 32], dtype=torch.int32).cuda()
    cache.k[1, :, 4:] = math.nan                     # behind the first sequence's end
    lse = torch.zeros(2, 4, device="cuda")
    lse[0, 1:] = -math.inf                           # rows that saw nothing add nothing
    m = cache.accumulate(cache.new_mass(), q, table, lens, lse)
    assert moe.coli_device_status() == moe.COLI_EDEVICE
    w = torch.exp((q[0, :1].double().cpu() @ torch.cat([k[0, 0], k[1, 0, :4]]).T) / 8)[0]
    got = torch.cat([m[0, 0], m[1, 0, :4]]).cpu().double()
    assert torch.allclose(got, w, rtol=1e-5, atol=0)
    assert not m[1, 0, 4:].any() and not m[3:].any() and (m[2] > 0).all()
    # one page in two sequences: both are added
    table = torch.tensor([[0, 1], [0, 3]], dtype=torch.int32).cuda()
    lens = torch.tensor([16, 16], dtype=torch.int32).cuda()
    one = [cache.accumulate(cache.new_mass(), q[i:i + 1], table[i:i + 1].contiguous(),
                            lens[i:i + 1], torch.zeros(1, 4, device="cuda")) for i in range(2)]
    two = cache.accumulate(cache.new_mass(), q, table, lens, torch.zeros(2, 4, device="cuda"))
    assert torch.allclose(two, one[0] + one[1], rtol=2.0 ** -22, atol=0)


def test_attention_mass_of_infinite_keys():
    g = ref.gen(32)
    for fmt in ("f32", "bf16"):
        cache, k, _ = ref.pool(g, fmt, 2, 16, 1, 64)
        q = queries(g, 1, 2, 64, fmt)
        q[..., 0] = 1.0
        cache.k[0, 0, 3, 0] = -math.inf              # score -inf: weight 0
        table = torch.tensor([[0]], dtype=torch.int32).cuda()
        lens = torch.tensor([16], dtype=torch.int32).cuda()
        m = cache.accumulate(cache.new_mass(), q, table, lens, torch.zeros(1, 2, device="cuda"))
        assert m[0, 0, 3] == 0 and torch.isfinite(m).all() and (m[0, 0, :3] > 0).all()


# ---- eviction ---------------------------------------------------------------------------------
EVICT = [  # fmt, B, hk, D, page, lens, keep, first, recent
    ("bf16", 1, 1, 64, 16, [40], 20, 1, 4), ("bf16", 4, 2, 128, 16, [0, 20, 900, 1303], 100, 4, 16),
    ("bf16", 2, 3, 8, 48, [500, 480], 333, 0, 0), ("f32", 2, 2, 80, 16, [300, 150], 47, 2, 45),
    ("f32", 1, 1, 256, 16, [65], 64, 0, 1), ("mxfp8", 3, 2, 128, 32, [700, 64, 301], 64, 1, 8),
    ("mxfp8", 2, 2, 256, 16, [640, 5], 16, 0, 3), ("mxfp4", 2, 2, 96, 16, [400, 100], 1, 0, 1),
    ("mxfp4", 2, 1, 32, 64, [9000, 8500], 2100, 4, 64),
    ("bf16", 1, 1, 16, 4096, [60000], 20000, 4, 64)]


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("fmt,B,hk,D,page,lens,keep,first,recent", EVICT)
def test_evict(fmt, B, hk, D, page, lens, keep, first, recent, in_place):
    g = ref.gen(B, hk, D, keep)
    per = -(-keep // page)
    n_pages = sum(-(-n // page) for n in lens) + B * per + 2
    cache, _, _ = ref.pool(g, fmt, n_pages, page, hk, D)
    table = ref.tables(g, lens, page, n_pages)
    into = ref.tables(g, [keep] * B, page, n_pages, table.flatten().tolist())
    mass = (torch.rand(n_pages, hk, page, generator=g) * 50).round() / 50     # with ties
    mass[torch.rand(mass.shape, generator=g) < 0.02] = math.nan
    pools = [x for x in (cache.k, cache.v, cache.k_scale, cache.v_scale) if x is not None]
    was = [x.cpu().clone() for x in pools] + [mass.clone()]
    want = [x.clone() for x in was]
    kept = torch.full((B, hk, keep), -1, dtype=torch.int32)
    dst = table if in_place else into
    for b, n in enumerate(lens):
        for h in range(hk):
            m = [float(mass[int(table[b, j // page]), h, j % page]) for j in range(n)]
            pick = ref.largest(m, keep, first, recent)
            for r, j in enumerate(pick):
                kept[b, h, r] = j
                if in_place and n <= keep:
                    continue
                for x, y in zip(want, was):
                    x[int(dst[b, r // page]), h, r % page] = y[int(table[b, j // page]), h,
                                                               j % page]
    mass = mass.cuda()
    got, held = cache.evict(mass, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), keep,
                            first=first, recent=recent, into=None if in_place else into.cuda())
    assert torch.equal(got.cpu(), kept) and held.tolist() == [min(n, keep) for n in lens]
    for x, y in zip(pools + [mass], want):
        assert torch.equal(x.cpu().view(torch.uint8), y.view(torch.uint8))


def test_evict_ties_of_zeros():
    # -0 and 0 are equal: the earlier ones stay
    g = ref.gen(42)
    cache, _, _ = ref.pool(g, "bf16", 8, 16, 1, 64)
    mass = torch.zeros(8, 1, 16)
    mass[::2] = -0.0
    mass[3, 0, 5] = 1.0
    table = torch.arange(8, dtype=torch.int32)[None].cuda()
    kept, _ = cache.evict(mass.cuda(), table, torch.tensor([128], dtype=torch.int32).cuda(), 40,
                          recent=1)
    assert kept[0, 0].tolist() == list(range(38)) + [53, 127]


def test_evict_with_bad_pages():
    g = ref.gen(41)
    cache, _, _ = ref.pool(g, "bf16", 8, 16, 1, 64)
    table = torch.tensor([[0, 8, 2]], dtype=torch.int32).cuda()
    mass = torch.rand(8, 1, 16, generator=g).cuda() + 1
    lens = torch.tensor([48], dtype=torch.int32).cuda()
    was = cache.k.clone()
    kept, held = cache.evict(mass, table, lens, 32)
    assert moe.coli_device_status() == moe.COLI_EDEVICE
    # the missing page's tokens count as -inf; what would go there is left out
    assert kept[0, 0].tolist() == list(range(16)) + list(range(32, 48)) and held.item() == 32
    assert torch.equal(cache.k, was)
    for bad in (-3, 49):
        kept, held = cache.evict(mass, torch.tensor([[0, 1, 2]], dtype=torch.int32).cuda(),
                                 torch.tensor([bad], dtype=torch.int32).cuda(), 48)
        assert moe.coli_device_status() == moe.COLI_EDEVICE
        assert held.item() == (0 if bad < 0 else 48)


def test_select_from_a_very_long_table():
    # more pages than shared memory holds keys for, and each page many times: equal scores
    g = ref.gen(79)
    n_pages, count, D = 200, 45001, 64
    cache, _, _ = ref.pool(g, "bf16", n_pages, 16, 1, D)
    bounds = cache.new_bounds()
    bounds.copy_(torch.randn(n_pages, 1, 2, D, generator=g).sort(2).values)
    table = torch.randint(0, n_pages, (1, count), generator=g).int()
    q = torch.randn(1, 3, D, generator=g).bfloat16().cuda()
    lens = torch.tensor([count * 16 - 3], dtype=torch.int32).cuda()
    box, qd = bounds.double().cpu(), q.double().cpu()
    by_page = [ref.score(qd[0], box[p, 0]) for p in range(n_pages)]
    scores = [by_page[p] for p in table[0].tolist()]
    for keep in (3, 700, 20000):
        got, held = cache.select_pages(q, bounds, table.cuda(), lens, keep, first=1, last=2)
        want = [int(table[0, j]) for j in ref.largest(scores, keep, 1, 2)]
        assert got[0, 0].tolist() == want and held.item() == keep * 16 - 3


# ---- streams, graphs, refusals -------------------------------------------------------------------
def all_calls(cache, q, own, lens, pre, prefix, bounds, mass, into):
    """One of each, on what one decode step has in hand."""
    out, lse = cache.attend_shared(q, pre, prefix, own, lens, return_lse=True)
    cache.page_bounds(bounds, own.flatten().contiguous(),
                      torch.full((own.numel(),), cache.page_size, dtype=torch.int32,
                                 device="cuda"))
    pages, held = cache.select_pages(q, bounds, own, lens, 3)
    sparse = cache.attend_selected(q, pages, held)
    cache.accumulate(mass, q, own, lens, lse)
    kept, new = cache.evict(mass, own, lens, 20, recent=2, into=into)
    return out, lse, pages, held, sparse, kept, new


def step_inputs(fmt, B=40, hq=8, hk=2, D=64, page=16, prefix=333):
    g = ref.gen(123)
    n_pre = -(-prefix // page)
    cache, _, _ = ref.pool(g, fmt, n_pre + B * 10, page, hk, D)
    pre = torch.arange(n_pre, dtype=torch.int32).cuda()
    ids = (n_pre + torch.randperm(B * 10, generator=g)).int()
    own = ids[:B * 8].reshape(B, 8).contiguous().cuda()
    into = ids[B * 8:].reshape(B, 2).contiguous().cuda()
    lens = torch.randint(0, 129, (B,), generator=g).int().cuda()
    q = torch.randn(B, hq, D, generator=g).to(ref.act(fmt)).cuda()
    return cache, q, own, lens, pre, prefix, cache.new_bounds(), cache.new_mass(), into


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "f32"])
def test_captured_and_replayed(fmt):
    a = step_inputs(fmt)
    cache, q, own, lens, mass = a[0], a[1], a[2], a[3], a[7]
    pools = [x for x in (cache.k, cache.v, cache.k_scale, cache.v_scale, mass) if x is not None]
    was = [x.clone() for x in pools]
    all_calls(*a)                                        # kernels loaded before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_calls(*a)
    for turn in range(3):
        for x, y in zip(pools, was):
            x.copy_(y)
        q.copy_(torch.randn(q.shape, generator=ref.gen(turn)).to(q.dtype))
        lens.copy_(torch.randint(0, 129, lens.shape, generator=ref.gen(turn, 1)))
        graph.replay()
        torch.cuda.synchronize()
        after = [x.clone() for x in pools]
        results = [x.clone() for x in got]
        for x, y in zip(pools, was):
            x.copy_(y)
        eager = all_calls(*a)
        for x, y in zip(results, eager):
            assert torch.equal(x, y)
        for x, y in zip(after, pools):
            assert torch.equal(x, y)


def test_two_streams_at_once():
    a, b = step_inputs("bf16"), step_inputs("mxfp8")
    want = [all_calls(*a), all_calls(*b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for x in (a, b):
            x[7].zero_()
        torch.cuda.synchronize()
        for s, x in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                got.append(all_calls(*x))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(g, w))


STREAM_CALLS = {
    "attend_shared": lambda c, x, t, n, s: c.attend_shared(x, t[0], 16, t, n, stream=s),
    "select_pages": lambda c, x, t, n, s: c.select_pages(x, c.boxes, t, n, 1, first=0, stream=s),
    "attend_selected": lambda c, x, t, n, s: c.attend_selected(
        x, t[:, None].expand(-1, 4, -1).contiguous(), n, stream=s),
    "accumulate": lambda c, x, t, n, s: c.accumulate(c.masses, x, t, n, c.lses, stream=s),
}


@pytest.mark.parametrize("name", list(STREAM_CALLS))
def test_inputs_let_go_of_are_not_given_away(name):
    B, h, D = 4096, 4, 64
    c = moe.PagedKVCache.empty(B // 16, 16, h, D, moe.BF16)
    c.boxes, c.masses = c.new_bounds(), c.new_mass()
    c.lses = torch.zeros(B, h, device="cuda")
    ids = (torch.arange(B, device="cuda") % 16).int()
    table = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    STREAM_CALLS[name](c, torch.randn(B, h, D, device="cuda").bfloat16(), table, ids, None)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    x = torch.ones(B, h, D, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)            # the call waits some 50 ms for its turn
    STREAM_CALLS[name](c, x, table, ids, side)
    where = x.data_ptr()
    del x
    others = [torch.empty(B, h, D, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    assert all(o.data_ptr() != where for o in others)
    assert not side.query()                       # the work was indeed still to come
    torch.cuda.synchronize()


def test_wrappers_refuse_what_does_not_fit():
    cache, q, own, lens, pre, prefix, bounds, mass, into = step_inputs("bf16")
    lse = torch.zeros(q.shape[:2], device="cuda")
    pages = torch.zeros(40, 2, 3, dtype=torch.int32, device="cuda")
    bad = [
        lambda: cache.attend_shared(q.float(), pre, prefix, own, lens),
        lambda: cache.attend_shared(q, pre[:5], prefix, own, lens),          # too few pages
        lambda: cache.attend_shared(q, pre.long(), prefix, own, lens),
        lambda: cache.attend_shared(q, pre.cpu(), prefix, own, lens),
        lambda: cache.attend_shared(q, pre, prefix, own[:3], lens),
        lambda: cache.attend_shared(q, pre, prefix, own, lens[:3]),
        lambda: cache.attend_shared(q, pre, prefix, own, lens, out=q[:3]),
        lambda: cache.page_bounds(bounds[:3], pre, pre),
        lambda: cache.page_bounds(bounds.float(), pre, pre),
        lambda: cache.page_bounds(bounds, pre, pre[:3]),
        lambda: cache.page_bounds(bounds, own, own),
        lambda: cache.select_pages(q, bounds.float(), own, lens, 3),
        lambda: cache.select_pages(q, bounds, own.t(), lens, 3),
        lambda: cache.select_pages(q, bounds, own, lens, 0),
        lambda: cache.attend_selected(q, pages[:, :1], lens),
        lambda: cache.attend_selected(q, pages[0], lens),
        lambda: cache.attend_selected(q, pages.long(), lens),
        lambda: cache.accumulate(mass[:3], q, own, lens, lse),
        lambda: cache.accumulate(mass, q, own, lens, lse[:, :3]),
        lambda: cache.accumulate(mass, q, own, lens, lse, known=lens[:3]),
        lambda: cache.evict(mass.double(), own, lens, 20),
        lambda: cache.evict(mass, own[0], lens, 20),
        lambda: cache.evict(mass, own, lens, 0),
        lambda: cache.evict(mass, own, lens, 20, into=into[:3]),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: cache.select_pages(q, bounds, own, lens, 3, first=2, last=2),
                 lambda: cache.evict(mass, own, lens, 20, first=10, recent=11),
                 lambda: cache.evict(mass, own, lens, 40, into=into),        # no room for 40
                 lambda: cache.attend_shared(q, pre, -1, own, lens)):
        with pytest.raises(moe.ColiError):
            call()


def test_no_sequences():
    cache, q, own, lens, pre, prefix, bounds, mass, into = step_inputs("bf16")
    z, zt, zl = q[:0], own[:0], lens[:0]
    assert cache.attend_shared(z, pre, prefix, zt, zl).shape == (0, 8, 64)
    pages, held = cache.select_pages(z, bounds, zt, zl, 3)
    assert pages.shape == (0, 2, 3) and held.shape == (0,)
    assert cache.attend_selected(z, pages, held).shape == (0, 8, 64)
    cache.accumulate(mass, z, zt, zl, torch.zeros(0, 8, device="cuda"))
    kept, new = cache.evict(mass, zt, zl, 5)
    assert kept.shape == (0, 2, 5) and new.shape == (0,)
    cache.page_bounds(bounds, zl, zl)


# ---- together ------------------------------------------------------------------------------------
def test_a_serving_loop_with_all_of_them():
    # a shared prompt, tokens of each sequence behind it, sparse attention over them, mass
    # and eviction, step after step; the cache and what is returned stay consistent
    g = ref.gen(99)
    B, hq, hk, D, page, prefix = 20, 8, 2, 64, 16, 150
    budget, n_own = 40, 8
    cache = moe.PagedKVCache.empty(10 + B * n_own, page, hk, D, moe.MXFP8)
    rotary = moe.Rotary.build(D, 1000)
    pre = torch.arange(10, dtype=torch.int32, device="cuda")
    own = (10 + torch.randperm(B * n_own, generator=g).reshape(B, n_own)).int().cuda()
    x = torch.randn(prefix, 2 * hk, D, generator=g).bfloat16().cuda()
    pos = torch.arange(prefix, dtype=torch.int32, device="cuda")
    cache.append(x[:, :hk], x[:, hk:], (pre[pos.long() // page] * page + pos % page).int(), rotary,
                 pos)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    bounds, mass = cache.new_bounds(), cache.new_mass()
    for step in range(60):
        x = torch.randn(B, hq + 2 * hk, D, generator=g).bfloat16().cuda()
        at = own.gather(1, (lens.long() // page)[:, None])[:, 0]
        q = cache.append(x[:, hq:hq + hk], x[:, hq + hk:], at * page + lens % page, rotary,
                         torch.full((B,), prefix + step, dtype=torch.int32, device="cuda"),
                         q=x[:, :hq])
        cache.page_bounds(bounds, at, lens % page + 1)
        lens += 1
        both, lse = cache.attend_shared(q, pre, prefix, own, lens, return_lse=True)
        pages, held = cache.select_pages(q, bounds, own, lens, 2)
        sparse, lse_s = cache.attend_selected(q, pages, held, return_lse=True)
        assert torch.isfinite(both.float()).all() and torch.isfinite(sparse.float()).all()
        # the whole context holds at least what a part of it does
        assert (lse >= lse_s - 1e-4).all()
        cache.accumulate(mass, q, own, lens, lse, known=lens - 1)
        if int(lens[0]) > budget + 8:
            kept, lens = cache.evict(mass, own, lens, budget, first=2, recent=8)
            assert (kept[..., 1:] > kept[..., :-1]).all() and (lens == budget).all()
            cache.page_bounds(bounds, own[:, :3].flatten().contiguous(),
                              torch.tensor([16, 16, 8] * B, dtype=torch.int32, device="cuda"))
    # what stands in the cache is what an attention over it by hand gives
    rows = [torch.stack([cache.read((own[b].long().repeat_interleave(page) * page +
                                     torch.arange(page, device="cuda").repeat(n_own)).int())[i]
                         for b in range(B)]).double().cpu() for i in range(2)]
    pr = [y.double().cpu() for y in cache.read(torch.arange(prefix, dtype=torch.int32,
                                                            device="cuda"))]
    n = lens.tolist()
    want, wl, tol, tl = attn_ref.attend(
        q, lambda b, h: torch.cat([pr[0][:, h], rows[0][b, :n[b], h]]),
        lambda b, h: torch.cat([pr[1][:, h], rows[1][b, :n[b], h]]), [prefix + m for m in n], hk,
        D ** -0.5)
    out = cache.attend_shared(q, pre, prefix, own, lens)
    assert ((out.cpu().double() - want).abs() <= tol + 2.0 ** -8 * want.abs()).all()
