"""Shared prefixes, chosen pages and eviction on the paths that only some calls take, against
their plain 64-bit forms (GPU)."""
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


def out_step(fmt):
    return 2.0 ** -24 if fmt == "f32" else 2.0 ** -8


# ---- choice of pages -----------------------------------------------------------------------
def page_scores(q, bounds):
    """fp64 [B][n_kv_heads][n_pages]: the largest score of each key head's queries."""
    q, box = q.double().cpu(), bounds.double().cpu()
    B, hq, D = q.shape
    q = q.view(B, box.shape[1], -1, D)
    s = torch.einsum("bhgd,phd->bhgp", q.clamp(min=0), box[:, :, 1]) + \
        torch.einsum("bhgd,phd->bhgp", q.clamp(max=0), box[:, :, 0])
    return s.amax(2)


def best_pages(scores, table, n, keep, first, last):
    """The pages of one list [n_pages] of scores that are taken, in the context's order."""
    s = scores[table[:n].long()].clone()
    if n <= keep:
        return table[:n].tolist() + [-1] * (keep - n)
    s[:first], s[n - last:] = math.inf, math.inf
    at = torch.sort(s, descending=True, stable=True).indices[:keep].sort().values
    return table[at].tolist()


def choose_guarded(cache, q, bounds, table, lens, keep, first, last):
    """The pages chosen and their lengths, with guard words behind both, which have to stay."""
    B, hk = q.shape[0], cache.n_kv_heads
    pages = torch.full((B * hk * keep + 4096,), 12345, dtype=torch.int32, device="cuda")
    held = torch.full((B + 64,), 12345, dtype=torch.int32, device="cuda")
    n = moe.coli_select_pages_scratch_bytes(cache.c, B, table.shape[1])
    scratch = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert moe.coli_select_pages(cache.c, bounds, q, q.stride(0), q.shape[1], B, table,
                                 table.shape[1], lens, keep, first, last, pages, held, scratch,
                                 n) == moe.COLI_OK
    assert (pages[B * hk * keep:] == 12345).all() and (held[B:] == 12345).all()
    return pages[:B * hk * keep].view(B, hk, keep).cpu(), held[:B].cpu()


@pytest.mark.parametrize("fmt", ["bf16", "f32"])
@pytest.mark.parametrize("B,hk,count", [(48, 4, 700), (48, 4, 5000), (1, 1, 300), (3, 2, 4097)])
def test_select_with_more_equal_pages_than_are_ranked_at_once(B, hk, count, fmt):
    # a query of zeros, and lists that name few pages many times: hundreds of scores are equal
    # to the last one chosen, and all of them are looked at again
    g = ref.gen(B, hk, count)
    n_pages, D = 24, 64
    cache, _, _ = ref.pool(g, fmt, n_pages, 16, hk, D)
    bounds = cache.new_bounds()
    bounds.copy_(torch.randn(n_pages, hk, 2, D, generator=g).sort(2).values)
    table = torch.randint(0, n_pages, (B, count), generator=g).int()
    lens = torch.randint(count // 2, count, (B,), generator=g).int() * 16 + 5
    lens[0] = count * 16
    q = torch.randn(B, 2 * hk, D, generator=g).to(ref.act(fmt))
    q[::3] = 0
    scores = page_scores(q, bounds)
    for keep, first, last in ((64, 1, 2), (290, 0, 1)):
        want = torch.tensor([[best_pages(scores[b, h], table[b], -(-int(lens[b]) // 16), keep,
                                         first, last) for h in range(hk)] for b in range(B)])
        for _ in range(4):
            got, held = choose_guarded(cache, q.cuda(), bounds, table.cuda(), lens.cuda(), keep,
                                       first, last)
            assert torch.equal(got, want.int())
            assert held.tolist() == [int(n) - max(0, -(-int(n) // 16) - keep) * 16 for n in lens]


@pytest.mark.parametrize("fmt", ["bf16", "f32", "mxfp8"])
@pytest.mark.parametrize("count", [100, 2000])
def test_select_among_scores_that_fp32_does_not_hold(fmt, count):
    # products of 2^-140 and below: fp32 sums of them are a few multiples of 2^-149, or 0
    g = ref.gen(count, 5)
    D, keep = 64, 20
    cache, _, _ = ref.pool(g, fmt, count, 16, 1, D)
    bounds = cache.new_bounds()
    bounds.copy_(torch.randn(count, 1, 2, D, generator=g).sort(2).values * 2.0 ** -76)
    q = (torch.randn(2, 3, D, generator=g) * 2.0 ** -70).to(ref.act(fmt))
    table = torch.stack([torch.randperm(count, generator=g) for _ in range(2)]).int()
    lens = torch.tensor([count * 16, count * 16 - 7], dtype=torch.int32)
    scores = page_scores(q, bounds)
    want = torch.tensor([[best_pages(scores[b, 0], table[b], count, keep, 1, 1)]
                         for b in range(2)])
    got, _ = choose_guarded(cache, q.cuda(), bounds, table.cuda(), lens.cuda(), keep, 1, 1)
    assert torch.equal(got, want.int())


@pytest.mark.parametrize("fmt,B,hk,D,count", [("bf16", 32, 8, 64, 1300), ("bf16", 64, 8, 128, 1100),
                                              ("bf16", 40, 8, 192, 1500), ("f32", 32, 8, 80, 900)])
def test_select_of_many_long_lists(fmt, B, hk, D, count):
    # more pages than the blocks of a list take at a time
    g = ref.gen(B, hk, D, count)
    n_pages = 2500
    keys = torch.zeros(n_pages, hk, 16, D, dtype=ref.act(fmt), device="cuda")    # not read
    cache = moe.PagedKVCache(keys, keys, head_dim=D)
    bounds = cache.new_bounds()
    bounds.copy_(torch.randn(n_pages, hk, 2, D, generator=g).sort(2).values)
    table = torch.stack([torch.randperm(n_pages, generator=g)[:count] for _ in range(B)]).int()
    lens = torch.randint(count // 3, count, (B,), generator=g).int() * 16 + 3
    lens[1] = count * 16
    q = torch.randn(B, 3 * hk, D, generator=g).to(ref.act(fmt))
    scores = page_scores(q, bounds)
    keep, first, last = 50, 1, 2
    want = torch.tensor([[best_pages(scores[b, h], table[b], -(-int(lens[b]) // 16), keep, first,
                                     last) for h in range(hk)] for b in range(B)])
    got, held = choose_guarded(cache, q.cuda(), bounds, table.cuda(), lens.cuda(), keep, first,
                               last)
    assert torch.equal(got, want.int())
    assert held.tolist() == [int(n) - max(0, -(-int(n) // 16) - keep) * 16 for n in lens]


# ---- attention mass --------------------------------------------------------------------------
def masses(cache, k, q, table, lens, window, scale, known, before, lse=None):
    """(want, tolerance) of accumulate over `before`, fp64 [n_pages][n_kv_heads][page_size],
    and the lse that it is given (None: attend's)."""
    n_pages, hk, page = before.shape
    G = q.shape[1] // hk
    if lse is None:
        _, lse = cache.attend(q, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                              window=window, scale=scale, return_lse=True)
    want, tol = before.double(), torch.zeros(before.shape, dtype=torch.float64)
    qd, ld = q.double().cpu(), lse.double().cpu()
    for b, n in enumerate(lens):
        lo = max(0, n - window) if window else 0
        j = torch.arange(lo, n)
        at = table[b].long()[j // page]
        for h in range(hk):
            r = slice(h * G, (h + 1) * G)
            w, t = ref.mass(qd[b, r], k[at, h, j % page], ld[b, r], scale)
            old = torch.where(j >= known[b], 0.0, want[at, h, j % page])
            want[at, h, j % page] = old + w
            # groups are added 8 or 16 heads at a time
            tol[at, h, j % page] = t + (1 + G // 8) * 2.0 ** -24 * (old + w)
    return want, tol, lse


MASS = [  # fmt, B, hq, hk, D, page, longest, window: several tiles a warp
    ("bf16", 64, 16, 8, 64, 16, 1500, 0), ("bf16", 64, 32, 8, 128, 48, 1100, 0),
    ("bf16", 150, 20, 1, 80, 128, 3000, 1777), ("f32", 64, 16, 8, 64, 48, 1000, 0),
    ("f32", 100, 20, 2, 128, 16, 1900, 900), ("f32", 64, 8, 4, 256, 128, 800, 0),
    ("mxfp8", 64, 16, 8, 64, 48, 1500, 0), ("mxfp8", 64, 8, 4, 128, 16, 1300, 1000),
    ("mxfp8", 100, 40, 2, 256, 128, 1400, 0), ("mxfp4", 64, 32, 8, 64, 128, 1600, 0),
    ("mxfp4", 150, 18, 1, 128, 48, 3000, 0), ("mxfp4", 64, 24, 4, 96, 16, 1200, 700)]


@pytest.mark.parametrize("fmt,B,hq,hk,D,page,longest,window", MASS)
def test_attention_mass_of_many_contexts(fmt, B, hq, hk, D, page, longest, window):
    g = ref.gen(B, hq, D, page)
    lens = torch.randint(0, longest + 1, (B,), generator=g).tolist()
    lens[:4] = [longest, 0, 1, longest - 1]
    n_pages = sum(-(-n // page) for n in lens) + 2
    cache, k, _ = ref.pool(g, fmt, n_pages, page, hk, D)
    table = ref.tables(g, lens, page, n_pages)
    q = torch.randn(B, hq, D, generator=g).to(ref.act(fmt)).cuda()
    before = torch.rand(n_pages, hk, page, generator=g)
    known = [max(0, n - 1 - b % 30) for b, n in enumerate(lens)]
    want, tol, lse = masses(cache, k, q, table, lens, window, D ** -0.5, known, before)
    tl, tk = (torch.tensor(x, dtype=torch.int32).cuda() for x in (lens, known))
    got = cache.accumulate(before.cuda(), q, table.cuda(), tl, lse, window=window, known=tk)
    assert ((got.cpu().double() - want).abs() <= tol).all()
    again = cache.accumulate(before.cuda(), q, table.cuda(), tl, lse, window=window, known=tk)
    assert torch.equal(got, again)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("hq,D", [(3, 64), (20, 128), (6, 256), (12, 96)])
@pytest.mark.parametrize("kind", ["spread", "small", "large"])
def test_attention_mass_of_queries_beyond_fp16(kind, hq, D, fmt):
    # elements 2^35 apart, or heads of 2^-90 or 2^90: fp16 holds no multiple of them
    g = ref.gen(hq, D, 4)
    lens = [700, 33]
    cache, k, _ = ref.pool(g, fmt, 60, 16, 1, D)
    table = ref.tables(g, lens, 16, 60)
    q = torch.randn(2, hq, D, generator=g)
    scale = D ** -0.5
    if kind == "spread":
        q[..., ::2] *= 2.0 ** 20
        q[..., 1::2] *= 2.0 ** -15
        scale *= 2.0 ** -20
    else:
        e = 90.0 if kind == "large" else -90.0
        q *= 2.0 ** e
        scale *= 2.0 ** -e
    q = q.bfloat16().cuda()
    before = torch.rand(60, 1, 16, generator=g)
    want, tol, lse = masses(cache, k, q, table, lens, 0, scale, lens, before)
    got = cache.accumulate(before.cuda(), q, table.cuda(),
                           torch.tensor(lens, dtype=torch.int32).cuda(), lse, scale=scale)
    assert ((got.cpu().double() - want).abs() <= tol).all()


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("kind", ["far keys", "small scale", "least keys"])
def test_attention_mass_of_extreme_scales(kind, fmt):
    # scores of ordinary size from factors at the ends of their ranges
    g = ref.gen(91)
    D, lens = 64, [100, 17]
    cache, _, _ = ref.pool(g, fmt, 12, 16, 1, D)
    q = torch.randn(2, 4, D, generator=g)
    scale = D ** -0.5
    if kind == "far keys":
        cache.k_scale[..., :2] = 127 + 112
        q *= 2.0 ** -77
        scale *= 2.0 ** -35
    elif kind == "small scale":
        cache.k_scale[..., :2] = 127 + 112
        scale *= 2.0 ** -112
    else:                                            # 2^-127, the least scale there is
        cache.k_scale[..., :2] = 0
        q *= 2.0 ** 77
        scale *= 2.0 ** 50
    k = attn_ref.decode(cache.k, cache.k_scale, fmt)
    table = ref.tables(g, lens, 16, 12)
    q = q.bfloat16().cuda()
    before = torch.rand(12, 1, 16, generator=g)
    lse = torch.stack([torch.logsumexp(scale * q[b].double().cpu() @ ref.context(
        k, table[b].tolist(), 0, n).T, -1) for b, n in enumerate(lens)]).float().cuda()
    want, tol, _ = masses(cache, k, q, table, lens, 0, scale, lens, before, lse)
    got = cache.accumulate(before.cuda(), q, table.cuda(),
                           torch.tensor(lens, dtype=torch.int32).cuda(), lse, scale=scale)
    assert torch.isfinite(got).all()
    assert ((got.cpu().double() - want).abs() <= tol).all()


# ---- shared prefix ---------------------------------------------------------------------------
def shared_case(fmt, hq, hk, D, page, prefix, own):
    """(cache, q, prefix pages, table, lens, k_of, v_of) of a batch behind a prefix."""
    g = ref.gen(len(own), hq, D, prefix)
    n_pre = -(-prefix // page)
    n_pages = n_pre + sum(-(-n // page) for n in own) + 2
    cache, k, v = ref.pool(g, fmt, n_pages, page, hk, D)
    pre = torch.randperm(n_pages, generator=g)[:n_pre].int()
    table = ref.tables(g, own, page, n_pages, pre.tolist())
    q = torch.randn(len(own), hq, D, generator=g).to(ref.act(fmt)).cuda()
    ahead = [[ref.context(x, pre.tolist(), h, prefix) for h in range(hk)] for x in (k, v)]

    def of(rows, first):
        return lambda b, h: torch.cat([first[h], ref.context(rows, table[b].tolist(), h, own[b])])

    return (cache, q, pre.cuda(), table.cuda(), torch.tensor(own, dtype=torch.int32).cuda(),
            of(k, ahead[0]), of(v, ahead[1]))


def held(out, lse, want, want_lse, tol, tol_lse, fmt):
    tol = tol * (1 + out_step(fmt)) + out_step(fmt) * want.abs()
    return ((out.cpu().double() - want).abs() <= tol).all() and \
        ((lse.cpu().double() - want_lse).abs() <= tol_lse).all()


SOME = [0, 1, 700, 3000, 17, 16, 513, 0, 1200]
OWN_CUT = [  # fmt, hq, hk, D, page, prefix, own: the own tokens are cut in pieces
    ("bf16", 32, 8, 64, 16, 5000, SOME), ("bf16", 16, 2, 128, 48, 20001, SOME[:3]),
    ("bf16", 12, 1, 256, 16, 3000, [2999]), ("bf16", 24, 2, 80, 64, 1000, SOME * 4),
    ("mxfp8", 32, 8, 64, 16, 5000, SOME), ("mxfp8", 16, 2, 128, 48, 20001, [700, 400, 0]),
    ("mxfp8", 24, 2, 96, 64, 1000, SOME * 4), ("mxfp4", 32, 8, 64, 32, 5000, SOME),
    ("mxfp4", 64, 4, 128, 16, 9000, SOME), ("mxfp4", 24, 2, 32, 64, 1000, SOME * 4),
    # few queries a key head, and fp32: the decode kernel takes the prefix too
    ("bf16", 8, 8, 64, 16, 3000, [900, 0, 2500]), ("mxfp8", 4, 4, 128, 16, 3000, [900, 0, 2500]),
    ("f32", 12, 4, 64, 16, 3000, SOME), ("f32", 8, 2, 128, 48, 900, SOME * 4)]


@pytest.mark.parametrize("fmt,hq,hk,D,page,prefix,own", OWN_CUT)
def test_shared_prefix_with_long_own_contexts(fmt, hq, hk, D, page, prefix, own):
    cache, q, pre, table, lens, k_of, v_of = shared_case(fmt, hq, hk, D, page, prefix, own)
    want = attn_ref.attend(q, k_of, v_of, [prefix + n for n in own], hk, D ** -0.5)
    call = lambda: cache.attend_shared(q, pre, prefix, table, lens, return_lse=True)
    out, lse = call()
    assert held(out, lse, *want, fmt)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = call()
    for _ in range(3):
        again[0].fill_(7), again[1].fill_(7)
        graph.replay()
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
        assert all(torch.equal(x, y) for x, y in zip(call(), (out, lse)))


@pytest.mark.parametrize("fmt,own", [("bf16", [0, 1, 700, 3000] + [300] * 40), ("mxfp8", [600, 1] * 20),
                                     ("mxfp4", [0, 2100] * 6)])
def test_shared_prefix_that_outlasts_the_own_tokens(fmt, own):
    # the own tokens are done while the prefix's products still run
    hq, hk, D, page, prefix = 32, 4, 64, 64, 40000
    cache, q, pre, table, lens, k_of, v_of = shared_case(fmt, hq, hk, D, page, prefix, own)
    want = attn_ref.attend(q, k_of, v_of, [prefix + n for n in own], hk, D ** -0.5)
    first = cache.attend_shared(q, pre, prefix, table, lens, return_lse=True)
    assert held(*first, *want, fmt)
    for _ in range(10):
        again = cache.attend_shared(q, pre, prefix, table, lens, return_lse=True)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


MANY_ROWS = [  # fmt, B, hq, hk, D, page, prefix: prefixes that the decode kernel reads
    ("f32", 40, 32, 4, 64, 16, 1500), ("f32", 130, 8, 2, 128, 48, 700),
    ("f32", 33, 24, 1, 256, 16, 401), ("f32", 100, 3, 3, 80, 64, 2000),
    ("mxfp8", 40, 16, 2, 160, 16, 900), ("mxfp8", 9, 4, 4, 256, 64, 2100),
    ("mxfp4", 33, 8, 1, 256, 48, 777), ("mxfp4", 100, 10, 2, 192, 16, 300),
    ("mxfp4", 3, 12, 4, 224, 32, 5000), ("mxfp8", 150, 40, 2, 192, 128, 200)]


@pytest.mark.parametrize("fmt,B,hq,hk,D,page,prefix", MANY_ROWS)
def test_shared_prefix_of_many_rows_on_the_decode_kernel(fmt, B, hq, hk, D, page, prefix):
    own = [b % 37 for b in range(B)]
    cache, q, pre, table, lens, k_of, v_of = shared_case(fmt, hq, hk, D, page, prefix, own)
    want = attn_ref.attend(q, k_of, v_of, [prefix + n for n in own], hk, D ** -0.5)
    out, lse = cache.attend_shared(q, pre, prefix, table, lens, return_lse=True)
    assert held(out, lse, *want, fmt)
    # pages that are left out
    pre = torch.full_like(pre, -1)
    out, lse = cache.attend_shared(q, pre, prefix, table, torch.zeros_like(lens), return_lse=True)
    assert moe.coli_device_status() == moe.COLI_EDEVICE
    assert not out.any() and (lse == -math.inf).all()


ODD = [("bf16", 40, 64), ("bf16", 80, 128), ("bf16", 40, 256), ("bf16", 1, 64), ("f32", 40, 64)]


@pytest.mark.parametrize("fmt,B,D", ODD)
def test_shared_prefix_of_infinite_scores(fmt, B, D):
    # keys of -inf weigh 0 (nothing else: zeros, -inf), keys of +inf and NaN make their own key
    # head's rows NaN, wherever in the prefix they lie
    g = ref.gen(B, D, 6)
    dt, n = ref.act(fmt), 300
    k = torch.ones(19, 5, 16, D, dtype=dt, device="cuda")
    v = torch.randn(19, 5, 16, D, generator=g).to(dt).cuda()
    k[:, 0] = -math.inf
    k[3:11, 1], k[18, 1, 3] = -math.inf, -math.inf
    k[17, 2, 5] = math.inf
    k[9, 3, 2, 1] = math.nan
    k[18, 4, 12:], v[18, 4, 12:] = math.nan, math.inf                # behind the prefix
    cache = moe.PagedKVCache(k, v, head_dim=D)
    q = torch.ones(B, 10, D, dtype=dt, device="cuda")
    pre = torch.arange(19, dtype=torch.int32, device="cuda")
    table = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    out, lse = cache.attend_shared(q, pre, n, table, lens, return_lse=True)
    assert not out[:, :2].any() and (lse[:, :2] == -math.inf).all()
    assert out[:, 4:8].isnan().all() and lse[:, 4:8].isnan().all()
    for h, gone in ((1, list(range(48, 176)) + [18 * 16 + 3]), (4, [])):
        keep = [j for j in range(n) if j not in gone]
        rows = v[:, h].reshape(-1, D)[keep].double().cpu()
        tol = 2.0 ** -8 if fmt == "bf16" else 2.0 ** -18
        err = (out[:, 2 * h:2 * h + 2].double().cpu() - rows.mean(0)).abs()
        assert (err <= tol * rows.abs().mean(0) + out_step(fmt) * rows.mean(0).abs()).all()
        want = math.log(len(keep)) + D ** 0.5
        assert ((lse[:, 2 * h:2 * h + 2] - want).abs() <= 2.0 ** -16 * want).all()


@pytest.mark.parametrize("fmt,B,D", ODD)
def test_shared_prefix_of_odd_values_and_queries(fmt, B, D):
    # an infinite value makes its element infinite or NaN and no other; a NaN query its own row
    cache, q, pre, table, lens, _, _ = shared_case(fmt, 8, 2, D, 16, 777, [b % 20 for b in range(B)])
    want, want_lse = cache.attend_shared(q, pre, 777, table, lens, return_lse=True)
    at = int(pre[30])
    cache.v[at, 0, 5, 3], cache.v[at, 1, 6, D - 1] = math.inf, math.nan
    out, lse = cache.attend_shared(q, pre, 777, table, lens, return_lse=True)
    assert torch.equal(lse, want_lse)
    hit = torch.zeros(8, D, dtype=torch.bool, device="cuda")
    hit[:4, 3], hit[4:, D - 1] = True, True
    assert not torch.isfinite(out[:, hit]).any() and torch.equal(out[:, ~hit], want[:, ~hit])
    cache.v[at, 0, 5, 3], cache.v[at, 1, 6, D - 1] = 1.0, 1.0
    want, want_lse = cache.attend_shared(q, pre, 777, table, lens, return_lse=True)
    q[0, 1, 7] = math.nan
    out, lse = cache.attend_shared(q, pre, 777, table, lens, return_lse=True)
    assert out[0, 1].isnan().all() and lse[0, 1].isnan()
    out[0, 1], lse[0, 1] = want[0, 1], want_lse[0, 1]
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("B,D", [(40, 64), (80, 128), (1, 64), (20, 256)])
def test_shared_prefix_of_nan_blocks_and_codes(B, D, fmt):
    own = [b % 20 for b in range(B)]
    cache, q, pre, table, lens, k_of, v_of = shared_case(fmt, 8, 2, D, 16, 777, own)
    exact = attn_ref.attend(q, k_of, v_of, [777 + n for n in own], 2, D ** -0.5)
    call = lambda: cache.attend_shared(q, pre, 777, table, lens, return_lse=True)
    want, want_lse = call()
    at, old = int(pre[30]), cache.v_scale[int(pre[30]), 0, 5, 1].clone()
    cache.v_scale[at, 0, 5, 1] = 255                                 # channels 32 to 63
    out, lse = call()
    assert out[:, :4, 32:64].isnan().all() and torch.equal(lse, want_lse)
    out[:, :4, 32:64] = want[:, :4, 32:64]
    assert held(out, lse, *exact, fmt)
    cache.v_scale[at, 0, 5, 1] = old
    if fmt == "mxfp8":
        old = cache.v[at, 1, 9, 6].clone()
        cache.v[at, 1, 9, 6] = 0x7f
        out, lse = call()
        assert out[:, 4:, 6].isnan().all() and torch.equal(lse, want_lse)
        out[:, 4:, 6] = want[:, 4:, 6]
        assert held(out, lse, *exact, fmt)
        cache.v[at, 1, 9, 6] = old
        old = cache.k[at, 1, 9, 6].clone()
        cache.k[at, 1, 9, 6] = 0xff
        out, lse = call()
        assert out[:, 4:].isnan().all() and lse[:, 4:].isnan().all()
        assert torch.equal(out[:, :4], want[:, :4]) and torch.equal(lse[:, :4], want_lse[:, :4])
        cache.k[at, 1, 9, 6] = old
    cache.k_scale[at, 0, 5, 0] = 255
    out, lse = call()
    assert out[:, :4].isnan().all() and lse[:, :4].isnan().all()
    assert torch.equal(out[:, 4:], want[:, 4:]) and torch.equal(lse[:, 4:], want_lse[:, 4:])


# ---- selected attention ----------------------------------------------------------------------
@pytest.mark.parametrize("fmt", list(ref.FMT))
@pytest.mark.parametrize("n", [40, 1500])
def test_selected_attention_of_odd_scores(fmt, n):
    # each key head has pages of its own: what is odd in one of them stays with its head
    hk, D, page, B = 4, 64, 16, 2
    g = ref.gen(n, 8)
    per = -(-n // page)
    cache, k, v = ref.pool(g, fmt, B * hk * per, page, hk, D)
    pages = torch.randperm(B * hk * per, generator=g).view(B, hk, per).int()
    lens = torch.full((B,), n, dtype=torch.int32)
    q = torch.randn(B, 3 * hk, D, generator=g).to(ref.act(fmt)).cuda()
    of = lambda rows: lambda b, h: ref.context(rows, pages[b, h].tolist(), h, n)
    exact = attn_ref.attend(q, of(k), of(v), [n] * B, hk, D ** -0.5)
    call = lambda x=q: cache.attend_selected(x, pages.cuda(), lens.cuda(), return_lse=True)
    want, want_lse = call()
    assert held(want, want_lse, *exact, fmt)
    # where a page lies in another head's list it is none of this one's keys
    at = int(pages[0, 1, 2])
    if fmt in attn_ref.EMAX:
        old, old_v = cache.k_scale[at].clone(), cache.v_scale[at].clone()
        cache.k_scale[at, :, 3, 0] = 255
    else:
        old, old_v = cache.k[at].clone(), cache.v[at].clone()
        cache.k[at, :, 3, 0] = math.nan
    out, lse = call()
    assert out[0, 3:6].isnan().all() and lse[0, 3:6].isnan().all()
    out[0, 3:6], lse[0, 3:6] = want[0, 3:6], want_lse[0, 3:6]
    assert held(out, lse, *exact, fmt)
    if fmt in attn_ref.EMAX:
        # block sums past fp32's range whose scores are not: keys of 2^100 against 2^-100
        cache.k_scale[at] = old
        cache.k_scale[:, 1, :, :2] += 110
        kk = k.clone()
        kk[:, 1] *= 2.0 ** 110
        x = q.clone()
        x[:, 3:6] *= 2.0 ** -105
        exact = attn_ref.attend(x, of(kk), of(v), [n] * B, hk, D ** -0.5)
        assert held(*call(x), *exact, fmt)
    else:
        # -inf scores weigh nothing, a list of them gives zeros
        cache.k[at] = old
        cache.k[pages[1, 2].long(), 2] = -math.inf
        cache.k[int(pages[0, 0, 1]), 0] = -math.inf
        x = q.abs()
        out, lse = call(x)
        assert not out[1, 6:9].any() and (lse[1, 6:9] == -math.inf).all()
        def seen(rows):
            def f(b, h):
                y = of(rows)(b, h)
                return torch.cat([y[:16], y[32:]]) if (b, h) == (0, 0) else y
            return f
        exact = [attn_ref.attend(x[b:b + 1], lambda _, h: seen(k)(b, h), lambda _, h: seen(v)(b, h),
                                 [n], hk, D ** -0.5) for b in range(B)]
        exact = [torch.cat(y) for y in zip(*exact)]
        for y, z in zip((out, lse), exact):
            y[1, 6:9] = z[1, 6:9].to(y)
        assert held(out, lse, *exact, fmt)


# ---- eviction --------------------------------------------------------------------------------
@pytest.mark.parametrize("lens", [[300, 500, 40], [9000, 4000, 8500], [60000, 10, 55000]])
def test_evict_with_masses_of_any_alignment(lens):
    # masses 4 bytes past a 16-byte boundary; `into` that is the table itself
    g = ref.gen(*lens)
    page, keep = 48, 33
    n_pages = sum(-(-n // page) for n in lens)
    cache, _, _ = ref.pool(g, "bf16", n_pages, page, 2, 8)
    table = ref.tables(g, lens, page, n_pages)
    wide = torch.rand(n_pages * 2 * page + 3, generator=g).cuda()
    tl = torch.tensor(lens, dtype=torch.int32).cuda()
    runs = []
    for off in (0, 1, 3):
        flat = wide.clone()
        flat[off:off + n_pages * 2 * page] = wide[:n_pages * 2 * page]
        mass = flat[off:off + n_pages * 2 * page].view(n_pages, 2, page)
        pools = [cache.k.clone(), cache.v.clone()]
        t = table.cuda()
        kept, held_ = cache.evict(mass, t, tl, keep, first=2, recent=5, into=t if off else None)
        runs.append([kept, held_, mass.clone(), cache.k.clone(), cache.v.clone()])
        cache.k.copy_(pools[0]), cache.v.copy_(pools[1])
    for b, n in enumerate(lens):
        for h in range(2):
            m = [float(wide[(int(table[b, j // page]) * 2 + h) * page + j % page])
                 for j in range(min(n, 600))] if n <= 600 else \
                wide.cpu()[(table[b].long()[torch.arange(n) // page] * 2 + h) * page +
                           torch.arange(n) % page].tolist()
            want = ref.largest(m, keep, 2, 5)
            assert runs[0][0][b, h, :len(want)].tolist() == want
    for run in runs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(run, runs[0]))


# ---- streams ---------------------------------------------------------------------------------
@pytest.mark.parametrize("name", ["page_bounds", "evict", "evict into"])
def test_inputs_on_another_stream_are_not_given_away(name):
    n_pages, page, hk, D, B = 4096, 16, 4, 64, 512
    cache = moe.PagedKVCache(*[torch.ones(n_pages, hk, page, D, dtype=torch.bfloat16,
                                          device="cuda") for _ in range(2)], head_dim=D)
    side = torch.cuda.Stream()
    ids = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
    bounds, mass = cache.new_bounds(), cache.new_mass()

    def call(stream):
        # the tensor that is let go of
        if name == "page_bounds":
            x = torch.full((1 << 20,), -1, dtype=torch.int32, device="cuda")
            if stream is not None:
                stream.wait_stream(torch.cuda.current_stream())
            cache.page_bounds(bounds, x, torch.ones_like(x) if stream is None else fills,
                              stream=stream)
        else:
            x = torch.zeros(B, 512, dtype=torch.int32, device="cuda")
            if stream is not None:
                stream.wait_stream(torch.cuda.current_stream())
            cache.evict(mass, x, lens, 4, into=into if name == "evict into" else None,
                        stream=stream)
        return x.data_ptr(), x.numel()

    fills, lens, into = torch.ones(1 << 20, dtype=torch.int32, device="cuda"), ids(B), ids(B)[:, None]
    call(None)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    where, n = call(side)
    others = [torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(3)]
    assert all(o.data_ptr() != where for o in others)
    assert not side.query()
    torch.cuda.synchronize()


def test_bounds_and_evictions_on_another_stream():
    g = ref.gen(15)
    cache, k, _ = ref.pool(g, "bf16", 64, 16, 2, 64)
    side = torch.cuda.Stream()
    pages = torch.randperm(64, generator=g).int().cuda()
    fills = torch.full((64,), 16, dtype=torch.int32, device="cuda")
    want = cache.page_bounds(cache.new_bounds(), pages, fills)
    table, lens = pages[None].contiguous(), torch.tensor([1000], dtype=torch.int32, device="cuda")
    mass = torch.rand(64, 2, 16, generator=g).cuda()
    box = cache.new_bounds()
    torch.cuda.synchronize()
    cache.page_bounds(box, pages, fills, stream=side)
    kept, held_ = cache.evict(mass.clone(), table, lens, 100, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(box, want)
    m = mass.cpu()[pages.long().cpu()].permute(1, 0, 2).reshape(2, -1)[:, :1000]
    for h in range(2):
        assert kept[0, h].tolist() == ref.largest(m[h].tolist(), 100, 0, 0)
    assert held_.tolist() == [100]


# ---- refusals --------------------------------------------------------------------------------
def test_wrappers_refuse_numbers_of_more_than_32_bits():
    # taken modulo 2^32, each of them would pass for another one
    cache, q, pre, table, lens, _, _ = shared_case("bf16", 8, 2, 64, 4096, 300, [40, 20])
    bounds, mass = cache.new_bounds(), cache.new_mass()
    lse = torch.zeros(2, 8, device="cuda")
    pre = torch.zeros(2 ** 20 + 1, dtype=torch.int32, device="cuda")
    was = mass.clone()
    for call in (lambda: cache.attend_shared(q, pre, 2 ** 32 + 300, table, lens),
                 lambda: cache.select_pages(q, bounds, table, lens, 3, first=2 ** 32),
                 lambda: cache.select_pages(q, bounds, table, lens, 3, last=2 ** 32 + 1),
                 lambda: cache.accumulate(mass, q, table, lens, lse, window=2 ** 32 + 5),
                 lambda: cache.evict(mass, table, lens, 10, first=2 ** 32 + 1),
                 lambda: cache.evict(mass, table, lens, 10, recent=-2 ** 32 + 1)):
        with pytest.raises(ValueError):
            call()
    assert torch.equal(mass, was)


@pytest.mark.parametrize("fmt,D", [("bf16", 64), ("bf16", 128), ("mxfp8", 64), ("mxfp4", 128)])
@pytest.mark.parametrize("B", [161, 344, 370, 410])
def test_shared_prefix_of_many_row_tiles(B, fmt, D):
    # 6, 11, 12 and 13 tiles of 128 rows a key head, alone or in pairs
    cache, q, pre, table, lens, k_of, v_of = shared_case(fmt, 8, 2, D, 16, 700, [b % 3 for b in range(B)])
    want = attn_ref.attend(q, k_of, v_of, [700 + b % 3 for b in range(B)], 2, D ** -0.5)
    out, lse = cache.attend_shared(q, pre, 700, table, lens, return_lse=True)
    assert held(out, lse, *want, fmt)


def test_a_prefix_without_pages_is_refused():
    cache, q, pre, table, lens, _, _ = shared_case("bf16", 8, 2, 64, 16, 30, [4, 2])
    with pytest.raises(ValueError):
        cache.attend_shared(q, None, 30, table, lens)


# ---- outputs and pages -----------------------------------------------------------------------
@pytest.mark.parametrize("fmt,hq,hk,D", [("bf16", 16, 2, 64), ("bf16", 4, 4, 72), ("mxfp8", 16, 2, 64),
                                         ("bf16", 12, 1, 256), ("f32", 8, 2, 80), ("mxfp4", 4, 4, 96)])
def test_outputs_in_wider_rows(fmt, hq, hk, D):
    own = [40, 0, 700, 1, 16] * 3
    cache, q, pre, table, lens, _, _ = shared_case(fmt, hq, hk, D, 16, 333, own)
    pages, seen = cache.select_pages(q, cache.new_bounds(), table, lens, 4)
    for call in (lambda **kw: cache.attend_shared(q, pre, 333, table, lens, **kw),
                 lambda **kw: cache.attend_shared(q, None, 0, table, lens, **kw),
                 lambda **kw: cache.attend_selected(q, pages, seen, **kw)):
        want = call()
        wide = torch.full((len(own), hq + 3, D), 9.0, dtype=q.dtype, device="cuda")
        out, lse = call(out=wide[:, 1:1 + hq] if D * q.element_size() % 16 == 0 else wide[:, :hq],
                        return_lse=True)
        assert torch.equal(out, want) and out.data_ptr() != want.data_ptr()
        assert (wide[:, 0] == 9).all() and (wide[:, 1 + hq:] == 9).all()
        assert lse.shape == (len(own), hq)


@pytest.mark.parametrize("fmt", list(ref.FMT))
@pytest.mark.parametrize("B", [3, 40])
def test_own_and_chosen_pages_outside_the_pool_are_left_out(B, fmt):
    own, prefix = [60, 33, 0, 2000 if B == 3 else 90] * (B // 3), 100
    own = own[:B]
    cache, q, pre, table, lens, k_of, v_of = shared_case(fmt, 8, 2, 64, 16, prefix, own)
    bad = table.clone()
    n_pages = cache.k.shape[0]
    bad[0, 1], bad[1, 0] = n_pages, -5
    gone = {0: [prefix + j for j in range(16, 32)], 1: [prefix + j for j in range(16)]}

    def left(rows):
        def f(b, h):
            x = rows(b, h)
            keep = [j for j in range(len(x)) if j not in gone.get(b, [])]
            return x[keep]
        return f

    n = [prefix + m - len(gone.get(b, [])) for b, m in enumerate(own)]
    want = attn_ref.attend(q, left(k_of), left(v_of), n, 2, 0.125)
    got = cache.attend_shared(q, pre, prefix, bad, lens, return_lse=True)
    assert moe.coli_device_status() == moe.COLI_EDEVICE
    assert held(*got, *want, fmt)
    # the same for lists of each key head's own, and for lengths that are none
    only = [lambda b, h, r=r: left(r)(b, h)[prefix:] for r in (k_of, v_of)]
    want = attn_ref.attend(q, *only, [m - prefix for m in n], 2, 0.125)
    lists = bad[:, None].expand(-1, 2, -1).contiguous()
    out, lse = cache.attend_selected(q, lists, lens, return_lse=True)
    assert moe.coli_device_status() == moe.COLI_EDEVICE
    none = torch.isinf(want[1])
    assert torch.equal(torch.isinf(lse).cpu(), none) and not out[none.cuda()].any()
    lse[none.cuda()], want[1][none] = 0, 0
    assert held(out, lse, *want, fmt)
    odd = lens.clone()
    odd[0], odd[1] = -7, table.shape[1] * 16 + 1
    whole = table.clamp(min=0)
    fine = odd.clamp(0, table.shape[1] * 16)
    a = cache.attend_shared(q, pre, prefix, whole, fine, return_lse=True)
    p0, s0 = cache.select_pages(q, cache.new_bounds(), whole, fine, 3)
    m0 = cache.accumulate(cache.new_mass(), q, whole, fine, a[1])
    assert moe.coli_device_status() == moe.COLI_OK
    b = cache.attend_shared(q, pre, prefix, whole, odd, return_lse=True)
    assert moe.coli_device_status() == moe.COLI_EDEVICE
    p1, s1 = cache.select_pages(q, cache.new_bounds(), whole, odd, 3)
    assert moe.coli_device_status() == moe.COLI_EDEVICE
    m1 = cache.accumulate(cache.new_mass(), q, whole, odd, a[1])
    assert moe.coli_device_status() == moe.COLI_EDEVICE
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert torch.equal(p0, p1) and torch.equal(s0, s1)
    # (pages of several sequences: sums in any order)
    assert torch.allclose(m0, m1, rtol=2.0 ** -20, atol=0)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_decode_attention_of_the_least_key_scales(fmt):
    # keys of 2^-127 against queries of 2^77 under a scale that makes ordinary scores of them
    g = ref.gen(92)
    D, lens, scale = 64, [100, 17], 2.0 ** 47
    cache, _, v = ref.pool(g, fmt, 12, 16, 1, D)
    cache.k_scale[..., :2] = 0
    k = attn_ref.decode(cache.k, cache.k_scale, fmt)
    table = ref.tables(g, lens, 16, 12)
    q = (torch.randn(2, 4, D, generator=g) * 2.0 ** 76).bfloat16().cuda()
    tl = torch.tensor(lens, dtype=torch.int32).cuda()
    rows = [lambda b, h, x=x: ref.context(x, table[b].tolist(), h, lens[b]) for x in (k, v)]
    want = list(attn_ref.attend(q, *rows, lens, 1, scale))
    # scores lie hundreds apart: a weight below 2^-126, the least normal fp32 number, may count as
    # 0, which is worth 2^-126 sum |v| at most (e^-124 here is 2^-179, an output of 3.6e-54)
    want[2] = want[2] + 2.0 ** -126 * torch.stack(
        [rows[1](b, 0).abs().sum(0) for b in range(2)])[:, None]
    assert held(*cache.attend(q, table.cuda(), tl, scale=scale, return_lse=True), *want, fmt)
    assert held(*cache.attend_selected(q, table[:, None].contiguous().cuda(), tl, scale=scale,
                                       return_lse=True), *want, fmt)


# ---- captured calls --------------------------------------------------------------------------
@pytest.mark.parametrize("before", ["nothing", "memset", "copy", "fork"])
def test_calls_captured_behind_other_work(before):
    # each call as the first of a graph, or behind a node that is no kernel
    own = [50, 0, 130, 16] * 10
    cache, q, pre, table, lens, _, _ = shared_case("bf16", 16, 4, 64, 16, 333, own)
    g = ref.gen(17)
    bounds = cache.new_bounds()
    bounds.copy_(torch.randn(bounds.shape, generator=g).sort(2).values)
    table = table.clamp(min=0)
    mass = torch.rand(cache.new_mass().shape, generator=g).cuda()
    some, host = torch.empty(1 << 20, device="cuda"), torch.empty(1 << 20).pin_memory()
    calls = {
        "all": lambda: cache.select_pages(q, bounds, table, lens, table.shape[1]),
        "few": lambda: cache.select_pages(q, bounds, table, lens, 3),
        "shared": lambda: cache.attend_shared(q, pre, 333, table, lens, return_lse=True),
        "selected": lambda: cache.attend_selected(q, table[:, None].expand(-1, 4, -1).contiguous(),
                                                  lens, return_lse=True),
        "evict": lambda: cache.evict(mass, table, lens.clamp(max=12), 12)}
    for name, call in calls.items():
        want = call()
        torch.cuda.synchronize()
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph):
            if before == "memset":
                some.zero_()
            elif before == "copy":
                some.copy_(host, non_blocking=True)
            elif before == "fork":
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    some.add_(1)
                torch.cuda.current_stream().wait_stream(side)
            got = call()
        for _ in range(2):
            for x in got:
                x.fill_(5)
            graph.replay()
            assert all(torch.equal(x, y) for x, y in zip(got, want)), name
