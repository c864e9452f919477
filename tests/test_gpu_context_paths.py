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
