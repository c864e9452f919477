"""Shared prefixes, chosen pages and eviction at the ends of their sizes (GPU)."""
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
    torch.cuda.empty_cache()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def every_call(cache, q, pre, table, lens, into):
    """Results of one of each on a pool whose pages hold something already."""
    prefix = pre.numel() * cache.page_size - 3
    out = list(cache.attend_shared(q, pre, prefix, table, lens, return_lse=True))
    used = table.flatten().contiguous()
    bounds = cache.new_bounds()
    cache.page_bounds(bounds, used, torch.full_like(used, cache.page_size))
    pages, seen = cache.select_pages(q, bounds, table, lens, 3)
    out += [bounds[used.long()], seen]
    out += list(cache.attend_selected(q, pages, seen, return_lse=True))
    mass = cache.new_mass()
    cache.accumulate(mass, q, table, lens, out[1])
    out.append(mass[used.long()])
    kept, left = cache.evict(mass, table, lens, 40, recent=2, into=into)
    rows = [cache.k, cache.v] + ([cache.k_scale, cache.v_scale] if cache.k_scale is not None else [])
    out += [kept, left, mass[into.flatten().long()]] + [x[into.flatten().long()] for x in rows]
    cache.evict(mass, into, left, 20, first=1)
    return out + [mass[into.flatten().long()]] + [x[into.flatten().long()] for x in rows]


@pytest.mark.parametrize("fmt,hk", [("bf16", 8), ("mxfp8", 16), ("f32", 4)])
def test_pools_past_4_gib(fmt, hk):
    """Byte offsets past 2^32 in keys, values and bounds' pages, on a pool whose first page
    would stand in for a wrapped offset: the same bits as on a small one."""
    D, page, B = 128, 64, 12
    g = ref.gen(hk, 3)
    n_small = 4 + B * 6
    small, _, _ = ref.pool(g, fmt, n_small, page, hk, D)
    n_big = (1 << 32) // (small.k[0].numel() * small.k.element_size()) + 200
    big = moe.PagedKVCache(*[None if x is None else torch.zeros(n_big, *x.shape[1:], dtype=x.dtype,
                                                                device="cuda")
                             for x in (small.k, small.v, small.k_scale, small.v_scale)], head_dim=D)
    move = torch.arange(n_small, device="cuda") + (n_big - n_small)
    for x, y in ((big.k, small.k), (big.v, small.v), (big.k_scale, small.k_scale),
                 (big.v_scale, small.v_scale)):
        if y is not None:
            x[move] = y
    ids = torch.randperm(n_small, generator=g).int().cuda()
    pre, table, into = ids[:4], ids[4:4 + B * 5].view(B, 5).contiguous(), ids[4 + B * 5:].view(B, 1)
    lens = torch.randint(0, 5 * page + 1, (B,), generator=g).int().cuda()
    q = torch.randn(B, 4 * hk, D, generator=g).to(ref.act(fmt)).cuda()
    to = n_big - n_small
    want = every_call(small, q, pre, table, lens, into.contiguous())
    got = every_call(big, q, pre + to, table + to, lens, (into + to).contiguous())
    assert len(got) == len(want)
    for x, y in zip(got, want):
        if x.is_floating_point():
            x, y = x.nan_to_num(7), y.nan_to_num(7)
        assert torch.equal(x, y)
    if fmt != "mxfp8":
        assert not big.k[:200].any() and not big.v[:200].any()


def test_the_most_sequences():
    """65535 sequences, short ones, in one call."""
    B, hq, hk, D, page, keep = 65535, 4, 2, 32, 16, 9
    g = torch.Generator(device="cuda").manual_seed(5)
    n_pages, n_pre = B + 13, 13
    pools = [torch.randn(n_pages, hk, page, D, generator=g, device="cuda").bfloat16()
             for _ in range(2)]
    cache = moe.PagedKVCache(*pools, head_dim=D)
    q = torch.randn(B, hq, D, generator=g, device="cuda").bfloat16()
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    pre, table = order[:n_pre].contiguous(), order[n_pre:].view(B, 1).contiguous()
    lens = torch.randint(0, page + 1, (B,), generator=g, device="cuda").int()
    out, lse = cache.attend_shared(q, pre, 200, table, lens, return_lse=True)
    k, v = (x.double() for x in pools)
    qd = q.double().view(B, hk, 2, D)
    ctx = [torch.cat([x[pre.long()].transpose(0, 1).reshape(hk, -1, D)[:, :200].expand(
        B, hk, 200, D), x[table[:, 0].long()]], 2) for x in (k, v)]
    s = torch.einsum("bhgd,bhnd->bhgn", qd, ctx[0]) * D ** -0.5
    seen = torch.arange(216, device="cuda") < 200 + lens[:, None]
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    p = torch.softmax(s, -1)
    want = torch.einsum("bhgn,bhnd->bhgd", p, ctx[1]).view(B, hq, D)
    mag = torch.einsum("bhgn,bhnd->bhgd", p, ctx[1].abs()).view(B, hq, D)
    # scores: 36 2^-22 of at most 60; weights 2^-16, the output's rounding
    assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -9 * mag).all()
    assert ((lse.double() - torch.logsumexp(s, -1).view(B, hq)).abs() <= 2.0 ** -10).all()
    del ctx, want, mag
    # own tokens alone: their masses, and the heaviest of them
    out, lse = cache.attend(q, table, lens, return_lse=True)
    mass = cache.accumulate(cache.new_mass(), q, table, lens, lse)
    w = torch.softmax(s[..., 200:], -1).nan_to_num(0).sum(2)
    assert ((mass[table[:, 0].long()].double() - w).abs() <= 2.0 ** -10 * w + 1e-30).all()
    one = mass[table[:, 0].long()]
    kept, left = cache.evict(mass, table, lens, keep, first=1, recent=2)
    assert torch.equal(left, lens.clamp(max=keep))
    at = torch.arange(page, device="cuda")
    key = one.masked_fill((at >= lens[:, None])[:, None], -math.inf)
    key = key.masked_fill(((at < 1) | (at >= lens[:, None] - 2))[:, None] &
                          (at < lens[:, None])[:, None], math.inf)
    pick = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :keep].sort(-1).values
    cut = lens > keep
    assert torch.equal(kept[cut], pick.int()[cut])
    assert (kept[~cut] == torch.where(at[:keep] < lens[~cut, None], at[:keep], -1)[:, None]).all()
    # and the better one of two pages, before the last
    bounds = cache.new_bounds()
    cache.page_bounds(bounds, order, torch.full_like(order, page))
    three = torch.randint(0, n_pages, (B, 3), generator=g, device="cuda").int()
    pages, seen = cache.select_pages(q, bounds, three, torch.full_like(lens, 3 * page - 4), 2,
                                     first=0)
    box = bounds.double()[three.long()]
    s = (torch.einsum("bhgd,bphd->bhgp", qd.clamp(min=0), box[:, :, :, 1]) +
         torch.einsum("bhgd,bphd->bhgp", qd.clamp(max=0), box[:, :, :, 0])).amax(2)
    best = torch.where(s[..., 1] > s[..., 0], three[:, 1:2], three[:, :1])
    assert (seen == 2 * page - 4).all()
    assert torch.equal(pages, torch.stack([best, three[:, 2:].expand(-1, hk)], -1))


@pytest.mark.parametrize("fmt", list(ref.FMT))
@pytest.mark.parametrize("hq,hk,D", [(1024, 1, 64), (1024, 256, 32), (1000, 8, 128)])
def test_the_most_heads(hq, hk, D, fmt):
    B, page, prefix = 2, 16, 150
    g = ref.gen(hq, hk, D)
    lens, n_pages = [77, 40], 10 + 10
    cache, k, v = ref.pool(g, fmt, n_pages, page, hk, D)
    pre = torch.arange(10, dtype=torch.int32)
    table = ref.tables(g, lens, page, n_pages, range(10))
    q = torch.randn(B, hq, D, generator=g).to(ref.act(fmt)).cuda()
    both = lambda rows: lambda b, h: torch.cat([ref.context(rows, pre.tolist(), h, prefix),
                                                ref.context(rows, table[b].tolist(), h, lens[b])])
    want, want_lse, tol, tol_lse = attn_ref.attend(q, both(k), both(v), [prefix + n for n in lens],
                                                   hk, D ** -0.5)
    tl = ints(lens)
    out, lse = cache.attend_shared(q, pre.cuda(), prefix, table.cuda(), tl, return_lse=True)
    step = 2.0 ** -24 if fmt == "f32" else 2.0 ** -8
    assert ((out.cpu().double() - want).abs() <= tol * (1 + step) + step * want.abs()).all()
    assert ((lse.cpu().double() - want_lse).abs() <= tol_lse).all()
    mass = cache.accumulate(cache.new_mass(), q, table.cuda(), tl, lse).cpu().double()
    bounds = cache.new_bounds()
    used = table.flatten()[table.flatten() >= 0].contiguous().cuda()
    cache.page_bounds(bounds, used, torch.full_like(used, page))
    pages, _ = cache.select_pages(q, bounds, table.cuda(), tl, 2)
    G, qd, box = hq // hk, q.double().cpu(), bounds.double().cpu()
    for b, n in enumerate(lens):
        at = table[b].long()[torch.arange(n) // page]
        for h in range(0, hk, 17 if hk > 8 else 1):
            r = slice(h * G, (h + 1) * G)
            w, t = ref.mass(qd[b, r], k[at, h, torch.arange(n) % page], lse[b, r].double().cpu(),
                            D ** -0.5)
            got = mass[at, h, torch.arange(n) % page]
            # sums of up to 1024 weights, 8 or 16 at a time
            assert ((got - w).abs() <= t + (1 + G // 8) * 2.0 ** -24 * w).all()
            count = -(-n // page)
            s = torch.stack([(qd[b, r].clamp(min=0) @ box[p, h, 1] +
                              qd[b, r].clamp(max=0) @ box[p, h, 0]).amax()
                             for p in table[b, :count].tolist()])
            best = [int(table[b, j]) for j in ref.largest(s.tolist(), 2, 1, 1)]
            assert pages[b, h].tolist() == best
