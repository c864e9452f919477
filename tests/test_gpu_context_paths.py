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
