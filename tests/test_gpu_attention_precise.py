"""Decode attention held to what each format's arithmetic admits, and every tile of a
context counted once (GPU)."""
import os
import sys

import pytest
import torch

import mixture_experts_gb300 as moe

sys.path.insert(0, os.path.dirname(__file__))
import attn_bound as ab  # noqa: E402

pytestmark = pytest.mark.gpu

FMT = {"f32": moe.F32, "bf16": moe.BF16, "mxfp8": moe.MXFP8, "mxfp4": moe.MXFP4}


@pytest.fixture(scope="module", autouse=True)
def built():
    moe.build()
    assert torch.cuda.is_available()


@pytest.fixture(autouse=True)
def clean_status():
    assert moe.coli_device_status() == moe.COLI_OK
    yield
    assert moe.coli_device_status() == moe.COLI_OK


def pool(fmt, k, v, lens, page, seed):
    """k, v [tokens][heads][D], sequence after sequence -> (cache, table, lengths), pages in no
    order and full of NaN past each context's end."""
    g = torch.Generator().manual_seed(seed)
    per = [-(-n // page) for n in lens]
    c = moe.PagedKVCache.empty(sum(per) + 2, page, k.shape[1], k.shape[2], FMT[fmt])
    for x in (c.k, c.v, c.k_scale, c.v_scale):
        if x is not None:
            x.view(torch.uint8).fill_(0xff)
    order = torch.randperm(sum(per) + 2, generator=g)
    table = torch.full((len(lens), max(1, max(per))), -1, dtype=torch.int32)
    slots, at = [], 0
    for b, n in enumerate(lens):
        ids = order[at:at + per[b]]
        at += per[b]
        table[b, :per[b]] = ids.int()
        j = torch.arange(n)
        slots.append(ids[j // page] * page + j % page)
    c.append(k.cuda(), v.cuda(), torch.cat(slots).int().cuda())
    return c, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("case", ab.CASES)
def test_within_what_the_format_admits(case, fmt):
    lens, hq, hk, D, page = case
    q, k, v = ab.inputs(case, fmt)
    c, table, sl = pool(fmt, k, v, lens, page, seed=D)
    got, lse = (x.cpu().double() for x in c.attend(q.cuda(), table, sl, return_lse=True))
    k, v = ab.stored(k, fmt), ab.stored(v, fmt)
    at, g = 0, hq // hk
    for b, n in enumerate(lens):
        for h in range(hk):
            r = slice(h * g, (h + 1) * g)
            out, want, tol, tol_lse = ab.bound(fmt, q[b, r].double(), k[at:at + n, h],
                                               v[at:at + n, h], D ** -0.5)
            assert ((got[b, r] - out).abs() <= tol).all()
            assert ((lse[b, r] - want).abs() <= tol_lse).all()
        at += n


def ragged(n, top):
    g = torch.Generator().manual_seed(n)
    return (torch.rand(n, generator=g) ** 2 * top).int().tolist()


MARKED = [  # lens, query heads, key heads, head_dim, page, window
    ([60001], 6, 2, 64, 64, 0), ([60001], 16, 1, 128, 16, 0), ([20011], 20, 1, 256, 48, 0),
    ([30000, 0, 1, 17, 9000, 16], 8, 2, 128, 32, 0), (ragged(40, 5000), 12, 4, 64, 16, 0),
    (ragged(40, 5000), 12, 4, 64, 16, 777), ([70000, 3], 4, 4, 64, 128, 4097),
    (ragged(300, 1500), 8, 1, 64, 16, 0), (ragged(150, 600), 16, 1, 128, 16, 33),
    (ragged(20, 1000), 40, 2, 64, 32, 0)]


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("lens,hq,hk,D,page,window", MARKED)
def test_every_tile_counts_once(lens, hq, hk, D, page, window, fmt):
    """Equal weights (scale 0), tile t of a sequence marked by a 1 in channel t % head_dim:
    a channel's output is its share of the keys in sight."""
    g = torch.Generator().manual_seed(3)
    dt = torch.float32 if fmt == "f32" else torch.bfloat16
    n = sum(lens)
    k = torch.randn(n, hk, D, generator=g).to(dt)
    v = torch.zeros(n, hk, D, dtype=dt)
    v[torch.arange(n), :, torch.cat([torch.arange(x) // 16 % D for x in lens])] = 1.0
    c, table, sl = pool(fmt, k, v, lens, page, seed=7)
    q = torch.randn(len(lens), hq, D, generator=g).to(dt).cuda()
    got, lse = (x.cpu().double() for x in
                c.attend(q, table, sl, scale=0.0, window=window, return_lse=True))
    for b, n in enumerate(lens):
        first = max(0, n - window) if window else 0
        if n == 0:
            assert not got[b].any() and (lse[b] == -torch.inf).all()
            continue
        out = torch.bincount(torch.arange(first, n) // 16 % D, minlength=D).double() / (n - first)
        tol, tol_lse = ab.flat_bound(fmt, out, n - first)
        assert ((got[b] - out).abs() <= tol).all()
        assert ((lse[b] - ab.log_of(n - first)).abs() <= tol_lse).all()


LEFT_OUT = ["first", "last", "run", "alternate", "third", "all but one", "all"]


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("B,hq,hk,D,page,n,window", [
    (1, 4, 1, 64, 16, 12000, 0), (1, 32, 2, 128, 32, 12000, 0), (3, 6, 2, 256, 16, 5000, 0),
    (96, 16, 8, 64, 16, 9000, 0), (64, 32, 2, 128, 64, 9000, 2500), (20, 8, 2, 64, 48, 900, 0)])
def test_left_out_pages_anywhere(B, hq, hk, D, page, n, window, fmt):
    """Pages outside the pool at the ends of long contexts, in runs longer than a block's
    piece, every second one: only they are missing, also where a warp takes more than 32 tiles.
    All sequences draw from the same pages, whose tiles are marked as above."""
    g = torch.Generator().manual_seed(B + n)
    dt = torch.float32 if fmt == "f32" else torch.bfloat16
    pages, per = 90, -(-n // page)
    c = moe.PagedKVCache.empty(pages, page, hk, D, FMT[fmt])
    j = torch.arange(pages * page)
    v = torch.zeros(len(j), hk, D, dtype=dt)
    v[j, :, j // 16 % D] = 1.0
    c.append(torch.randn(len(j), hk, D, generator=g).to(dt).cuda(), v.cuda(), j.int().cuda())
    table = torch.randint(0, pages, (B, per), generator=g).int()
    lens = n - torch.arange(B) * 7 % 50
    bad = torch.tensor([pages, -1, -7, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    for b in range(B):
        at = torch.arange(per)
        kind = LEFT_OUT[b % len(LEFT_OUT)] if B > 1 else "run"
        out = {"first": at < 3, "last": at >= per - 2, "run": (at > per // 5) & (at < per // 2),
               "alternate": at % 2 == 1, "third": at % 3 == b % 3, "all but one": at != per - 2,
               "all": at >= 0}[kind]
        table[b] = torch.where(out, bad[(at + b) % len(bad)], table[b])
    q = torch.randn(B, hq, D, generator=g).to(dt).cuda()
    got, lse = (x.cpu().double() for x in c.attend(
        q, table.cuda(), lens.int().cuda(), scale=0.0, window=window, return_lse=True))
    assert moe.coli_device_status() == moe.COLI_EDEVICE
    for b in range(B):
        m = int(lens[b])
        key = torch.arange(max(0, m - window) if window else 0, m)
        at = table[b, key // page].long()
        key, at = key[(at >= 0) & (at < pages)], at[(at >= 0) & (at < pages)]
        if len(key) == 0:
            assert not got[b].any() and (lse[b] == -torch.inf).all()
            continue
        out = torch.bincount((at * page + key % page) // 16 % D, minlength=D).double() / len(key)
        tol, tol_lse = ab.flat_bound(fmt, out, m)
        assert ((got[b] - out).abs() <= tol).all()
        assert ((lse[b] - ab.log_of(len(key))).abs() <= tol_lse).all()
