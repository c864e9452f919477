"""Rotary positions, the paged key-value cache and its decode attention
against their plain 64-bit forms (GPU)."""
import math
import os
import sys

import pytest
import torch

import mixture_experts_gb300 as moe

sys.path.insert(0, os.path.dirname(__file__))
import attn_ref  # noqa: E402

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


def act(fmt):
    return torch.float32 if fmt == "f32" else torch.bfloat16


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def gen(*key):
    return torch.Generator().manual_seed(sum((i + 1) * 7919 * int(k) for i, k in enumerate(key)))


# ---- rotary ---------------------------------------------------------------------------
@pytest.mark.parametrize("rot,n,base,scaling,factor,orig", [
    (2, 5, 10000.0, 0, 1.0, 0), (64, 1000, 10000.0, 0, 1.0, 0), (128, 700, 1e6, 1, 8.0, 0),
    (20, 333, 500.0, 2, 4.0, 0), (128, 400, 10000.0, 3, 16.0, 4096), (256, 17, 5e5, 3, 2.0, 100)])
def test_rope_table(rot, n, base, scaling, factor, orig):
    amp = 0.1 * math.log(factor) + 1
    r = moe.Rotary.build(rot, n, base=base, scaling=scaling, factor=factor,
                         original_positions=orig, amplitude=amp)
    a = attn_ref.rope_angles(n, rot, base, scaling, factor, orig)
    want = torch.stack([a.cos(), a.sin()], -1) * amp
    # rounded once to fp32 (2^-24 amp), and the fp64 angle's own error: a few
    # 2^-52 of the angle
    tol = 2.0 ** -24 * amp + a[..., None] * 2.0 ** -48
    assert ((r.table.cpu().double() - want).abs() <= tol).all()


def test_rope_table_far_positions():
    # the angle is formed in fp64: a position near 10^6 is as exact as a small one
    n = 1_000_003
    r = moe.Rotary.build(4, n)
    a = attn_ref.rope_angles(n, 4)[-1000:]
    want = torch.stack([a.cos(), a.sin()], -1)
    assert ((r.table[-1000:].cpu().double() - want).abs() <= 2.0 ** -24 + 2.0 ** -28).all()


ROPE_CASES = [(1, 1, 0, 8, 8), (3, 4, 2, 64, 64), (7, 5, 1, 80, 20), (33, 12, 4, 96, 48),
              (5, 8, 8, 128, 128), (130, 32, 8, 128, 64), (2, 3, 3, 256, 256), (9, 2, 1, 72, 72),
              (4, 6, 2, 16, 2), (1500, 8, 2, 64, 32), (1201, 16, 4, 40, 22)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,hq,hk,D,rot", ROPE_CASES)
def test_rope(T, hq, hk, D, rot, layout, dtype):
    g = gen(T, hq, D, rot)
    n = 5000
    r = moe.Rotary(moe.Rotary.build(rot, n).table, layout)
    qkv = randn(g, T, (hq + 2 * hk + 1) * D, dtype=dtype)
    cut = qkv.unflatten(-1, (-1, D))
    q, k = cut[:, :hq], cut[:, hq:hq + hk]          # token stride beyond the heads' own
    pos = torch.randint(0, n, (T,), generator=g).int().cuda()
    qo, ko = moe.rope(r, pos, q, k if hk else None)
    for x, got in ((q, qo), (k, ko)):
        if got is None:
            continue
        want, mag = attn_ref.rotate(x, r.table, pos, layout)
        # two products and their sum, each rounded in fp32, then the output type
        tol = 2 * 2.0 ** -24 * mag + 2.0 ** -24 * want.abs()
        if dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * want.abs()
        assert got.dtype == dtype and ((got.cpu().double() - want).abs() <= tol).all()
        # elements past rot_dim are the input's bits
        assert torch.equal(got[..., rot:], x[..., rot:])
    # in place gives the same bits, and writes nothing beside the heads
    rest = cut[:, hq + hk:].clone()
    moe.rope(r, pos, q, k if hk else None, q_out=q, k_out=k if hk else None)
    assert torch.equal(q, qo) and (not hk or torch.equal(k, ko))
    assert torch.equal(cut[:, hq + hk:], rest)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_inverse_is_its_gradient(layout):
    g = gen(11, 3)
    T, h, D, rot, n = 19, 3, 64, 48, 300
    r = moe.Rotary(moe.Rotary.build(rot, n).table, layout)
    pos = torch.randint(0, n, (T,), generator=g).int().cuda()
    x, dy = randn(g, T, h, D), randn(g, T, h, D)
    dx, _ = moe.rope(r, pos, dy, inverse=True)
    want, mag = attn_ref.rotate(dy, r.table, pos, layout, inverse=True)
    assert ((dx.cpu().double() - want).abs() <= 3 * 2.0 ** -24 * mag).all()
    # against differences: the map is linear, so f(x + e) - f(x) = f(e) up to
    # fp32 rounding of values below 8
    u = randn(g, T, h, D)
    y0, _ = moe.rope(r, pos, x)
    y1, _ = moe.rope(r, pos, x + u)
    lhs = ((y1.double() - y0.double()) * dy.double()).sum()
    rhs = (u.double() * dx.double()).sum()
    assert abs(float(lhs - rhs)) <= T * h * D * 8 * 2.0 ** -23 * float(dy.abs().max())
    # and back again
    back, _ = moe.rope(r, pos, y0, inverse=True)
    assert ((back - x).abs() <= 16 * 2.0 ** -24 * x.abs().max()).all()


def test_rope_bad_positions_are_copied_and_latched():
    g = gen(5)
    r = moe.Rotary.build(64, 50)
    q = randn(g, 6, 4, 64, dtype=torch.bfloat16)
    pos = torch.tensor([0, 49, 50, -1, 2 ** 31 - 1, 7], dtype=torch.int32).cuda()
    out, _ = moe.rope(r, pos, q)
    assert moe.coli_device_status() == moe.COLI_EDEVICE
    assert torch.equal(out[2:5], q[2:5]) and torch.equal(out[0], q[0])
    assert not torch.equal(out[1], q[1]) and not torch.equal(out[5], q[5])


# ---- cache ------------------------------------------------------------------------------
def pools(c):
    return [x for x in (c.k, c.v, c.k_scale, c.v_scale) if x is not None]


def stored(c, slots, side):
    """The raw rows (codes, scales or None) of slots, [N][heads][..] on the CPU."""
    page, off = slots // c.page_size, slots % c.page_size
    codes, scales = (c.k, c.k_scale) if side == "k" else (c.v, c.v_scale)
    s = None if scales is None else scales[page, :, off].cpu()
    return codes[page, :, off].cpu(), s


CACHE_CASES = [(1, 1, 64, 16, 3), (5, 2, 96, 16, 4), (33, 8, 128, 48, 5), (100, 4, 64, 32, 9),
               (260, 3, 256, 64, 8), (2600, 4, 128, 128, 24)]


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("T,hk,D,page,pages", CACHE_CASES)
@pytest.mark.parametrize("rope", ["none", "half", "interleaved"])
def test_append_and_read(T, hk, D, page, pages, fmt, rope):
    g = gen(T, hk, D, page)
    c = moe.PagedKVCache.empty(pages, page, hk, D, FMT[fmt])
    for p in pools(c):
        p.view(torch.uint8).fill_(0x5a)             # what must stay as it is
    before = [p.clone() for p in pools(c)]
    hq = 2 * hk
    dt = act(fmt)
    qkv = randn(g, T, (hq + 2 * hk) * D, dtype=torch.float32)
    qkv = (qkv * torch.exp2(torch.randint(-6, 6, (T, 1), generator=g).float()).cuda()).to(dt)
    cut = qkv.unflatten(-1, (-1, D))
    q, k, v = cut[:, :hq], cut[:, hq:hq + hk], cut[:, hq + hk:]
    slots = torch.randperm(pages * page, generator=g)[:T].int()
    skip = torch.arange(T) % 7 == 3
    sent = torch.where(skip, -1, slots).int().cuda()
    rows = slots[~skip].cuda()
    if rope == "none":
        c.append(k, v, sent)
        k32 = k.float().cpu()
    else:
        r = moe.Rotary(moe.Rotary.build(D // 2 if T % 2 else D, 900).table, rope)
        pos = torch.randint(0, 900, (T,), generator=g).int().cuda()
        qo = c.append(k, v, sent, rotary=r, positions=pos, q=q)
        assert torch.equal(qo, moe.rope(r, pos, q)[0])
        k32 = attn_ref.rotate32(k, r.table, pos, rope)
    for side, x in (("k", k32), ("v", v.float().cpu())):
        codes, scales = stored(c, rows, side)
        x = x[~skip]
        if fmt in ("f32", "bf16"):
            assert torch.equal(codes, x.to(dt))     # bit for bit
        else:
            want_c, want_s = attn_ref.quantise(x, fmt)
            assert torch.equal(scales[..., :D // 32], want_s)
            assert torch.equal(codes, want_c)
        got = c.read(sent)[0 if side == "k" else 1]
        back = attn_ref.decode(codes, scales, fmt)
        assert torch.equal(got[~skip.cuda()].cpu().double(), back.to(dt).double())
        assert not got[skip.cuda()].any()
    # nothing else in the pools has changed
    c2 = [p.clone() for p in pools(c)]
    page_i, off = (rows // page).long(), (rows % page).long()
    for now, old in zip(c2, before):
        used = D // 32 if now.dtype == torch.uint8 and now.shape[-1] not in (D, D // 2) else \
            now.shape[-1]
        now[page_i, :, off, :used] = old[page_i, :, off, :used] if used != now.shape[-1] else \
            old[page_i, :, off]
        assert torch.equal(now.view(torch.uint8), old.view(torch.uint8))


def test_read_one_side_and_bad_slots():
    g = gen(8)
    c = moe.PagedKVCache.empty(4, 16, 2, 64, moe.MXFP8)
    k, v = randn(g, 64, 2, 64, dtype=torch.bfloat16), randn(g, 64, 2, 64, dtype=torch.bfloat16)
    c.append(k, v, torch.arange(64).int().cuda())
    slots = torch.tensor([5, 64, -1, -2, 63], dtype=torch.int32).cuda()
    out = torch.full((5, 3 * 128), 7.0, dtype=torch.bfloat16, device="cuda")
    # one output only, its rows wider than the heads
    assert moe.coli_kv_read(c.c, slots, 5, None, 0, out[:, 128:], 384) == moe.COLI_OK
    assert moe.coli_device_status() == moe.COLI_EDEVICE     # 64 and -2
    both = c.read(torch.tensor([5, 63], dtype=torch.int32).cuda())[1]
    assert torch.equal(out[[0, 4], 128:256].reshape(2, 2, 64), both)
    assert not out[1:4, 128:256].any() and (out[:, :128] == 7).all() and (out[:, 256:] == 7).all()


def test_append_bad_slots_and_positions_are_skipped_and_latched():
    g = gen(9)
    c = moe.PagedKVCache.empty(2, 16, 2, 64, moe.BF16)
    r = moe.Rotary.build(64, 10)
    k, q = (randn(g, 4, 2, 64, dtype=torch.bfloat16) for _ in range(2))
    slots = torch.tensor([3, 32, -5, 7], dtype=torch.int32).cuda()
    pos = torch.tensor([1, 2, 3, 10], dtype=torch.int32).cuda()
    qo = c.append(k, k, slots, rotary=r, positions=pos, q=q)
    assert moe.coli_device_status() == moe.COLI_EDEVICE
    assert torch.equal(qo[3], q[3])
    used = c.k.abs().sum(dim=(1, 3)).reshape(-1).cpu()
    assert used[3] > 0 and used[:3].sum() + used[4:].sum() == 0


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_quantiser_edges(fmt):
    """Zeros of both signs, subnormals, the largest values, ties, NaN and infinity."""
    D = 64
    x = torch.zeros(10, 1, D)
    x[1] = -0.0
    x[2, 0, :32] = 2.0 ** -133                       # below the smallest scale times emax
    x[2, 0, 32:] = torch.linspace(-1, 1, 32) * 2.0 ** -126
    x[3] = torch.linspace(-3.38e38, 3.38e38, D)
    x[4] = torch.linspace(-7.75, 7.75, D)            # every tie of E2M1
    x[5] = torch.arange(D) * 8.0                     # E4M3 ties, and 448 < |x| < 512
    x[6, 0, 5] = math.nan
    x[7, 0, 40] = -math.inf
    x[8, 0, 0] = 1.0
    x[9] = torch.tensor([2.0 ** -i for i in range(D)])
    x = x.bfloat16()
    c = moe.PagedKVCache.empty(1, 16, 1, D, FMT[fmt])
    slots = torch.arange(10).int().cuda()
    c.append(x.cuda(), x.cuda(), slots)
    want_c, want_s = attn_ref.quantise(x.float(), fmt)
    codes, scales = stored(c, slots.long(), "v")
    assert torch.equal(scales[..., :2], want_s) and torch.equal(codes, want_c)
    got = c.read(slots)[0].cpu()
    assert got[6, 0, :32].isnan().all() and got[7, 0, 32:].isnan().all()
    want = attn_ref.decode(want_c, want_s, fmt).bfloat16()
    assert torch.equal(got.nan_to_num(3.0), want.nan_to_num(3.0))


# ---- attention ---------------------------------------------------------------------------
def make_context(fmt, lens, hk, D, page, seed, spare=2, k_amp=1.0):
    """A pool holding contexts of the given lengths in scattered pages. What
    lies past each context's end is NaN (f32, bf16) or NaN codes and scales."""
    g = gen(seed, hk, D, page, len(lens))
    per = [-(-n // page) for n in lens]
    pages = sum(per) + spare
    c = moe.PagedKVCache.empty(pages, page, hk, D, FMT[fmt])
    for p in pools(c):
        p.view(torch.uint8).fill_(0xff)              # NaN in every format
    order = torch.randperm(pages, generator=g)
    table = torch.full((len(lens), max(1, max(per))), -1, dtype=torch.int32)
    at = 0
    slots = []
    for b, n in enumerate(lens):
        ids = order[at:at + per[b]]
        at += per[b]
        table[b, :per[b]] = ids.int()
        j = torch.arange(n)
        slots.append(ids[j // page] * page + j % page)
    slots = torch.cat(slots)
    total = max(1, len(slots))
    k = randn(g, total, hk, D) * k_amp
    k = k * torch.exp(0.5 * randn(g, 1, hk, D))
    v = randn(g, total, hk, D) * torch.exp2(torch.randint(-3, 3, (total, hk, 1),
                                                         generator=g).float()).cuda()
    if len(slots):
        c.append(k.to(act(fmt)), v.to(act(fmt)), slots.int().cuda())
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    dec = {}
    for side in "kv":
        codes, scales = stored(c, slots.cuda().long(), side)
        dec[side] = attn_ref.decode(codes, scales, fmt)
    rows = {s: (lambda b, h, s=s: dec[s][starts[b]:starts[b + 1], h]) for s in "kv"}
    return c, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), rows, g


def check(got, lse, ref, fmt):
    want, want_lse, tol, tol_lse = ref
    if fmt != "f32":
        tol = tol + 2.0 ** -8 * want.abs()
    else:
        tol = tol + 2.0 ** -23 * want.abs()
    got, lse = got.cpu().double(), lse.cpu().double()
    assert ((got - want).abs() <= tol).all(), float(((got - want).abs() - tol).max())
    empty = torch.isinf(want_lse)
    assert torch.equal(torch.isinf(lse), empty) and (lse[empty] < 0).all()
    assert ((lse - want_lse).abs()[~empty] <= tol_lse[~empty]).all()
    assert not got[empty].any()


ATTN_CASES = [
    # lens, hq, hk, D, page, window
    ([1], 1, 1, 64, 16, 0),
    ([0], 4, 2, 64, 16, 0),
    ([15, 16, 17, 0, 1, 33], 8, 2, 128, 16, 0),
    ([100, 1, 255, 256, 257], 8, 8, 128, 32, 0),            # a key head a query head
    ([300, 77], 12, 1, 64, 48, 0),                           # one key head, odd group
    ([513, 64, 0], 20, 4, 96, 16, 0),
    ([1000], 32, 2, 128, 64, 0),                             # 16 query heads a key head
    ([700, 31], 40, 2, 128, 128, 0),                         # 20: past a tile of 8 or 16
    ([260, 129], 6, 2, 256, 16, 0),
    ([900, 300, 299, 301, 5], 8, 2, 128, 16, 300),           # window inside a page
    ([64, 65, 1], 4, 4, 64, 64, 1),                          # only the new token
    ([5000, 20, 333], 16, 4, 128, 16, 0),
    ([9000], 8, 1, 64, 32, 4097),
    ([2500], 71, 1, 64, 16, 0),
]


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("lens,hq,hk,D,page,window", ATTN_CASES)
def test_attention(lens, hq, hk, D, page, window, fmt):
    c, table, sl, rows, g = make_context(fmt, lens, hk, D, page, seed=sum(lens) + hq)
    q = randn(g, len(lens), hq, D, dtype=act(fmt))
    got, lse = c.attend(q, table, sl, window=window, return_lse=True)
    ref = attn_ref.attend(q, rows["k"], rows["v"], lens, hk, D ** -0.5, window)
    check(got, lse, ref, fmt)


@pytest.mark.parametrize("fmt", ["bf16", "f32"])
@pytest.mark.parametrize("D", [8, 24, 40, 80, 112, 192, 200, 248])
def test_attention_odd_head_sizes(D, fmt):
    lens = [130, 3, 47]
    c, table, sl, rows, g = make_context(fmt, lens, 2, D, 16, seed=D)
    q = randn(g, 3, 6, D, dtype=act(fmt))
    got, lse = c.attend(q, table, sl, return_lse=True)
    check(got, lse, attn_ref.attend(q, rows["k"], rows["v"], lens, 2, D ** -0.5), fmt)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("D", [32, 160, 192, 224])
def test_attention_mx_head_sizes(D, fmt):
    lens = [130, 3, 47, 200]
    c, table, sl, rows, g = make_context(fmt, lens, 2, D, 32, seed=D)
    q = randn(g, 4, 10, D, dtype=act(fmt))
    got, lse = c.attend(q, table, sl, return_lse=True)
    check(got, lse, attn_ref.attend(q, rows["k"], rows["v"], lens, 2, D ** -0.5), fmt)


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0, 1e-6])
def test_attention_scales(scale, fmt):
    """A scale of 0 (plain means), a negative one, one that makes single keys win."""
    lens = [200, 50]
    c, table, sl, rows, g = make_context(fmt, lens, 2, 64, 16, seed=4)
    q = randn(g, 2, 4, 64, dtype=act(fmt))
    got, lse = c.attend(q, table, sl, scale=scale, return_lse=True)
    check(got, lse, attn_ref.attend(q, rows["k"], rows["v"], lens, 2, scale), fmt)


@pytest.mark.parametrize("fmt", list(FMT))
def test_attention_growing_scores(fmt):
    """Keys whose scores grow along the context, so the running maximum moves
    at every tile, then fall again; q of very small and very large size."""
    D, n = 64, 1200
    c, table, sl, rows, g = make_context(fmt, [n, n, n], 1, D, 16, seed=12)
    ramp = torch.cat([torch.linspace(-3, 3, 900), torch.linspace(3, -3, 300)])
    k = (ramp[:, None, None] * torch.ones(1, 1, D)).to(act(fmt)).cuda()
    slot = []
    for b in range(3):
        j = torch.arange(n)
        slot.append(table[b].cpu().long()[j // 16] * 16 + j % 16)
    slot = torch.cat(slot)
    v = randn(g, 3 * n, 1, D, dtype=act(fmt))
    c.append(k.repeat(3, 1, 1), v, slot.int().cuda())
    dec = {s: attn_ref.decode(*stored(c, slot.cuda(), s), fmt) for s in "kv"}
    rows = {s: (lambda b, h, s=s: dec[s][b * n:(b + 1) * n, h]) for s in "kv"}
    q = torch.ones(3, 4, D)
    q[1] *= 2.0 ** -20
    q[2] *= 12.0
    q = q.to(act(fmt)).cuda()
    got, lse = c.attend(q, table, sl, return_lse=True)
    check(got, lse, attn_ref.attend(q, rows["k"], rows["v"], [n] * 3, 1, D ** -0.5), fmt)


def one_sequence(fmt, k, v, page=16):
    """A cache holding k, v [n][heads][D] as one sequence -> (cache, table, lengths, rows)."""
    n, hk, D = k.shape
    c = moe.PagedKVCache.empty(-(-n // page) + 1, page, hk, D, FMT[fmt])
    slots = torch.arange(n).int().cuda() + page          # from page 1 on
    c.append(k.to(act(fmt)).cuda(), v.to(act(fmt)).cuda(), slots)
    dec = {s: attn_ref.decode(*stored(c, slots.long(), s), fmt) for s in "kv"}
    table = (torch.arange(-(-n // page)) + 1).int().cuda()[None]
    rows = {s: (lambda b, h, s=s: dec[s][:, h]) for s in "kv"}
    return c, table, torch.tensor([n]).int().cuda(), rows


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("hq", [4, 16])
def test_attention_values_of_very_different_size(fmt, hq):
    """Value rows scaled by 2^-40 .. 2^40, in blocks of channels of their own sizes."""
    g = gen(41, hq)
    n, D = 700, 64
    k = torch.randn(n, 1, D, generator=g)
    v = torch.randn(n, 1, D, generator=g)
    v = v * torch.exp2(torch.randint(-40, 41, (n, 1, 1), generator=g).float())
    v[..., 32:] *= 2.0 ** -20
    c, table, sl, rows = one_sequence(fmt, k, v)
    q = randn(g, 1, hq, D, dtype=act(fmt))
    got, lse = c.attend(q, table, sl, return_lse=True)
    check(got, lse, attn_ref.attend(q, rows["k"], rows["v"], [n], 1, D ** -0.5), fmt)


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("hq", [2, 12])
def test_attention_large_values_under_tiny_weights(fmt, hq):
    """The largest values belong to keys of weight 2^-50 and less; the rest decide."""
    g = gen(43, hq)
    n, D = 400, 64
    k = torch.randn(n, 1, D, generator=g) * 0.1
    v = torch.randn(n, 1, D, generator=g)
    far = torch.arange(n) % 5 == 0
    k[far] = -1.0
    v[far] *= 2.0 ** 30
    c, table, sl, rows = one_sequence(fmt, k, v)
    q = (torch.ones(1, hq, D) * 6.0 + 0.1 * torch.randn(1, hq, D, generator=g)).to(act(fmt)).cuda()
    got, lse = c.attend(q, table, sl, return_lse=True)
    check(got, lse, attn_ref.attend(q, rows["k"], rows["v"], [n], 1, D ** -0.5), fmt)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("step", [1, 2, 3, -1, -2])
@pytest.mark.parametrize("hq,D", [(4, 64), (16, 128), (3, 256)])
def test_attention_value_scales_that_climb_or_fall(hq, D, step, fmt):
    """Every 16 keys the values grow (or shrink) by 2^step, each block of channels
    by a binary step of its own beside that, so that scales pass every distance
    from the largest seen before."""
    g = gen(53, hq, D)
    n = 720
    k = torch.randn(n, 1, D, generator=g)
    v = torch.randn(n, 1, D, generator=g)
    block = torch.arange(D) // 32
    first = -60 if step == 3 else 0  # 44 steps of 3 from 1 on would pass the largest bf16
    v = v * torch.exp2((first + torch.arange(n) // 16 * step)[:, None, None] + block * 3.0)
    c, table, sl, rows = one_sequence(fmt, k, v)
    q = randn(g, 1, hq, D, dtype=act(fmt))
    got, lse = c.attend(q, table, sl, return_lse=True)
    check(got, lse, attn_ref.attend(q, rows["k"], rows["v"], [n], 1, D ** -0.5), fmt)


@pytest.mark.parametrize("fmt", list(FMT))
def test_attention_queries_with_one_large_element(fmt):
    """One element 2^10 times the rest, where the keys are zero: the scores come from
    the small elements alone."""
    g = gen(59)
    n, D, hq = 500, 64, 8
    k = torch.randn(n, 1, D, generator=g)
    k[..., 5] = 0.0
    v = torch.randn(n, 1, D, generator=g)
    c, table, sl, rows = one_sequence(fmt, k, v)
    q = (1 + torch.rand(1, hq, D, generator=g)) * torch.where(
        torch.rand(1, hq, D, generator=g) < 0.5, -1.0, 1.0)
    q[..., 5] = 1.5 * 2.0 ** 10
    q = q.to(act(fmt)).cuda()
    got, lse = c.attend(q, table, sl, return_lse=True)
    check(got, lse, attn_ref.attend(q, rows["k"], rows["v"], [n], 1, D ** -0.5), fmt)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_attention_extreme_scales(fmt):
    """Blocks at the ends of E8M0: keys of 2^100 and 2^-100 against queries of the other
    size, and values of 2^-120."""
    g = gen(47)
    n, D = 100, 64
    k = torch.randn(n, 1, D, generator=g) * 2.0 ** 100
    k[::3] *= 2.0 ** -200
    v = torch.randn(n, 1, D, generator=g) * 2.0 ** -118
    c, table, sl, rows = one_sequence(fmt, k, v)
    q = (torch.randn(1, 4, D, generator=g) * 2.0 ** -101).to(act(fmt)).cuda()
    got, lse = c.attend(q, table, sl, return_lse=True)
    check(got, lse, attn_ref.attend(q, rows["k"], rows["v"], [n], 1, D ** -0.5), fmt)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_attention_nan_blocks_and_codes(fmt):
    """A NaN scale, whatever its codes, and an E4M3 NaN code: in a key the head's
    outputs are NaN, in a value the channels of the block (or the code's own)."""
    g = gen(53)
    n, D = 90, 64
    base = one_sequence(fmt, torch.randn(n, 1, D, generator=g), torch.randn(n, 1, D, generator=g))
    q = randn(g, 1, 3, D, dtype=torch.bfloat16)
    c, table, sl, rows = base
    want, _, tol, _ = attn_ref.attend(q, rows["k"], rows["v"], [n], 1, D ** -0.5)
    page, off = 1 + 40 // 16, 40 % 16
    c.v_scale[page, 0, off, 1] = 255                     # channels 32..63 of key 40
    got = c.attend(q, table, sl)
    assert got[..., 32:].isnan().all()
    err = (got.cpu().double() - want).abs()[..., :32]
    assert (err <= (tol + 2.0 ** -8 * want.abs())[..., :32]).all()
    c.v_scale[page, 0, off, 1] = 120
    if fmt == "mxfp8":
        old = int(c.v[page, 0, off, 5])
        c.v[page, 0, off, 5] = 0x7f
        got = c.attend(q, table, sl)
        assert got[..., 5].isnan().all()
        keep = torch.arange(D) != 5
        assert not got[..., keep].isnan().any()
        c.v[page, 0, off, 5] = old
        c.k[page, 0, off, 9] = 0xff
        assert c.attend(q, table, sl).isnan().all()
        c.k[page, 0, off, 9] = 0
    c.k_scale[page, 0, off, 0] = 255
    out, lse = c.attend(q, table, sl, return_lse=True)
    assert out.isnan().all() and lse.isnan().all()
    # out of sight it does not matter
    got = c.attend(q, table, sl, window=90 - 41)
    assert not got.isnan().any()


@pytest.mark.parametrize("fmt", list(FMT))
def test_attention_sequences_share_pages(fmt):
    """Two sequences with a common prefix in the same pages, different lengths."""
    g = gen(59)
    D, page = 64, 16
    k, v = torch.randn(64, 2, D, generator=g), torch.randn(64, 2, D, generator=g)
    c = moe.PagedKVCache.empty(5, page, 2, D, FMT[fmt])
    slots = torch.arange(64).int().cuda()
    c.append(k.to(act(fmt)).cuda(), v.to(act(fmt)).cuda(), slots)
    dec = {s: attn_ref.decode(*stored(c, slots.long(), s), fmt) for s in "kv"}
    table = torch.tensor([[0, 1, 2], [0, 1, 3]]).int().cuda()
    order = [list(range(48)), list(range(32)) + list(range(48, 64))]
    lens = [41, 48]
    q = randn(g, 2, 4, D, dtype=act(fmt))
    got, lse = c.attend(q, table, torch.tensor(lens).int().cuda(), return_lse=True)
    ref = attn_ref.attend(q, lambda b, h: dec["k"][order[b], h], lambda b, h: dec["v"][order[b], h],
                          lens, 2, D ** -0.5)
    check(got, lse, ref, fmt)


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("D", [160, 256])
@pytest.mark.parametrize("hq", [24, 40])
def test_attention_wide_heads_in_large_groups(D, hq, fmt):
    lens = [1500, 0, 33, 400]
    c, table, sl, rows, g = make_context(fmt, lens, 2, D, 32, seed=D + hq)
    q = randn(g, 4, hq, D, dtype=act(fmt))
    got, lse = c.attend(q, table, sl, return_lse=True)
    check(got, lse, attn_ref.attend(q, rows["k"], rows["v"], lens, 2, D ** -0.5), fmt)


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("window", [1, 17, 200])
def test_attention_small_windows_of_long_contexts(window, fmt):
    """Many segments of a tile or two beside a few whole ones."""
    g = gen(61, window)
    lens = [3000, 1, 0, 2999] + torch.randint(1, 3000, (41,), generator=g).tolist()
    c, table, sl, rows, g = make_context(fmt, lens, 2, 64, 16, seed=8)
    q = randn(g, len(lens), 6, 64, dtype=act(fmt))
    got, lse = c.attend(q, table, sl, window=window, return_lse=True)
    check(got, lse, attn_ref.attend(q, rows["k"], rows["v"], lens, 2, 0.125, window), fmt)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("B", [1, 3, 31, 33, 300])
def test_attention_batches_past_the_block_table_of_one_launch(B, fmt):
    """Lengths from 0 to 2500 under a table of more than 1024 tokens, any batch size."""
    g = gen(67, B)
    lens = (torch.rand(B, generator=g) ** 4 * 2500).int().tolist()
    lens[0] = 2500
    c, table, sl, rows, g = make_context(fmt, lens, 1, 64, 16, seed=B)
    q = randn(g, B, 4, 64, dtype=act(fmt))
    got, lse = c.attend(q, table, sl, return_lse=True)
    check(got, lse, attn_ref.attend(q, rows["k"], rows["v"], lens, 1, 0.125), fmt)


@pytest.mark.parametrize("fmt", list(FMT))
def test_attention_many_ragged_sequences(fmt):
    g = gen(77)
    lens = torch.randint(0, 400, (150,), generator=g).tolist()
    c, table, sl, rows, g = make_context(fmt, lens, 2, 64, 16, seed=3)
    q = randn(g, len(lens), 8, 64, dtype=act(fmt))
    got, lse = c.attend(q, table, sl, return_lse=True)
    check(got, lse, attn_ref.attend(q, rows["k"], rows["v"], lens, 2, 0.125), fmt)


@pytest.mark.parametrize("fmt", list(FMT))
def test_attention_one_long_context(fmt):
    """One sequence over the whole GPU: many parts joined."""
    n, D = 60_001, 64
    c, table, sl, rows, g = make_context(fmt, [n], 2, D, 64, seed=6)
    q = randn(g, 1, 6, D, dtype=act(fmt))
    got, lse = c.attend(q, table, sl, return_lse=True)
    check(got, lse, attn_ref.attend(q, rows["k"], rows["v"], [n], 2, D ** -0.5), fmt)


@pytest.mark.parametrize("fmt", ["bf16", "f32"])
def test_attention_infinite_scores(fmt):
    """Keys of -inf against positive queries: weight 0; a row with nothing else
    gives zeros; +inf and NaN scores give NaN in their own row only."""
    D, dt = 64, act(fmt)
    c = moe.PagedKVCache.empty(8, 16, 1, D, FMT[fmt])
    g = gen(2)
    v = randn(g, 64, 1, D, dtype=dt)
    k = torch.ones(64, 1, D, dtype=dt, device="cuda")
    k[0:16] = -math.inf                 # sequence 0: nothing visible
    k[16:24] = -math.inf                # sequence 1: the first half
    k[40] = math.inf                    # sequence 2
    k[50, 0, 3] = math.nan              # sequence 3
    c.append(k, v, torch.arange(64).int().cuda())
    table = torch.arange(4).int().cuda()[:, None]
    sl = torch.full((4,), 16, dtype=torch.int32).cuda()
    q = torch.ones(4, 2, D, dtype=dt, device="cuda")
    out, lse = c.attend(q, table, sl, return_lse=True)
    assert not out[0].any() and (lse[0] == -math.inf).all()
    want = v[24:32, 0].double().mean(0)
    tol = (2.0 ** -7 if fmt == "bf16" else 2.0 ** -18) * v[24:32, 0].abs().double().mean(0)
    assert ((out[1].double() - want).abs() <= tol).all()
    assert out[2:].isnan().all() and lse[2:].isnan().all()


def test_attention_nan_query_stays_in_its_row():
    lens = [40, 40]
    c, table, sl, rows, g = make_context("bf16", lens, 1, 64, 16, seed=1)
    q = randn(g, 2, 4, 64, dtype=torch.bfloat16)
    want = c.attend(q, table, sl)
    q2 = q.clone()
    q2[0, 1, 9] = math.nan
    got = c.attend(q2, table, sl)
    assert got[0, 1].isnan().all()
    keep = torch.ones(2, 4, dtype=torch.bool)
    keep[0, 1] = False
    assert torch.equal(got.cpu()[keep], want.cpu()[keep])


@pytest.mark.parametrize("fmt", list(FMT))
def test_attention_bad_pages_and_lengths_are_left_out_and_latched(fmt):
    D, hk = 64, 2
    lens = [64, 64, 64]
    c, table, sl, rows, g = make_context(fmt, lens, hk, D, 16, seed=21)
    q = randn(g, 3, 4, D, dtype=act(fmt))
    bad = table.clone()
    bad[1, 2] = c.k.shape[0]            # one past the pool
    bad[2, 0] = -7
    sl2 = sl.clone()
    sl2[0] = -3
    got, lse = c.attend(q, bad, sl2, return_lse=True)
    assert moe.coli_device_status() == moe.COLI_EDEVICE
    keep = {1: [0, 1, 3], 2: [1, 2, 3]}

    def part(side):
        def rows_of(b, h):
            if b == 0:
                return rows[side](b, h)[:0]
            return torch.cat([rows[side](b, h)[16 * p:16 * p + 16] for p in keep[b]])
        return rows_of
    ref = attn_ref.attend(q, part("k"), part("v"), [0, 48, 48], hk, D ** -0.5)
    check(got, lse, ref, fmt)
    # a length past the table's pages is cut to them
    got, lse = c.attend(q, table, torch.full_like(sl, 1000), return_lse=True)
    assert moe.coli_device_status() == moe.COLI_EDEVICE
    check(got, lse, attn_ref.attend(q, rows["k"], rows["v"], lens, hk, D ** -0.5), fmt)


@pytest.mark.parametrize("fmt", list(FMT))
def test_attention_parts_join_through_lse(fmt):
    lens = [640]
    c, table, sl, rows, g = make_context(fmt, lens, 2, 64, 16, seed=31)
    q = randn(g, 1, 4, 64, dtype=act(fmt))
    whole, lse = c.attend(q, table, sl, return_lse=True)
    parts = []
    for a, b in ((0, 12), (12, 40)):
        o, s = c.attend(q, table[:, a:b].contiguous(), torch.tensor([(b - a) * 16]).int().cuda(),
                        return_lse=True)
        parts.append((o.double(), s.double()))
    s = torch.stack([p[1] for p in parts])
    w = torch.softmax(s, 0)[..., None]
    joined = (torch.stack([p[0] for p in parts]) * w).sum(0)
    big = torch.stack([p[0].abs() for p in parts]).amax(0)
    # each part and the whole are rounded to the output type and carry weights
    # of at most 2^-9 off
    tol = (2.0 ** -23 if fmt == "f32" else 2.0 ** -8) * 2 * big + 2 * (
        2.0 ** -15 if fmt == "f32" else 2.0 ** -9) * attn_ref.attend(
            q, rows["k"], lambda b, h: rows["v"](b, h).abs(), lens, 2, 0.125)[0].cuda()
    assert ((joined - whole.double()).abs() <= tol).all()
    assert ((torch.logsumexp(s, 0) - lse).abs() <= 2.0 ** -14).all()


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_attention_strided_rows(fmt):
    """q as a slice of a fused projection's output, out as a slice of a wider buffer."""
    lens = [70, 200]
    D, hq, hk = 128, 8, 2
    c, table, sl, rows, g = make_context(fmt, lens, hk, D, 16, seed=5)
    qkv = randn(g, 2, hq + 2 * hk, D, dtype=torch.bfloat16)
    wide = torch.full((2, hq + 3, D), 9.0, dtype=torch.bfloat16, device="cuda")
    c.attend(qkv[:, :hq], table, sl, out=wide[:, :hq])
    want = c.attend(qkv[:, :hq].contiguous(), table, sl)
    assert torch.equal(wide[:, :hq], want) and (wide[:, hq:] == 9).all()


@pytest.mark.parametrize("fmt", list(FMT))
def test_pools_past_4_gib(fmt):
    """Byte offsets past 2^32 (and element offsets past 2^31 for bf16)."""
    hk, D, page = 8, 128, 64
    row = D * {"f32": 4, "bf16": 2, "mxfp8": 1, "mxfp4": 0.5}[fmt]
    pages = int((4.6e9 if fmt != "bf16" else 5.4e9) // (hk * page * row)) + 1
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}.get(fmt, torch.uint8)
    cols = D // 2 if fmt == "mxfp4" else D
    k = torch.empty(pages, hk, page, cols, dtype=dt, device="cuda")
    v = torch.empty_like(k)
    sc = [torch.empty(pages, hk, page, 4, dtype=torch.uint8, device="cuda") for _ in range(2)] \
        if fmt.startswith("mx") else [None, None]
    c = moe.PagedKVCache(k, v, *sc, head_dim=D)
    g = gen(15)
    n = 100
    ids = torch.tensor([pages - 1, pages - 2])
    j = torch.arange(n)
    slots = ids[j // page] * page + j % page
    kk, vv = (randn(g, n, hk, D, dtype=act(fmt)) for _ in range(2))
    c.append(kk, vv, slots.int().cuda())
    dec = {s: attn_ref.decode(*stored(c, slots.cuda(), s), fmt) for s in "kv"}
    want, _ = attn_ref.quantise(vv.float(), fmt) if fmt.startswith("mx") else (vv.cpu(), None)
    assert torch.equal(stored(c, slots.cuda(), "v")[0], want)
    got = c.read(slots.int().cuda())
    assert torch.equal(got[0].cpu().double(), dec["k"].to(act(fmt)).double())
    q = randn(g, 1, 16, D, dtype=act(fmt))
    out, lse = c.attend(q, ids.int().cuda()[None], torch.tensor([n]).int().cuda(),
                        return_lse=True)
    check(out, lse, attn_ref.attend(q, lambda b, h: dec["k"][:, h], lambda b, h: dec["v"][:, h],
                                    [n], hk, D ** -0.5), fmt)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_other_stream_and_graph(fmt):
    """The same bits on another stream, given as a stream or a raw handle, and
    from a captured graph after its inputs changed."""
    lens = [500, 20, 77]
    D, hq, hk = 128, 8, 2
    c, table, sl, rows, g = make_context(fmt, lens, hk, D, 16, seed=9)
    q = randn(g, 3, hq, D, dtype=torch.bfloat16)
    q2 = randn(g, 3, hq, D, dtype=torch.bfloat16)
    r = moe.Rotary.build(D, 600)
    pos = sl - 1

    def step(x, stream=None):
        y, _ = moe.rope(r, pos, x, stream=stream)
        return c.attend(y, table, sl, stream=stream)
    want, want2 = step(q), step(q2)
    assert torch.equal(step(q), want)                 # the same call, the same bits
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = step(q, side), step(q2, side.cuda_stream)
    side.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want2)
    x = q.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step(x)
    torch.cuda.current_stream().wait_stream(side)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    x.copy_(q2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want2)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_graph_of_a_cut_context(fmt):
    """A captured call whose contexts are cut and joined (two kernels), replayed
    after its lengths and queries changed, beside calls on another stream."""
    lens = [5000, 0, 70, 3000]
    c, table, sl, rows, g = make_context(fmt, lens, 2, 128, 16, seed=19)
    q, q2 = (randn(g, 4, 8, 128, dtype=torch.bfloat16) for _ in range(2))
    sl2 = torch.tensor([4000, 0, 16, 1]).int().cuda()
    want, want2 = c.attend(q, table, sl), c.attend(q2, table, sl2)
    side = torch.cuda.Stream()
    x, n = q.clone(), sl.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.attend(x, table, n)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = c.attend(x, table, n)
    torch.cuda.current_stream().wait_stream(side)
    side.wait_stream(torch.cuda.current_stream())
    graph.replay()
    others = [c.attend(q2, table, sl2, stream=side) for _ in range(5)]
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert all(torch.equal(o, want2) for o in others)
    x.copy_(q2)
    n.copy_(sl2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want2)


def test_empty_calls():
    c = moe.PagedKVCache.empty(2, 16, 2, 64, moe.BF16)
    z = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    c.append(z, z, none)
    assert c.read(none)[0].shape == (0, 2, 64)
    out = c.attend(z, torch.zeros(0, 3, dtype=torch.int32, device="cuda"), none)
    assert out.shape == (0, 2, 64)
    r = moe.Rotary.build(64, 4)
    assert moe.rope(r, none, z, z)[0].shape == (0, 2, 64)


def test_wrappers_reject_wrong_tensors():
    c = moe.PagedKVCache.empty(2, 16, 2, 64, moe.BF16)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(3, dtype=torch.int32, device="cuda")
    table = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    r = moe.Rotary.build(64, 4)
    for bad in (lambda: c.append(x.float(), x, ids), lambda: c.append(x, x[:2], ids),
                lambda: c.append(x, x, ids.long()), lambda: c.append(x, x, ids[:2]),
                lambda: c.append(x, x, ids, rotary=r), lambda: c.append(x.transpose(0, 1), x, ids),
                lambda: c.append(x, x, ids, rotary=r, positions=ids, q=x[:2]),
                lambda: c.read(ids.float()), lambda: c.attend(x, table.long(), ids),
                lambda: c.attend(x, table[:2], ids), lambda: c.attend(x, table, ids[:2]),
                lambda: c.attend(x[..., :32], table, ids),
                lambda: c.attend(x, table, ids, out=x.clone()[:2]),
                lambda: moe.rope(r, ids, x.half()), lambda: moe.rope(r, ids[:2], x),
                lambda: moe.rope(r, ids, x, x[:2]), lambda: moe.rope(r, ids, x, q_out=x.float())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(moe.ColiError):
        c.attend(torch.zeros(3, 3, 64, dtype=torch.bfloat16, device="cuda"), table, ids)
