"""Decode attention at the ends of what its types hold: values and scales of very
different size, weights that vanish, keys and queries near the largest and smallest
numbers, queries of a wide range (GPU)."""
import math
import os
import sys

import pytest
import torch

import mixture_experts_gb300 as moe

sys.path.insert(0, os.path.dirname(__file__))
import attn_ref  # noqa: E402
import test_gpu_attention as base  # noqa: E402

pytestmark = pytest.mark.gpu

FMT, act, randn, check, one_sequence = base.FMT, base.act, base.randn, base.check, base.one_sequence
MX = ["mxfp8", "mxfp4"]


@pytest.fixture(scope="module", autouse=True)
def built():
    moe.build()
    assert torch.cuda.is_available()


@pytest.fixture(autouse=True)
def clean_status():
    assert moe.coli_device_status() == moe.COLI_OK
    yield
    assert moe.coli_device_status() == moe.COLI_OK


def gen(*key):
    return torch.Generator().manual_seed(sum((i + 3) * 104729 * int(k) for i, k in enumerate(key)))


def compare(c, table, sl, rows, q, fmt, scale=None):
    """attend() against the 64-bit form, over all of one sequence."""
    hk, D = c.n_kv_heads, c.head_dim
    got, lse = c.attend(q, table, sl, scale=scale, return_lse=True)
    check(got, lse, attn_ref.attend(q, rows["k"], rows["v"], sl.tolist(), hk,
                                    D ** -0.5 if scale is None else scale), fmt)


# ---- values whose scales lie further apart than a 16-bit operand's range ------------------
HEADS = [(4, 64), (16, 128), (8, 128), (3, 256), (16, 256)]


@pytest.mark.parametrize("fmt", MX)
@pytest.mark.parametrize("place", [0, 137, 399])
@pytest.mark.parametrize("hq,D", HEADS)
def test_a_large_value_of_no_weight(hq, D, place, fmt):
    """One value of 2^60 under a key whose weight is 0; the rest lie near 2^-60."""
    g = gen(1, hq, D, place)
    n = 400
    k = 0.1 * torch.randn(n, 1, D, generator=g)
    v = torch.randn(n, 1, D, generator=g) * 2.0 ** -60
    k[place] = -20.0                                  # about -20 D^0.5 * 6: e^-900 and less
    v[place] *= 2.0 ** 120
    c, table, sl, rows = one_sequence(fmt, k, v)
    q = (6.0 + 0.1 * torch.randn(1, hq, D, generator=g)).bfloat16().cuda()
    compare(c, table, sl, rows, q, fmt)


@pytest.mark.parametrize("fmt", MX)
@pytest.mark.parametrize("far", [40, 100, 150])
def test_a_large_value_that_one_head_alone_sees(far, fmt):
    """Heads of one group: for the even ones the large value decides, for the odd ones
    it has no weight and the rest do."""
    g = gen(2, far)
    n, D, hq = 300, 64, 8
    k = 0.1 * torch.randn(n, 1, D, generator=g)
    v = torch.randn(n, 1, D, generator=g) * 2.0 ** (-far / 2)
    k[50] = 20.0
    v[50] *= 2.0 ** (far / 2)
    v[50] *= 2.0 ** (far / 2)                         # (2^150 itself is past fp32)
    c, table, sl, rows = one_sequence(fmt, k, v)
    sign = torch.where(torch.arange(hq) % 2 == 0, 1.0, -1.0)[None, :, None]
    q = (sign * (6.0 + 0.1 * torch.randn(1, hq, D, generator=g))).bfloat16().cuda()
    compare(c, table, sl, rows, q, fmt)


@pytest.mark.parametrize("fmt", MX)
@pytest.mark.parametrize("hq,D", HEADS)
def test_values_that_shrink_as_the_scores_rise(hq, D, fmt):
    """Large values first, at small scores; each later run of keys scores far higher and
    holds values 2^45 times smaller, so every earlier sum loses its weight."""
    g = gen(3, hq, D)
    n = 800
    run = torch.arange(n) // 200
    k = (run[:, None, None] * 4.0 + 0.1 * torch.randn(n, 1, D, generator=g))
    v = torch.randn(n, 1, D, generator=g) * torch.exp2(60.0 - 45.0 * run)[:, None, None]
    c, table, sl, rows = one_sequence(fmt, k, v)
    q = (6.0 + 0.1 * torch.randn(1, hq, D, generator=g)).bfloat16().cuda()
    compare(c, table, sl, rows, q, fmt)


@pytest.mark.parametrize("fmt", MX)
@pytest.mark.parametrize("byte", [0, 1, 200, 254])
@pytest.mark.parametrize("hq,D", [(4, 64), (16, 128)])
def test_zeros_under_any_scale(hq, D, byte, fmt):
    """Value blocks of zeros count for nothing, whatever their scale byte says."""
    g = gen(4, hq, D, byte)
    n = 250
    k = torch.randn(n, 1, D, generator=g)
    v = torch.randn(n, 1, D, generator=g)
    v[::3] = 0.0
    c, table, sl, rows = one_sequence(fmt, k, v)
    at = torch.arange(0, n, 3).cuda() + 16
    c.v_scale[at // 16, 0, at % 16, :D // 32] = byte
    q = randn(g, 1, hq, D, dtype=torch.bfloat16)
    compare(c, table, sl, rows, q, fmt)


# ---- sums near the largest number --------------------------------------------------------
@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("n,top", [(3, 125), (200, 119), (12000, 112)])
def test_sums_of_large_values_stay_finite(n, top, fmt):
    """Equal weights over n values of about 2^top: their plain sum is finite, and so is
    the result."""
    g = gen(5, n, top)
    D = 64
    k = torch.zeros(n, 1, D)
    v = (1.0 + torch.rand(n, 1, D, generator=g)) * 2.0 ** top
    c, table, sl, rows = one_sequence(fmt, k, v)
    q = randn(g, 1, 4, D, dtype=act(fmt))
    compare(c, table, sl, rows, q, fmt)


@pytest.mark.parametrize("fmt", list(FMT))
def test_large_values_under_rising_weights(fmt):
    """Scores that rise by less than the running maximum's slack after the first keys."""
    g = gen(6)
    n, D = 512, 64
    k = torch.zeros(n, 1, D)
    k[256:] = 0.65                                    # 0.65 * 64 / 8 = 5.2: a factor of 2^7.5
    v = (1.0 + torch.rand(n, 1, D, generator=g)) * 2.0 ** 118
    c, table, sl, rows = one_sequence(fmt, k, v)
    q = torch.ones(1, 4, D).to(act(fmt)).cuda()
    compare(c, table, sl, rows, q, fmt)


# ---- keys and queries of opposite extremes -----------------------------------------------
@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("e", [60, 100, 110, 118])
@pytest.mark.parametrize("hq,D", [(4, 64), (16, 128), (8, 256)])
def test_large_keys_and_small_queries(hq, D, e, fmt):
    g = gen(7, hq, D, e)
    n = 150
    k = torch.randn(n, 1, D, generator=g) * 2.0 ** e
    v = torch.randn(n, 1, D, generator=g)
    c, table, sl, rows = one_sequence(fmt, k, v)
    q = (torch.randn(1, hq, D, generator=g) * 2.0 ** -e).to(act(fmt)).cuda()
    compare(c, table, sl, rows, q, fmt)


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("hq,D", [(4, 64), (16, 128), (8, 256)])
def test_small_keys_and_large_queries(hq, D, fmt):
    """Keys whose blocks take the smallest scale, 2^-127, against queries that bring the
    scores back to ordinary size."""
    g = gen(8, hq, D)
    n = 150
    e = 125 if fmt == "mxfp4" else 119
    k = (torch.randn(n, 1, D, generator=g) * 0.2).clamp(-1, 1) * 2.0 ** -e
    v = torch.randn(n, 1, D, generator=g)
    c, table, sl, rows = one_sequence(fmt, k, v)
    if fmt in MX:
        assert not c.k_scale[1, 0, :, :2].any()
    q = (torch.randn(1, hq, D, generator=g).clamp(-3, 3) * 2.0 ** (e + 1)).to(act(fmt)).cuda()
    compare(c, table, sl, rows, q, fmt)


# ---- queries of a wide range -----------------------------------------------------------------
@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("e", [13, 14, 16, 20, 28, 33, 40])
@pytest.mark.parametrize("hq,D", [(8, 64), (16, 128), (4, 128), (12, 256)])
def test_queries_with_large_elements_that_meet_zeros(hq, D, e, fmt):
    """Elements 2^e times the rest, some heads' first or last, where the keys are zero:
    the scores come from the small elements alone."""
    g = gen(9, hq, D, e)
    n = 300
    k = torch.randn(n, 1, D, generator=g)
    k[..., 5] = 0.0
    k[..., D - 1] = 0.0
    v = torch.randn(n, 1, D, generator=g)
    c, table, sl, rows = one_sequence(fmt, k, v)
    q = (1 + torch.rand(1, hq, D, generator=g)) * torch.where(
        torch.rand(1, hq, D, generator=g) < 0.5, -1.0, 1.0)
    q[:, ::2, 5] = 1.5 * 2.0 ** e
    q[:, 1::3, D - 1] = -1.25 * 2.0 ** e
    q = q.to(act(fmt)).cuda()
    compare(c, table, sl, rows, q, fmt)


@pytest.mark.parametrize("fmt", MX)
@pytest.mark.parametrize("what", ["inf", "nan"])
def test_a_query_that_is_no_number_stays_in_its_head(what, fmt):
    g = gen(10)
    n, D = 200, 64
    c, table, sl, rows = one_sequence(fmt, torch.randn(n, 1, D, generator=g),
                                      torch.randn(n, 1, D, generator=g))
    q = randn(g, 1, 4, D, dtype=torch.bfloat16)
    want, _, tol, _ = attn_ref.attend(q, rows["k"], rows["v"], [n], 1, D ** -0.5)
    q[0, 2, 7] = math.inf if what == "inf" else math.nan
    got = c.attend(q, table, sl).cpu().double()
    assert got[0, 2].isnan().all()
    keep = torch.tensor([0, 1, 3])
    assert ((got - want).abs() <= tol + 2.0 ** -8 * want.abs())[0, keep].all()


@pytest.mark.parametrize("fmt", MX)
@pytest.mark.parametrize("lens,hq,hk,D,page,window", [
    ([3000, 0, 41, 777], 6, 2, 96, 48, 0), ([2500, 16, 1], 24, 2, 64, 16, 1000),
    ([6000], 20, 1, 256, 32, 0), ([900, 900, 33], 4, 4, 160, 16, 300), ([400, 5, 60], 16, 1, 128, 64, 0)])
def test_far_values_in_windows_cut_contexts_and_beside_left_out_pages(lens, hq, hk, D, page,
                                                                      window, fmt):
    """Some warps' tiles hold values of 2^60 under no weight, some pages are outside the pool."""
    import test_gpu_attention_precise as precise
    import attn_bound as ab
    g = gen(11, hq, D, page)
    n = sum(lens)
    k = 0.1 * torch.randn(n, hk, D, generator=g)
    v = torch.randn(n, hk, D, generator=g) * 2.0 ** -60
    far = torch.rand(n, generator=g) < 0.01
    k[far], v[far] = -20.0, v[far] * 2.0 ** 120
    k, v = k.bfloat16(), v.bfloat16()
    c, table, sl = precise.pool(fmt, k, v, lens, page, seed=5)
    table[0, 1] = c.k.shape[0] + 3
    q = (6.0 + 0.1 * torch.randn(len(lens), hq, D, generator=g)).bfloat16().cuda()
    got, lse = c.attend(q, table, sl, window=window, return_lse=True)
    # (a left-out page before the window is not looked up)
    seen = max(0, lens[0] - window) if window else 0
    assert moe.coli_device_status() == (moe.COLI_EDEVICE if seen < 2 * page else moe.COLI_OK)
    k, v = ab.stored(k, fmt), ab.stored(v, fmt)
    starts = [sum(lens[:b]) for b in range(len(lens))]
    keep = []
    for b, m in enumerate(lens):
        j = torch.arange(max(0, m - window) if window else 0, m)
        keep.append(starts[b] + (j[j // page != 1] if b == 0 else j))
    ref = attn_ref.attend(q, lambda b, h: k[keep[b], h], lambda b, h: v[keep[b], h],
                          [len(x) for x in keep], hk, D ** -0.5)
    check(got, lse, ref, fmt)
