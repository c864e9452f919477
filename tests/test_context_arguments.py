"""The entry points for shared prefixes, chosen pages and eviction reject bad arguments before
anything is launched, and the plain forms their GPU tests use agree with torch (CPU only)."""
import math
import os
import sys

import pytest
import torch

import mixture_experts_gb300 as moe
from mixture_experts_gb300 import _build

sys.path.insert(0, os.path.dirname(__file__))
import context_ref as ref  # noqa: E402

FAKE = 1 << 20  # never dereferenced: validation fails first
OTHER = FAKE + (1 << 16)


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return moe.lib()


def cache(**kw):
    c = moe.coli_kv_cache(FAKE, FAKE, FAKE, FAKE, 8, 16, 2, 64, moe.BF16)
    for n, v in kw.items():
        setattr(c, n, v)
    return c


def cfg(heads=4, window=0, scale=0.125):
    return moe.coli_attn_config(heads, window, scale)


def call(name, c=None, **kw):
    """The call with arguments that pass every check but for those given; it is only made with
    one that does not."""
    args = {
        "coli_shared_attention": dict(
            cache=c or cache(), cfg=cfg(), q=FAKE, q_stride=256, B=2, prefix_pages=FAKE,
            prefix_len=20, block_table=FAKE, max_pages=4, seq_lens=FAKE, out=OTHER,
            out_stride=256, lse=FAKE, scratch=FAKE, scratch_bytes=1 << 40),
        "coli_page_bounds": dict(cache=c or cache(), pages=FAKE, fills=FAKE, N=3, bounds=FAKE),
        "coli_select_pages": dict(
            cache=c or cache(), bounds=FAKE, q=FAKE, q_stride=256, n_q_heads=4, B=2,
            block_table=FAKE, max_pages=4, seq_lens=FAKE, keep=3, first=1, last=1, pages=FAKE,
            lens=OTHER, scratch=FAKE, scratch_bytes=1 << 40),
        "coli_selected_attention": dict(
            cache=c or cache(), cfg=cfg(), q=FAKE, q_stride=256, B=2, pages=FAKE, max_pages=400,
            lens=FAKE, out=OTHER, out_stride=256, lse=FAKE, scratch=FAKE, scratch_bytes=1 << 40),
        "coli_attention_mass": dict(
            cache=c or cache(), cfg=cfg(), q=FAKE, q_stride=256, B=2, block_table=FAKE,
            max_pages=4, seq_lens=FAKE, lse=FAKE, known=FAKE, mass=FAKE),
        "coli_kv_evict": dict(
            cache=c or cache(), mass=FAKE, B=2, block_table=FAKE, max_pages=4, seq_lens=FAKE,
            keep=20, first=1, recent=4, into=OTHER, into_pages=2, kept=FAKE, new_lens=OTHER),
    }[name]
    args.update(kw)
    return getattr(moe, name)(stream=0, **args)


CALLS = ["coli_shared_attention", "coli_page_bounds", "coli_select_pages",
         "coli_selected_attention", "coli_attention_mass", "coli_kv_evict"]
ATTN = [dict(cfg=None), dict(cfg=cfg(heads=0)), dict(cfg=cfg(heads=3)), dict(cfg=cfg(heads=1026)),
        dict(cfg=cfg(scale=math.inf)), dict(cfg=cfg(scale=math.nan)), dict(cfg=cfg(window=-1)),
        dict(q=None), dict(q=FAKE + 8), dict(q_stride=255), dict(q_stride=64), dict(B=-1),
        dict(B=65536)]
TABLE = [dict(block_table=None), dict(block_table=FAKE + 2), dict(seq_lens=None),
         dict(seq_lens=FAKE + 1), dict(max_pages=0), dict(max_pages=1 << 28)]
OUT = [dict(out=None), dict(out=FAKE), dict(out=OTHER + 4), dict(out_stride=128),
       dict(lse=FAKE + 3), dict(cfg=cfg(window=5)), dict(scratch=None), dict(scratch=FAKE + 8),
       dict(scratch_bytes=8)]
BAD = (
    [("coli_shared_attention", x) for x in ATTN + TABLE + OUT + [
        dict(prefix_len=-1), dict(prefix_len=2 ** 31 - 16), dict(prefix_pages=None),
        dict(prefix_pages=FAKE + 2)]] +
    [("coli_page_bounds", x) for x in [
        dict(pages=None), dict(pages=FAKE + 1), dict(fills=None), dict(fills=FAKE + 2), dict(N=-1),
        dict(N=(1 << 24) + 1), dict(bounds=None), dict(bounds=FAKE + 8)]] +
    [("coli_select_pages", x) for x in TABLE + [
        dict(n_q_heads=0), dict(n_q_heads=5), dict(n_q_heads=2000), dict(q=None),
        dict(q=FAKE + 2), dict(q_stride=100), dict(B=-1), dict(B=65536), dict(bounds=None),
        dict(bounds=FAKE + 4), dict(keep=0), dict(keep=1), dict(first=-1), dict(last=0),
        dict(first=2 ** 31 - 1, last=2 ** 31 - 1), dict(keep=2 ** 30), dict(pages=None),
        dict(lens=None), dict(lens=FAKE), dict(scratch=None), dict(scratch=FAKE + 4),
        dict(scratch_bytes=2 * 2 * 4 * 8 - 1)]] +
    [("coli_selected_attention", x) for x in ATTN + OUT + [
        dict(pages=None), dict(lens=None), dict(max_pages=0)]] +
    [("coli_attention_mass", x) for x in ATTN + TABLE + [
        dict(lse=None), dict(lse=FAKE + 2), dict(known=FAKE + 1), dict(mass=None),
        dict(mass=FAKE + 2)]] +
    [("coli_kv_evict", x) for x in TABLE + [
        dict(mass=None), dict(mass=FAKE + 2), dict(B=-1), dict(B=65536), dict(keep=0),
        dict(keep=4), dict(first=-1), dict(recent=-1), dict(into=OTHER + 2), dict(into_pages=1),
        dict(into_pages=0), dict(into_pages=1 << 28), dict(kept=None), dict(new_lens=None),
        dict(new_lens=FAKE), dict(first=2 ** 31 - 1, recent=2 ** 31 - 1),
        dict(keep=2 ** 30, into_pages=1 << 26)]])


@pytest.mark.parametrize("name,bad", BAD)
def test_bad_arguments_are_rejected(name, bad):
    assert call(name, **bad) == moe.COLI_EINVAL
    assert moe.last_error()


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("bad", [dict(dtype=9), dict(head_dim=60), dict(page_size=24),
                                 dict(n_kv_heads=0), dict(n_pages=0), dict(k=None),
                                 dict(dtype=moe.MXFP4, k_scale=None)])
def test_bad_caches_are_rejected(name, bad):
    assert call(name, c=cache(**bad)) == moe.COLI_EINVAL


@pytest.mark.parametrize("name", CALLS)
def test_nothing_to_do(name):
    kw = dict(N=0) if name == "coli_page_bounds" else dict(B=0)
    assert call(name, **kw) == moe.COLI_OK


def test_scratch_sizes():
    c = cache()
    assert moe.coli_select_pages_scratch_bytes(c, 3, 100) == 3 * 2 * 100 * 8
    assert moe.coli_select_pages_scratch_bytes(c, 0, 100) == 0
    assert moe.coli_select_pages_scratch_bytes(c, 3, 0) == 0
    assert moe.coli_select_pages_scratch_bytes(cache(dtype=9), 3, 10) == 0
    # two sides' means and pairs at least
    assert moe.coli_shared_attention_scratch_bytes(c, 3, 8) >= 2 * 3 * 8 * (64 * 4 + 8)
    for bad in (dict(B=0, n_q_heads=8), dict(B=3, n_q_heads=5), dict(B=3, n_q_heads=0),
                dict(B=65536, n_q_heads=8)):
        assert moe.coli_shared_attention_scratch_bytes(c, **bad) == 0


def test_plain_forms():
    g = ref.gen(3)
    # the score is the largest over the box's corners
    q, box = torch.randn(3, 4, generator=g).double(), torch.randn(2, 4, generator=g).double()
    box = box.sort(0).values
    corners = torch.cartesian_prod(*[box[:, d] for d in range(4)])
    assert math.isclose(ref.score(q, box), float((q @ corners.T).max()), rel_tol=1e-12)
    # the largest places, against a stable sort
    for n, keep, first, last in ((9, 4, 1, 1), (9, 9, 0, 1), (30, 7, 0, 0), (5, 8, 2, 2)):
        v = torch.randint(0, 4, (n,), generator=g).double()
        got = ref.largest(v.tolist(), keep, first, last)
        w = v.clone()
        w[:first], w[n - last:] = math.inf, math.inf
        order = torch.sort(w, descending=True, stable=True).indices[:keep]
        if n > keep:
            assert got == order.sort().values.tolist()
        else:
            assert got == list(range(n))
    # masses of a context sum to the number of heads
    k = torch.randn(50, 4, generator=g).double()
    s = q @ k.T * 0.5
    w, tol = ref.mass(q, k, torch.logsumexp(s, -1), 0.5)
    assert math.isclose(float(w.sum()), 3.0, rel_tol=1e-12) and (tol < 1e-5).all()
