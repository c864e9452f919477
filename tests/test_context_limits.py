"""The calls for long contexts refuse lengths and lists that their kernels cannot count in 32
bits, before anything is launched (CPU only)."""
import os
import sys

import pytest

import mixture_experts_gb300 as moe
from mixture_experts_gb300 import _build

sys.path.insert(0, os.path.dirname(__file__))
from test_context_arguments import cache, call  # noqa: E402

MOST = 2 ** 31 - 2 ** 16


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return moe.lib()


def refused(name, c=None, **kw):
    assert call(name, c=c, **kw) == moe.COLI_EINVAL
    assert any(n in moe.last_error() for n in kw), moe.last_error()


@pytest.mark.parametrize("length", [MOST + 1, 2 ** 31 - 1000, 2 ** 31 - 129, 2 ** 31 - 17,
                                    2 ** 31 - 1])
@pytest.mark.parametrize("dtype", [moe.F32, moe.BF16, moe.MXFP8, moe.MXFP4])
def test_prefixes_near_two_to_the_31(dtype, length):
    # tiles of 128 tokens are counted, and pages looked up 512 tokens ahead, past the last token
    refused("coli_shared_attention", c=cache(dtype=dtype), prefix_len=length)


@pytest.mark.parametrize("page,max_pages", [(16, 2 ** 27 - 4095), (16, 2 ** 27 - 1),
                                            (48, (2 ** 31 - 1) // 48), (4096, 2 ** 19 - 15),
                                            (4096, 2 ** 19 - 1)])
@pytest.mark.parametrize("name", ["coli_shared_attention", "coli_select_pages",
                                  "coli_selected_attention", "coli_attention_mass",
                                  "coli_kv_evict"])
def test_contexts_near_two_to_the_31(name, page, max_pages):
    # a context's pages are counted from its last token + page_size - 1, and its tokens by strides
    # of up to 1024 past the last
    refused(name, c=cache(page_size=page, n_pages=4), max_pages=max_pages)
    assert moe.coli_select_pages_scratch_bytes(cache(page_size=page, n_pages=4), 1, max_pages) == 0
    assert moe.coli_select_pages_scratch_bytes(cache(page_size=page, n_pages=4), 1,
                                               MOST // page) == 2 * 8 * (MOST // page)


@pytest.mark.parametrize("keep", [MOST + 1, 2 ** 31 - 1024, 2 ** 31 - 64, 2 ** 31 - 1])
def test_lists_near_two_to_the_31(keep):
    # a block walks a list in strides of up to 1024 entries
    one = dict(c=cache(n_kv_heads=1), B=1, keep=keep)
    refused("coli_select_pages", n_q_heads=4, **one)
    refused("coli_kv_evict", into=None, **one)
    refused("coli_kv_evict", into=None, max_pages=1, first=0, recent=0, **one)


@pytest.mark.parametrize("into_pages", [2 ** 27 - 4095, 2 ** 27 - 1])
def test_new_pages_near_two_to_the_31(into_pages):
    refused("coli_kv_evict", c=cache(n_kv_heads=1), B=1, into_pages=into_pages)
