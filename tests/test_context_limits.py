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
