"""The decode example runs the attention-side operators and the MoE layer together (GPU)."""
import os
import sys

import pytest

import mixture_experts_gb300 as moe

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxfp4"])
def test_decode_block(fmt):
    moe.build()
    import decode_block
    # bf16 outputs are rounded to 2^-9 and carry weights rounded as much at most; the
    # plain form reads MX values back as bf16 exactly
    assert decode_block.main(["--format", fmt, "--batch", "3", "--prompt", "70", "--steps", "4",
                              "--check"]) <= 2.0 ** -8
