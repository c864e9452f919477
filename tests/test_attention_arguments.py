"""Refusals of the attention-side entry points and wrappers (CPU only)."""
import math

import pytest

import mixture_experts_gb300 as moe
from mixture_experts_gb300 import _build

FAKE = 1 << 20  # never dereferenced: validation fails first


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return moe.lib()


# ---- rotary table -----------------------------------------------------------------------
@pytest.mark.parametrize("field,value", [
    ("scaling", 16), ("scaling", 18), ("scaling", 20), ("base", 1.0), ("base", 0.5),
    ("beta_slow", 0.0), ("beta_slow", -1.0), ("beta_fast", 1.0), ("original_positions", 0),
    ("factor", 0.0), ("beta_slow", math.nan)])
def test_yarn_over_the_index_rejects(field, value):
    cfg = moe.coli_rope_config(64, moe.ROPE_YARN_INDEX, 4096, 10000.0, 4.0, 32.0, 1.0, 1.0)
    setattr(cfg, field, value)
    assert moe.coli_rope_table(cfg, 128, FAKE, stream=0) == moe.COLI_EINVAL
    assert moe.last_error()
