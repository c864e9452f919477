"""YaRN's two ramps: over the turns a pair makes, and over its index (GPU)."""
import math

import pytest
import torch

import mixture_experts_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    moe.build()
    assert torch.cuda.is_available()


def frequencies(rot, base, factor, orig, fast, slow):
    """The ramp over the index, from its definition: pair i makes
    orig base^(-2 i / rot) / (2 pi) turns over the trained context."""
    def at(turns):
        return rot * math.log(orig / (2 * math.pi * turns)) / (2 * math.log(base))
    lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), rot - 1)
    w = []
    for i in range(rot // 2):
        x = base ** (-2.0 * i / rot)
        keep = 1.0 - min(1.0, max(0.0, (i - lo) / (hi - lo if hi != lo else 0.001)))
        w.append(x * keep + x / factor * (1.0 - keep))
    return torch.tensor(w, dtype=torch.float64)


@pytest.mark.parametrize("rot,base,factor,orig,fast,slow", [
    (128, 10000.0, 16.0, 4096, 32.0, 1.0), (64, 10000.0, 40.0, 4096, 32.0, 1.0),
    (128, 1e6, 4.0, 32768, 32.0, 1.0), (20, 500.0, 2.0, 100, 8.0, 0.5), (2, 10.0, 8.0, 64, 4.0, 2.0)])
def test_yarn_over_the_index(rot, base, factor, orig, fast, slow):
    n, amp = 300, 0.1 * math.log(factor) + 1
    r = moe.Rotary.build(rot, n, base=base, scaling=moe.ROPE_YARN_INDEX, factor=factor,
                         original_positions=orig, beta_fast=fast, beta_slow=slow, amplitude=amp)
    a = torch.arange(n, dtype=torch.float64)[:, None] * frequencies(rot, base, factor, orig, fast,
                                                                    slow)
    want = torch.stack([a.cos(), a.sin()], -1) * amp
    # rounded once to fp32, and the fp64 angle's own error
    tol = 2.0 ** -24 * amp + a[..., None] * 2.0 ** -48
    assert ((r.table.cpu().double() - want).abs() <= tol).all()
    assert moe.coli_device_status() == moe.COLI_OK


def test_the_two_ramps_differ_only_between_their_ends():
    kw = dict(base=10000.0, factor=16.0, original_positions=4096)
    a, b = (moe.Rotary.build(128, 2, scaling=s, **kw).table[1, :, 1].cpu().double().asin()
            for s in (moe.ROPE_YARN, moe.ROPE_YARN_INDEX))
    ratio = (a / b)[1:]                             # (sin 1 of pair 0: the same in both)
    far = (ratio - 1).abs() > 1e-5
    # the pairs of 32 turns and of 1 lie at 20.9 and 45.04
    assert far.sum() >= 20 and not far[:19].any() and not far[46:].any()
    assert 1.5 < max(float(ratio.max()), 1 / float(ratio.min())) < 4.0
