"""The bound that the precise attention tests hold the kernels to lets plain results pass
and fails each mistake it exists for (CPU only)."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))
import attn_bound as ab  # noqa: E402


def parts(case, fmt):
    lens, hq, hk, D, page = case
    q, k, v = ab.inputs(case, fmt)
    k, v = ab.stored(k, fmt), ab.stored(v, fmt)
    at, g = 0, hq // hk
    for b, n in enumerate(lens):
        for h in range(hk):
            yield q[b, h * g:(h + 1) * g].double(), k[at:at + n, h], v[at:at + n, h]
        at += n


def passes(fmt, got, ref):
    out, lse, tol, tol_lse = ref
    return bool(((ab.rounded(got[0], fmt) - out).abs() <= tol).all()
                and ((got[1].float().double() - lse).abs() <= tol_lse).all())


@pytest.mark.parametrize("fmt", list(ab.OUT))
@pytest.mark.parametrize("case", ab.CASES)
def test_bound_passes_plain_results(case, fmt):
    for q, k, v in parts(case, fmt):
        s = (q @ k.T) * k.shape[1] ** -0.5
        ref = ab.bound(fmt, q, k, v, k.shape[1] ** -0.5)
        assert passes(fmt, (torch.softmax(s, -1) @ v, torch.logsumexp(s, -1)), ref)
        # in plain fp32 steps too
        s = (q.float() @ k.float().T) * k.shape[1] ** -0.5
        e = torch.exp(s - s.amax(-1, keepdim=True))
        got = (e @ v.float()) / e.sum(-1, keepdim=True)
        assert passes(fmt, (got.double(), torch.logsumexp(s, -1).double()), ref)


@pytest.mark.parametrize("fmt,name", [(f, n) for f in ab.OUT for n in ab.MISTAKES[f]])
def test_bound_fails_lost_bits(fmt, name):
    """In half of the cases at least."""
    f = ab.MISTAKES[fmt][name]
    shown = sum(not all(passes(fmt, f(fmt, q, k, v, k.shape[1] ** -0.5),
                               ab.bound(fmt, q, k, v, k.shape[1] ** -0.5))
                        for q, k, v in parts(case, fmt)) for case in ab.CASES)
    assert 2 * shown >= len(ab.CASES)


@pytest.mark.parametrize("fmt", list(ab.OUT))
@pytest.mark.parametrize("name", list(ab.LOST))
@pytest.mark.parametrize("case", ab.CASES)
def test_bound_fails_lost_tiles(case, fmt, name):
    f = ab.LOST[name]
    for q, k, v in parts(case, fmt):
        if k.shape[0] > 16:
            assert not passes(fmt, f(fmt, q, k, v, k.shape[1] ** -0.5),
                              ab.bound(fmt, q, k, v, k.shape[1] ** -0.5))


@pytest.mark.parametrize("fmt", list(ab.OUT))
@pytest.mark.parametrize("n,D", [(60001, 64), (60001, 256), (6000, 64), (700, 128)])
def test_marked_tiles_show_one_lost_or_doubled(n, D, fmt):
    """Scale 0, and tile t marked by a 1 in channel t % D: any one tile left out or taken
    twice is past the bound of its channel, and of the log-sum-exp."""
    out = torch.bincount(torch.arange(n) // 16 % D, minlength=D).double() / n
    tol, tol_lse = ab.flat_bound(fmt, out, n)
    for lost in (0, 1, 30, n // 16 - 1):
        for times in (0, 2):
            m = n + (times - 1) * 16
            wrong = out * n / m
            wrong[lost % D] += (times - 1) * 16 / m
            assert (ab.rounded(wrong, fmt) - out).abs()[lost % D] > tol[lost % D]
            assert abs(ab.log_of(m) - ab.log_of(n)) > tol_lse
