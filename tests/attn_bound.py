"""What the decode attention's arithmetic may be off by, format by format, and the mistakes
that such a bound has to show (plain 64-bit forms on the CPU).

A warp matrix product D = A x B + C is off by at most 2^-20 of its largest term (10 x 2^-24
measured over random and one-signed operands of every type used). Beyond that, per format:

  scores      the query and key elements' own loss, and one product after the other over the
              head: F32 3 D/8 of them on elements cut in two tf32 parts (each 2^-21 off, the
              low x low product left out, 2^-20), BF16 D/16, MX 2 D/32, a third for small elements,
              and D/32 additions in fp32;
  weights     2^-21 for the exponential; F32 two parts as above; BF16 a bf16 number and one
              for what its rounding left, 2^-8 each; MX fp16, 2^-11, with 2^-25 absolute below
              2^-14, where the largest weight is 2^14 at the least, so 2^-39 of it;
  sums        the products of the tiles of one warp (F32 6 a tile, BF16 2, MX 1 or 2), then
              fp32 additions over warps and parts of a context, 2^-23 each;
  output      one rounding to the output type.
"""
import math

import torch

import attn_ref

MX = ("mxfp8", "mxfp4")
PER_TILE = {"f32": 6, "bf16": 2, "mxfp8": 2, "mxfp4": 2}
WEIGHT = {"f32": 2.0 ** -19, "bf16": 2.0 ** -16, "mxfp8": 2.0 ** -11, "mxfp4": 2.0 ** -11}
OUT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "mxfp8": 2.0 ** -8, "mxfp4": 2.0 ** -8}


def score_error(fmt, q, k):
    """Of each q . k, [g][n]: the products' steps are off in proportion to the largest
    number among their terms, a product or the sum up to some 8 elements."""
    D = k.shape[1]
    terms = q[:, None] * k[None]
    top = torch.maximum(terms.cumsum(-1)[..., 7::8].abs().amax(-1), terms.abs().amax(-1))
    if fmt == "f32":
        return 2.0 ** -19 * terms.abs().sum(-1) + (3 * D / 8) * 2.0 ** -20 * top
    if fmt == "bf16":
        return (D / 16) * 2.0 ** -20 * top
    return ((3 * D / 32) * 2.0 ** -20 + (D / 32 + 3) * 2.0 ** -23) * top


def bound(fmt, q, k, v, scale, tiles=None, joins=24):
    """q [g][D], k, v [n][D] in 64 bits -> out, lse and how far a kernel's may be off.
    tiles: most tiles of 16 keys that one warp takes (4 warps or more share a context)."""
    n, D = k.shape
    s = (q @ k.T) * scale
    p = torch.softmax(s, -1)
    out, lse = p @ v, torch.logsumexp(s, -1)
    if tiles is None:
        tiles = n // 64 + 2
    ds = score_error(fmt, q, k).amax(-1) * abs(scale) + 2.0 ** -22 * s.abs().amax(-1)
    sums = tiles * PER_TILE[fmt] * 2.0 ** -20 + joins * 2.0 ** -23
    rel = torch.expm1(2 * ds) + WEIGHT[fmt] + 2.0 ** -20 + sums
    tol = rel[:, None] * (p @ v.abs()) + OUT[fmt] * out.abs()
    if fmt in MX:
        tol = tol + 2.0 ** -38 * v.abs().amax(0)
    return out, lse, tol, ds + 2.0 ** -20 + (tiles + joins) * 2.0 ** -23 + lse.abs() * 2.0 ** -22


def flat_bound(fmt, out, n):
    """The same for equal weights over n keys (scale 0) of values that are not negative."""
    tiles, joins = n // 64 + 2, 24
    rel = WEIGHT[fmt] + 2.0 ** -20 + tiles * PER_TILE[fmt] * 2.0 ** -20 + joins * 2.0 ** -23
    return (rel + OUT[fmt]) * out, 2.0 ** -20 + (tiles + joins) * 2.0 ** -23 + log_of(
        max(n, 1)) * 2.0 ** -22


def rounded(x, fmt):
    return (x.float() if fmt == "f32" else x.bfloat16()).double()


def cut(x, bits):
    """x with that many significant bits, nearest even."""
    e = torch.exp2(torch.frexp(x)[1].double() - bits)
    return torch.where(x == 0, x, torch.round(x / e) * e)


# Each takes (fmt, q, k, v, scale) to the (out, lse) of a kernel with one mistake.
def _weights_of(bits):
    def f(fmt, q, k, v, scale):
        s = (q @ k.T) * scale
        e = torch.exp(s - s.amax(-1, keepdim=True))
        return (cut(e, bits) @ v) / e.sum(-1, keepdim=True), torch.logsumexp(s, -1)
    return f


def _elements_of(bits, side):
    def f(fmt, q, k, v, scale):
        s = ((cut(q, bits) if side == "q" else q) @ (cut(k, bits) if side == "k" else k).T) * scale
        return torch.softmax(s, -1) @ (cut(v, bits) if side == "v" else v), torch.logsumexp(s, -1)
    return f


def _tile(t, times):
    def f(fmt, q, k, v, scale):
        at = torch.arange(k.shape[0])
        at = torch.cat([at[:16 * t], at[16 * t:16 * t + 16].repeat(times), at[16 * t + 16:]])
        s = (q @ k[at].T) * scale
        return torch.softmax(s, -1) @ v[at], torch.logsumexp(s, -1)
    return f


MISTAKES = {
    "f32": {"weights in one tf32 part": _weights_of(11), "values in one": _elements_of(11, "v"),
            "queries in one": _elements_of(11, "q"), "keys in one": _elements_of(11, "k")},
    "bf16": {"weights in one bf16 part": _weights_of(8)},
    "mxfp8": {"weights in 8 bits": _weights_of(8), "queries in 4 bits": _elements_of(4, "q")},
    "mxfp4": {"weights in 8 bits": _weights_of(8), "queries in 4 bits": _elements_of(4, "q")},
}
LOST = {"a tile left out": _tile(1, 0), "a tile taken twice": _tile(0, 2)}

# lens, query heads, key heads, head_dim, page
CASES = [([2, 3, 5, 17, 40], 8, 2, 64, 16), ([2, 130, 3, 33], 16, 1, 128, 32),
         ([3, 4, 60, 2], 6, 2, 256, 16), ([700, 2], 10, 1, 64, 48)]


def inputs(case, fmt, seed=0):
    """(q [B][hq][D], k, v [tokens][hk][D]) as they go in, on the CPU: scores of ordinary
    spread whose magnitudes stay small, so that the bound on them does too."""
    lens, hq, hk, D, page = case
    g = torch.Generator().manual_seed(1000 * D + 17 * hq + seed)
    dt = torch.float32 if fmt == "f32" else torch.bfloat16
    q = torch.randn(len(lens), hq, D, generator=g) * 0.25
    k = torch.randn(sum(lens), hk, D, generator=g)
    v = torch.randn(sum(lens), hk, D, generator=g)
    return q.to(dt), k.to(dt), v.to(dt)


def stored(x, fmt):
    """What a cache of this format holds of x, in 64 bits."""
    if fmt not in MX:
        return x.double()
    return attn_ref.decode(*attn_ref.quantise(x.float(), fmt), fmt)


def log_of(n):
    return math.log(n) if n else -math.inf
