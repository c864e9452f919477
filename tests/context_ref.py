"""Plain 64-bit forms of what keeps long contexts affordable over the paged cache, on the
CPU: page bounds and the pages they choose, attention mass, eviction; and pools of random
numbers to run them on."""
import math

import torch

import attn_ref
import mixture_experts_gb300 as moe

FMT = {"f32": moe.F32, "bf16": moe.BF16, "mxfp8": moe.MXFP8, "mxfp4": moe.MXFP4}


def gen(*key):
    return torch.Generator().manual_seed(sum((i + 1) * 7919 * int(k) for i, k in enumerate(key)))


def act(fmt):
    return torch.float32 if fmt == "f32" else torch.bfloat16


def pool(g, fmt, n_pages, page, hk, D, device="cuda"):
    """A cache of random numbers and its keys and values in fp64 [n_pages][hk][page][D]."""
    shape = (n_pages, hk, page)
    if fmt in attn_ref.EMAX:
        codes, scales = [], []
        for _ in range(2):
            if fmt == "mxfp8":
                c = torch.randint(0, 256, (*shape, D), generator=g).to(torch.uint8)
                c = torch.where((c & 127) == 127, c & 0xf0, c)      # no NaN codes
                lo = 118
            else:
                c = torch.randint(0, 256, (*shape, D // 2), generator=g).to(torch.uint8)
                lo = 124
            pad = (D // 32 + 3) // 4 * 4
            s = torch.randint(lo, lo + 3, (*shape, pad), generator=g).to(torch.uint8)
            s[..., D // 32:] = 255                                  # never read
            codes.append(c)
            scales.append(s)
        rows = [attn_ref.decode(c, s, fmt) for c, s in zip(codes, scales)]
        args = codes + scales
    else:
        args = [torch.randn(*shape, D, generator=g).to(act(fmt)) for _ in range(2)]
        rows = [x.double() for x in args]
    args = [x.to(device) for x in args]
    return moe.PagedKVCache(*args, head_dim=D), rows[0], rows[1]


def tables(g, lens, page, n_pages, taken=()):
    """int32 [B][max] of different pages in no order, -1 past each sequence's last."""
    free = [p for p in torch.randperm(n_pages, generator=g).tolist() if p not in set(taken)]
    per = [-(-n // page) for n in lens]
    t = torch.full((len(lens), max(1, max(per))), -1, dtype=torch.int32)
    for b, n in enumerate(per):
        for i in range(n):
            t[b, i] = free.pop()
    return t


def context(rows, pages, h, n):
    """fp64 [n][D] of head h over a list of pages."""
    if n == 0:
        return rows[0, h, :0]
    return torch.cat([rows[p, h] for p in pages[:-(-n // rows.shape[2])]])[:n]


def bounds(k, page, h, fill):
    x = k[page, h, :fill]
    return torch.stack([x.min(0).values, x.max(0).values])


def score(q, box):
    """q [group][D], box [2][D], fp64: the largest score of the group's heads."""
    best = -math.inf
    for row in q.tolist():
        x = sum(a * (hi if a > 0 else lo) for a, lo, hi in
                zip(row, box[0].tolist(), box[1].tolist()) if a != 0)
        if math.isnan(x):
            return -math.inf
        best = max(best, x)
    return best


def largest(values, keep, first, last):
    """Places of the `keep` largest of a list (NaN: -inf; equal: the earlier), the first
    and last ones among them, rising."""
    n = len(values)
    if n <= keep:
        return list(range(n))
    values = [-math.inf if math.isnan(v) else v for v in values]
    must = [j for j in range(n) if j < first or j >= n - last]
    rest = sorted((j for j in range(n) if first <= j < n - last), key=lambda j: (-values[j], j))
    return sorted(must + rest[:keep - len(must)])


def mass(q, k, lse, scale):
    """fp64 weights of one key head's context: sum over the heads of exp(scale q.k - lse), and
    the bound of an fp32 kernel's error: a score of D products is off by at most
    ds = (D + 4) 2^-22 |scale| sum |q||k|, the difference to lse and its exponential by 2^-22 of
    |score| + |lse| more and 2^-20 for the exponential itself."""
    s = (q @ k.T) * scale
    out, tol = torch.zeros(k.shape[0], dtype=torch.float64), torch.zeros(k.shape[0],
                                                                         dtype=torch.float64)
    for i in range(q.shape[0]):
        if lse[i] == -math.inf:
            continue
        w = torch.exp(s[i] - lse[i])
        ds = (q.shape[1] + 4) * 2.0 ** -22 * abs(scale) * (k.abs() @ q[i].abs())
        out += w
        tol += w * (torch.expm1(ds + 2.0 ** -22 * (s[i].abs() + abs(lse[i]))) + 2.0 ** -20)
    return out, tol + out * q.shape[0] * 2.0 ** -24
