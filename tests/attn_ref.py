"""Plain 64-bit forms of the attention-side operators, on the CPU: rotary
tables and rotation, the cache formats' quantiser and decoder, attention over
a paged context, and the error bounds the kernels' fp32 steps admit."""
import math

import torch

GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
EMAX = {"mxfp8": 8, "mxfp4": 2}


def rope_angles(n, rot, base=10000.0, scaling=0, factor=1.0, orig=0, fast=32.0, slow=1.0):
    if scaling == 2:
        base = base * factor ** (rot / (rot - 2))
    w = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == 1:
        w = [x / factor for x in w]
    if scaling == 3:
        out = []
        for x in w:
            keep = min(1.0, max(0.0, (orig * x / (2 * math.pi) - slow) / (fast - slow)))
            out.append(x * keep + x / factor * (1 - keep))
        w = out
    return torch.arange(n, dtype=torch.float64)[:, None] * torch.tensor(w, dtype=torch.float64)


def rotate(x, table, pos, layout, inverse=False):
    """(rotated rows, sum of the magnitudes of the two products) in fp64."""
    x = x.double().cpu()
    half = table.shape[1]
    cs = table.double().cpu()[pos.long().cpu()][:, None]
    c, s = cs[..., 0], -cs[..., 1] if inverse else cs[..., 1]
    y, mag = x.clone(), x.abs()
    ia = torch.arange(half) if layout == "half" else 2 * torch.arange(half)
    ib = ia + half if layout == "half" else ia + 1
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = (a * c).abs() + (b * s).abs()
    mag[..., ib] = (b * c).abs() + (a * s).abs()
    return y, mag


def rotate32(x, table, pos, layout):
    """The same in fp32, each product and the sum rounded on its own."""
    x = x.float().cpu()
    half = table.shape[1]
    cs = table.cpu()[pos.long().cpu()][:, None]
    c, s = cs[..., 0], cs[..., 1]
    y = x.clone()
    ia = torch.arange(half) if layout == "half" else 2 * torch.arange(half)
    ib = ia + half if layout == "half" else ia + 1
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


def quantise(x, fmt):
    """fp32 [..][D] -> (codes, scale bytes), block by block from the formats'
    definition: a scan over the representable values."""
    x = x.double().cpu()
    blocks = x.reshape(-1, 32)
    if fmt == "mxfp8":
        vals = [(c, (c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10))
                for c in range(127)]
        sign = 128
    else:
        vals, sign = list(enumerate(GRID)), 8
    grid = torch.tensor([v for _, v in vals], dtype=torch.float64)
    codes = torch.zeros(blocks.shape, dtype=torch.int64)
    scales = torch.zeros(blocks.shape[0], dtype=torch.int64)
    for i, b in enumerate(blocks):
        if not torch.isfinite(b).all():
            scales[i] = 255
            continue
        amax = float(b.abs().max())
        e = 0 if amax == 0 else max(-127, math.frexp(amax)[1] - 1 - EMAX[fmt])
        scales[i] = e + 127
        v = b * 2.0 ** -e
        a = v.abs().clamp(max=float(grid[-1]))
        hi = torch.searchsorted(grid, a).clamp(max=len(vals) - 1)
        lo = (hi - 1).clamp(min=0)
        dl, dh = a - grid[lo], grid[hi] - a
        near = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
        codes[i] = near + sign * torch.signbit(v)
    codes = codes.reshape(x.shape).to(torch.uint8)
    if fmt == "mxfp4":
        codes = codes[..., 0::2] | (codes[..., 1::2] << 4)
    return codes, scales.reshape(*x.shape[:-1], -1).to(torch.uint8)


def decode(codes, scales, fmt):
    """fp64 rows of stored ones (F32 / BF16 rows pass through)."""
    if fmt not in EMAX:
        return codes.double().cpu()
    codes, scales = codes.cpu().int(), scales.cpu()
    if fmt == "mxfp8":
        lut = torch.tensor([(-1.0 if c & 128 else 1.0) * (
            math.nan if c & 127 == 127 else (c & 7) * 2.0 ** -9 if (c & 127) < 8 else
            (8 + (c & 7)) * 2.0 ** (((c >> 3) & 15) - 10)) for c in range(256)],
            dtype=torch.float64)
        v = lut[codes]
    else:
        lut = torch.tensor(GRID + [-g for g in GRID], dtype=torch.float64)
        v = torch.stack([lut[codes & 15], lut[codes >> 4]], -1).flatten(-2)
    s = torch.exp2(scales[..., :v.shape[-1] // 32].double() - 127)
    s = torch.where(scales[..., :v.shape[-1] // 32] == 255, math.nan, s)
    return v * s.repeat_interleave(32, -1)


def attend(q, k_of, v_of, lens, n_kv_heads, scale, window=0):
    """q [B][hq][D]; k_of(b, h) / v_of(b, h): fp64 [len][D] rows of the context.
    -> out, lse (fp64) and the bound of an fp32 kernel's error on each:

    a score is a sum of D products in fp32 (each addition off by at most 2^-22 of
    the running magnitude, the tensor core's worst), so it is off by at most
    ds = (D + 4) 2^-22 |scale| sum |q||k|; its weight is then off by a factor
    within exp(2 ds) (numerator and normaliser) and 2^-20 for the exponentials.
    Weights rounded to bf16 add 2^-9, the sum over n keys n 2^-22, all of
    sum p |v|. lse is off by ds + (n + 16) 2^-22 + |lse| 2^-22."""
    B, hq, D = q.shape
    g = hq // n_kv_heads
    q = q.double().cpu()
    out = torch.zeros(B, hq, D, dtype=torch.float64)
    lse = torch.full((B, hq), -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b, n in enumerate(lens):
        lo = max(0, n - window) if window else 0
        if n == 0:
            continue
        for h in range(n_kv_heads):
            k, v = k_of(b, h)[lo:n], v_of(b, h)[lo:n]
            r = slice(h * g, (h + 1) * g)
            s = (q[b, r] @ k.T) * scale
            p = torch.softmax(s, -1)
            out[b, r] = p @ v
            lse[b, r] = torch.logsumexp(s, -1)
            ds = ((D + 4) * 2.0 ** -22 * abs(scale) * (q[b, r].abs() @ k.abs().T)).amax(-1)
            rel = torch.expm1(2 * ds) + 2.0 ** -20 + 2.0 ** -9 + (n - lo) * 2.0 ** -22
            tol[b, r] = rel[:, None] * (p @ v.abs())
            tol_lse[b, r] = ds + (n - lo + 16) * 2.0 ** -22 + lse[b, r].abs() * 2.0 ** -22
    return out, lse, tol, tol_lse
