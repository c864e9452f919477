"""Measured cases of the attention-side operators: rotary positions, the paged
key-value cache's write and read, and the attention of one new token over it.

Each case is one pass through one operator as a decode or prefill step calls
it. `run` computes it with elementary torch operations in fp32 (`own` false)
or through the package's entry points (`own` true), on the same inputs.
"""
import math

import torch

own = False

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of the E2M1 codes 0..7
EMAX = {"mxfp8": 8, "mxfp4": 2}                  # exponent of the largest E4M3 / E2M1 value
ROW_BYTES = {"f32": 4.0, "bf16": 2.0, "mxfp8": 1.0, "mxfp4": 0.5}


# ---- cases -------------------------------------------------------------------------
def listed():
    return [
        # one decode step of 32 sequences: every head of q and k turned by its position
        dict(name="rope_decode", op="rope", T=32, hq=32, hk=8, D=128, rot=128, layout="half",
             scaling="none", n_pos=32768, act="bf16"),
        # a long prompt batch, pairs interleaved, half of each head rotated, positions
        # interpolated for a longer context
        dict(name="rope_prefill", op="rope", T=16384, hq=32, hk=8, D=128, rot=64,
             layout="interleaved", scaling="linear", n_pos=65536, act="bf16"),
        # fp32 layer, odd token count, head size 80 with a quarter rotated (pairs 10 apart)
        dict(name="rope_odd_f32", op="rope", T=1021, hq=20, hk=4, D=80, rot=20, layout="half",
             scaling="yarn", n_pos=131072, act="f32"),
        # the same decode step writing its keys and values into an 8-bit cache, q and k
        # rotated on the way
        dict(name="append_decode_mxfp8", op="append", T=32, hq=32, hk=8, D=128, rot=128,
             layout="half", scaling="none", n_pos=32768, fmt="mxfp8", page=16, pages=1024),
        # a prompt batch written into the 8-bit cache
        dict(name="append_prefill_mxfp8", op="append", T=16384, hq=32, hk=8, D=128, rot=128,
             layout="half", scaling="ntk", n_pos=65536, fmt="mxfp8", page=64, pages=320),
        # a ragged batch stored in 4 bits and read back (swapping a cache out and in)
        dict(name="store_mxfp4", op="store", T=4099, hk=4, D=64, fmt="mxfp4", page=32, pages=160),
        # a long 8-bit context read back to bf16 (prefix reuse by a prefill)
        dict(name="read_mxfp8", op="read", T=65536, hk=8, D=128, fmt="mxfp8", page=64,
             pages=1280),
        # one user, short context: latency
        dict(name="attn_one_short", op="attn", B=1, hq=32, hk=8, D=128, fmt="bf16", page=16,
             len_lo=777, len_hi=777, window=0),
        # a decode batch of ragged contexts
        dict(name="attn_batch_bf16", op="attn", B=32, hq=32, hk=8, D=128, fmt="bf16", page=16,
             len_lo=300, len_hi=8192, window=0),
        # a larger decode batch on the 8-bit cache
        dict(name="attn_batch_mxfp8", op="attn", B=64, hq=32, hk=8, D=128, fmt="mxfp8", page=64,
             len_lo=1000, len_hi=16384, window=0),
        # one user with half a million tokens of context
        dict(name="attn_one_long", op="attn", B=1, hq=32, hk=8, D=128, fmt="bf16", page=64,
             len_lo=500009, len_hi=500009, window=0),
        # many short sessions on a 4-bit cache, 16 query heads a key head, sliding window
        dict(name="attn_window_mxfp4", op="attn", B=160, hq=64, hk=4, D=128, fmt="mxfp4", page=32,
             len_lo=1, len_hi=9000, window=4096),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "store", "read", "attn", "attn", "attn"])
    hk = rng.choice([1, 2, 4, 8, 8, 16])
    hq = hk * rng.choice([1, 2, 4, 5, 8, 16])
    if op == "rope":
        D = rng.choice([64, 80, 96, 128, 128, 256])
        rot = rng.choice([D, D, D // 2, D // 4])
        return dict(op=op, T=_log_int(rng, 1, 500000 // ((hq + hk) * D // 128 + 1)), hq=hq, hk=hk,
                    D=D, rot=rot, layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                    n_pos=_log_int(rng, 4096, 200000), act=rng.choice(["bf16", "bf16", "f32"]))
    fmt = rng.choice(["bf16", "mxfp8", "mxfp8", "mxfp4", "f32"])
    D = rng.choice([64, 96, 128, 128, 256] + ([80] if fmt in ("bf16", "f32") else []))
    page = rng.choice([16, 16, 32, 48, 64, 128])
    if op in ("append", "store", "read"):
        most = {"append": 400000 // ((hq + 2 * hk) * D // 128 + 1),
                "store": 300000 // (hk * D // 64 + 1), "read": 500000 // (hk * D // 128 + 1)}[op]
        T = _log_int(rng, 1, most)
        c = dict(op=op, T=T, hk=hk, D=D, fmt=fmt, page=page,
                 pages=T // page + 1 + _log_int(rng, 1, 64))
        if op == "append":
            if fmt == "mxfp4":
                c["fmt"] = "mxfp8"  # 4-bit codes have no tensor type to be returned in: "store"
            rot = rng.choice([D, D, D // 2])
            c.update(hq=hq, rot=rot, layout=rng.choice(["half", "interleaved"]),
                     scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                     n_pos=_log_int(rng, 4096, 200000))
        return c
    row = 2 * hk * D * ROW_BYTES[fmt]
    B = _log_int(rng, 1, 160)
    hi = max(2, min(_log_int(rng, 16, 300000), int(1.5e9 / (B * row)),
                    int(4e9 / (B * 2 * hk * D * 4))))
    lo = rng.choice([0, 1, max(1, hi // 3), hi])
    return dict(op="attn", B=B, hq=hq, hk=hk, D=D, fmt=fmt, page=page, len_lo=lo, len_hi=hi,
                window=rng.choice([0, 0, 0, _log_int(rng, 1, 4096)]))


def _lengths(case):
    """Context length of each sequence: spread over [len_lo, len_hi], both ends
    taken (a property of the case, not of the seed)."""
    B, lo, hi = case["B"], case["len_lo"], case["len_hi"]
    out = [hi if b == 0 else lo if b == 1 else lo + (b * 2654435761 >> 7) % (hi - lo + 1)
           for b in range(B)]
    return out


def work(case):
    op, D, hk = case["op"], case["D"], case["hk"]
    if op == "rope":
        e = 4 if case["act"] == "f32" else 2
        n = case["T"] * (case["hq"] + hk)
        return {"bytes": 2 * n * D * e + case["T"] * (4 * case["rot"] + 4),
                "flops": 3 * n * case["rot"]}
    fmt = case["fmt"]
    row = D * ROW_BYTES[fmt] + (D // 32 if fmt in EMAX else 0)  # one head's key or value
    e = 4 if fmt == "f32" else 2
    if op == "attn":
        n = sum(min(x, case["window"]) if case["window"] else x for x in _lengths(case))
        return {"bytes": n * 2 * hk * row + case["B"] * case["hq"] * (2 * D * e + 4)
                + 4 * n / case["page"],
                "flops": 4 * n * case["hq"] * D}
    T = case["T"]
    if op == "append":
        return {"bytes": T * (2 * hk * (D * e + row) + 2 * case["hq"] * D * e + 4 * case["rot"]
                              + 8),
                "flops": 3 * T * (case["hq"] + hk) * case["rot"]}
    n = T * 2 * hk
    if op == "read":
        return {"bytes": n * (row + D * e) + 4 * T, "flops": n * D}
    return {"bytes": n * (2 * D * e + 2 * row) + 4 * T, "flops": 3 * n * D}


# ---- inputs ------------------------------------------------------------------------
def _gen(seed, salt=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + salt)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _table(case):
    """[n_pos][rot/2][2] cosines and sines of the scaled frequencies: what a
    program builds once. linear: positions / 4; ntk: base * 4^(r/(r-2)); yarn:
    frequencies blended between kept and divided by 4 over the turns they make in
    8192 positions (1 to 32), amplitude 0.1 ln 4 + 1."""
    r, base, factor, amp = case["rot"], 10000.0, 4.0, 1.0
    i = torch.arange(r // 2, dtype=torch.float64, device="cuda")
    if case["scaling"] == "ntk" and r > 2:
        base *= factor ** (r / (r - 2))
    w = base ** (-2 * i / r)
    if case["scaling"] == "linear":
        w = w / factor
    if case["scaling"] == "yarn":
        turns = 8192 * w / (2 * math.pi)
        keep = ((turns - 1) / 31).clamp(0, 1)
        w = w * keep + w / factor * (1 - keep)
        amp = 0.1 * math.log(factor) + 1
    a = torch.arange(case["n_pos"], dtype=torch.float64, device="cuda")[:, None] * w
    return torch.stack([a.cos() * amp, a.sin() * amp], -1).float()


def _e2m1(v):
    """Code of the nearest E2M1 value (ties to the even code), |v| saturated at 6."""
    a = v.abs().clamp(max=6.0)
    mids = torch.tensor([(GRID[j] + GRID[j + 1]) / 2 for j in range(7)], device=v.device,
                        dtype=v.dtype)
    code = torch.bucketize(a, mids, right=False)
    code = code + ((code < 7) & (code % 2 == 1) & (a == mids[code.clamp(max=6)]))
    return code.to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)


def _quantise(x, fmt):
    """fp32 [..][D] -> (codes, scale bytes [..][D/32]): OCP Microscaling blocks of
    32, scale 2^(floor(log2 amax) - emax), elements rounded to nearest even."""
    g = x.unflatten(-1, (-1, 32))
    amax = g.abs().amax(-1)
    ex = torch.where(amax > 0, torch.frexp(amax)[1] - 1 - EMAX[fmt], 0).clamp(-127, 127)
    inv = ((127 - ex) << 23).to(torch.int32).view(torch.float32)  # 2^-ex, exact
    v = (g * inv[..., None]).flatten(-2)
    if fmt == "mxfp8":
        code = v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        code = _e2m1(v)
        code = code[..., 0::2] | (code[..., 1::2] << 4)
    return code, (ex + 127).to(torch.uint8)


def _dequantise(code, scale, fmt, dtype=torch.float32):
    if fmt == "mxfp8":
        v = code.view(torch.float8_e4m3fn).to(dtype)
    else:
        grid = torch.tensor(GRID + tuple(-x for x in GRID), device=code.device, dtype=dtype)
        v = grid[torch.stack([code & 15, code >> 4], -1).flatten(-2).int()]
    s = (scale.int() << 23).view(torch.float32).to(dtype)  # 2^(scale - 127)
    return (v.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def _new_pool(case, g=None):
    """A pool of pages [pages][hk][page][row] for keys and one for values, with scale
    rows padded to 4 bytes; filled with a context's values (some key channels
    larger than others) when g is given."""
    hk, D, fmt, page, pages = case["hk"], case["D"], case["fmt"], case["page"], case["pages"]
    shape = (pages, hk, page)
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}.get(fmt, torch.uint8)
    cols = D // 2 if fmt == "mxfp4" else D
    state = {n: torch.zeros(*shape, cols, dtype=dt, device="cuda") for n in ("kc", "vc")}
    for n in ("ks", "vs"):
        state[n] = (torch.zeros(*shape, (D // 32 + 3) // 4 * 4, dtype=torch.uint8, device="cuda")
                    if fmt in EMAX else None)
    if g is not None:
        loud = torch.exp(0.5 * _randn(g, hk, 1, D))
        step = max(1, (1 << 26) // (hk * page * D))
        for p in range(0, pages, step):
            q = min(pages, p + step)
            for n, s, amp in (("kc", "ks", loud), ("vc", "vs", 1.0)):
                x = _randn(g, q - p, hk, page, D) * amp
                if fmt in EMAX:
                    state[n][p:q], state[s][p:q, ..., :D // 32] = _quantise(x, fmt)
                else:
                    state[n][p:q] = x.to(dt)
    return state


def prepare(case, seed):
    g = _gen(seed)
    op, D, hk = case["op"], case["D"], case["hk"]
    if op == "attn":
        lens = _lengths(case)
        page = case["page"]
        per = [-(-x // page) for x in lens]
        need = sum(per)
        case = dict(case, pages=need + 3)
        state = _new_pool(case, g)
        order = torch.randperm(need + 3, generator=g, device="cuda")[:need].int()
        table = torch.full((case["B"], max(1, max(per))), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(per):  # pages of a sequence in no order
            table[b, :n] = order[at:at + n]
            at += n
        dt = torch.float32 if case["fmt"] == "f32" else torch.bfloat16
        # q is a slice of the fused projection's output
        qkv = _randn(g, case["B"], (case["hq"] + 2 * hk) * D).to(dt)
        q = qkv[:, :case["hq"] * D].unflatten(-1, (case["hq"], D))
        state.update(case=case, q=q, table=table,
                     lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        return state
    T = case["T"]
    dt = torch.float32 if case.get("act", case.get("fmt")) == "f32" else torch.bfloat16
    hq = case.get("hq", 0)
    state = _new_pool(case, g if op == "read" else None) if op != "rope" else {}
    qkv = _randn(g, T, (hq + 2 * hk) * D).to(dt)
    cut = qkv.unflatten(-1, (-1, D))
    state.update(case=case, q=cut[:, :hq], k=cut[:, hq:hq + hk], v=cut[:, hq + hk:])
    if "rot" in case:
        state["rope_table"] = _table(case)
        state["pos"] = torch.randint(0, case["n_pos"], (T,), generator=g, device="cuda").int()
    if op != "rope":  # the tokens' places in the pool, pages in no order
        n = case["pages"]
        order = torch.randperm(n, generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        state["slots"] = (order[t // case["page"]] * case["page"] + t % case["page"]).int()
    return state


# ---- one pass ----------------------------------------------------------------------
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _returned(state):
    """The cache as it stands: 8-bit codes as the numbers they are, scale bytes."""
    if state["case"]["fmt"] == "mxfp8":
        return [state["kc"].view(torch.float8_e4m3fn), state["ks"],
                state["vc"].view(torch.float8_e4m3fn), state["vs"]]
    return [state["kc"], state["vc"]]


def _run_own(state):
    import mixture_experts_gb300 as moe
    case = state["case"]
    op = case["op"]
    if "handles" not in state:  # what a program keeps: views of its pool and its table
        state["handles"] = (
            moe.PagedKVCache(state["kc"], state["vc"], state["ks"], state["vs"],
                             case["D"]) if "kc" in state else None,
            moe.Rotary(state["rope_table"], case["layout"]) if "rot" in case else None)
    cache, rotary = state["handles"]
    if op == "rope":
        return moe.rope(rotary, state["pos"], state["q"], state["k"])
    if op == "append":
        q = cache.append(state["k"], state["v"], state["slots"], rotary=rotary,
                         positions=state["pos"], q=state["q"])
        return [q] + _returned(state)
    if op == "store":
        cache.append(state["k"], state["v"], state["slots"])
        return cache.read(state["slots"])
    if op == "read":
        return cache.read(state["slots"])
    return cache.attend(state["q"], state["table"], state["lens"], window=case["window"],
                        return_lse=True)


def _rotate(x, state):
    """fp32 rotation of the first rot elements of each head."""
    case = state["case"]
    r = case["rot"]
    cs = state["rope_table"][state["pos"].long()][:, None]
    c, s = cs[..., 0], cs[..., 1]
    x = x.float()
    if case["layout"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        return torch.cat([a * c - b * s, b * c + a * s, x[..., r:]], -1)
    a, b = x[..., 0:r:2], x[..., 1:r:2]
    y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([y, x[..., r:]], -1)


def _write(state, codes, scales, x):
    case = state["case"]
    slot = state["slots"].long()
    p, o = slot // case["page"], slot % case["page"]
    if case["fmt"] in EMAX:
        code, scale = _quantise(x, case["fmt"])
        state[codes][p, :, o] = code
        state[scales][:, :, :, :case["D"] // 32][p, :, o] = scale
    else:
        state[codes][p, :, o] = x.to(state[codes].dtype)


def _rows(state, codes, scales, p, o):
    """fp32 rows [..][hk][D] of the cache's places (page p, offset o)."""
    case = state["case"]
    x = state[codes][p, :, o]
    if case["fmt"] in EMAX:
        return _dequantise(x, state[scales][p, :, o][..., :case["D"] // 32], case["fmt"])
    return x.float()


def _run_plain(state):
    case = state["case"]
    op, D, hk = case["op"], case["D"], case["hk"]
    if op == "rope":
        return (_rotate(state["q"], state).to(state["q"].dtype),
                _rotate(state["k"], state).to(state["k"].dtype))
    if op == "append":
        q = _rotate(state["q"], state).to(state["q"].dtype)
        _write(state, "kc", "ks", _rotate(state["k"], state))
        _write(state, "vc", "vs", state["v"].float())
        return [q] + _returned(state)
    if op == "store":
        _write(state, "kc", "ks", state["k"].float())
        _write(state, "vc", "vs", state["v"].float())
    if op in ("store", "read"):
        slot = state["slots"].long()
        p, o = slot // case["page"], slot % case["page"]
        dt = state["k"].dtype
        return (_rows(state, "kc", "ks", p, o).to(dt), _rows(state, "vc", "vs", p, o).to(dt))
    # attention: every sequence padded to the longest, masked softmax
    B, hq, page = case["B"], case["hq"], case["page"]
    table, lens = state["table"].clamp(min=0).long(), state["lens"]
    L = table.shape[1] * page

    def context(codes, scales):
        x = state[codes][table]                      # [B][pages][hk][page][row]
        if case["fmt"] in EMAX:
            x = _dequantise(x, state[scales][table][..., :D // 32], case["fmt"])
        return x.float().transpose(1, 2).reshape(B, hk, L, D)

    j = torch.arange(L, device="cuda")
    last = lens[:, None]
    seen = j < last
    if case["window"]:
        seen = seen & (j >= last - case["window"])
    seen = seen[:, None, None]
    q = state["q"].float().reshape(B, hk, hq // hk, D)
    s = torch.matmul(q, context("kc", "ks").transpose(-1, -2)) * (D ** -0.5)
    s = torch.where(seen, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(s - top)
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, context("vc", "vs")) / torch.where(total > 0, total, 1.0)
    lse = torch.log(total) + top
    return o.reshape(B, hq, D).to(state["q"].dtype), lse.reshape(B, hq)


# ---- the definition in 64 bits -----------------------------------------------------
def _turn64(x, table, pos, rot, layout):
    """The rotation as a product of complex numbers."""
    t = table[pos.long()].double()
    z = torch.view_as_complex(t)[:, None]
    x = x.double()
    if layout == "half":
        y = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * z
        y = torch.cat([y.real, y.imag], -1)
    else:
        y = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], rot // 2, 2)) * z
        y = torch.view_as_real(y).reshape(*x.shape[:-1], rot)
    return torch.cat([y, x[..., rot:]], -1)


def _mx64(x, fmt):
    """(element values before the scale, exponent of the scale) of 64-bit rows."""
    blocks = x.reshape(*x.shape[:-1], -1, 32)
    amax = blocks.abs().max(-1).values
    e = torch.where(amax > 0, torch.floor(torch.log2(torch.where(amax > 0, amax, 1.0))), 0.0)
    e = torch.where(torch.exp2(e) > amax, e - 1, e)          # log2 may round up
    e = torch.where(torch.exp2(e + 1) <= amax, e + 1, e)
    e = torch.where(amax > 0, e - EMAX[fmt], 0.0)
    v = blocks * torch.exp2(-e)[..., None]
    # spacing of the format's values around v: 2^(exponent of v) / 2^(mantissa bits)
    bits, low, top = (3, -6, 448.0) if fmt == "mxfp8" else (1, 0, 6.0)
    n = torch.frexp(v)[1].double() - 1
    step = torch.exp2(n.clamp(min=low) - bits)
    v = (torch.round(v / step) * step).clamp(-top, top)
    return v, e


def _decode64(codes, scales, fmt):
    if fmt not in EMAX:
        return codes.double()
    if fmt == "mxfp8":
        c = torch.arange(256, device="cuda")
        e, m = (c >> 3) & 15, c & 7
        mag = torch.where(e == 0, m.double() * 2.0 ** -9,
                          (8 + m.double()) * torch.exp2(e.double() - 10))
        v = torch.where(c >= 128, -mag, mag)[codes.int()]
    else:
        c = torch.arange(16, device="cuda")
        e, m = (c >> 1) & 3, c & 1
        mag = torch.where(e == 0, m.double() * 0.5, (2 + m.double()) * torch.exp2(e.double() - 2))
        lut = torch.where(c >= 8, -mag, mag)
        v = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.float64,
                        device="cuda")
        v[..., 0::2], v[..., 1::2] = lut[(codes & 15).int()], lut[(codes >> 4).int()]
    s = torch.exp2(scales[..., :v.shape[-1] // 32].double() - 127)
    return v * s.repeat_interleave(32, -1)


def exact(case, seed):
    state = prepare(case, seed)
    op, D, hk = case["op"], case["D"], case["hk"]
    fmt = case.get("fmt")
    if op == "rope":
        return tuple(_turn64(state[n], state["rope_table"], state["pos"], case["rot"],
                             case["layout"]) for n in ("q", "k"))
    if op in ("append", "store", "read"):
        slot = state["slots"].long()
        at = (slot // case["page"], slice(None), slot % case["page"])
    if op == "append":
        rot = [state["rope_table"], state["pos"], case["rot"], case["layout"]]
        out = [_turn64(state["q"], *rot)]
        for codes, scales, x in (("kc", "ks", _turn64(state["k"], *rot)),
                                 ("vc", "vs", state["v"].double())):
            if fmt == "mxfp8":
                values = torch.zeros(state[codes].shape, dtype=torch.float64, device="cuda")
                v, e = _mx64(x, fmt)
                values[at] = v.flatten(-2)
                out += [values, None]
            else:
                values = state[codes].double()
                values[at] = x
                out.append(values)
        return out
    if op == "store":
        def stored(x):
            x = x.double()
            if fmt not in EMAX:
                return x
            v, e = _mx64(x, fmt)
            return (v * torch.exp2(e)[..., None]).flatten(-2)
        return stored(state["k"]), stored(state["v"])
    if op == "read":
        return tuple(_decode64(state[c][at], state[s][at] if fmt in EMAX else None, fmt)
                     for c, s in (("kc", "ks"), ("vc", "vs")))
    B, hq, page = case["B"], case["hq"], case["page"]
    out = torch.zeros(B, hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(case)):
        lo = max(0, n - case["window"]) if case["window"] else 0
        if n == 0:
            continue
        pages = state["table"][b, lo // page:-(-n // page)].long()
        skip = lo - lo // page * page
        for h in range(hk):
            def keys(codes, scales):
                sc = state[scales][pages, h] if fmt in EMAX else None
                return _decode64(state[codes][pages, h], sc, fmt).reshape(-1, D)[skip:skip + n - lo]
            g = slice(h * (hq // hk), (h + 1) * (hq // hk))
            s = state["q"][b, g].double() @ keys("kc", "ks").T / math.sqrt(D)
            lse[b, g] = torch.logsumexp(s, -1)
            out[b, g] = torch.softmax(s, -1) @ keys("vc", "vs")
    return out, lse
