"""Measured cases of what keeps long contexts affordable over the paged key-value
cache: attention of a batch that shares a long prefix, attention over pages that a
cheap score selects, and eviction by accumulated attention weight.

Each case is one pass through one operator as a decode step (or the step between
two) calls it. `run` computes it with elementary torch operations (`own` false) or
through the package's entry points (`own` true), on the same inputs.
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
        # a few chats behind one short system prompt: latency
        dict(name="shared_short", op="shared", B=8, hq=32, hk=8, D=128, fmt="bf16", page=16,
             prefix=1500, len_lo=1, len_hi=300),
        # a decode batch behind one long document
        dict(name="shared_batch_bf16", op="shared", B=64, hq=32, hk=8, D=128, fmt="bf16", page=16,
             prefix=32768, len_lo=16, len_hi=512),
        # a large batch on an 8-bit cache, the prefix ending inside a page
        dict(name="shared_large_mxfp8", op="shared", B=128, hq=64, hk=8, D=128, fmt="mxfp8",
             page=64, prefix=40009, len_lo=1, len_hi=1000),
        # fp32 layer with heads of 80, one sequence with nothing of its own yet
        dict(name="shared_odd_f32", op="shared", B=5, hq=20, hk=4, D=80, fmt="f32", page=48,
             prefix=777, len_lo=0, len_hi=99),
        # a decode step's newest pages get their bounds again
        dict(name="bounds_decode", op="bounds", pages=64, hk=8, D=128, fmt="bf16", page=32),
        # the bounds of a long prompt's 8-bit pages, the last of them part filled
        dict(name="bounds_prompt_mxfp8", op="bounds", pages=4099, hk=8, D=128, fmt="mxfp8",
             page=64),
        # one user with half a million tokens of context, 64 pages of it read
        dict(name="sparse_one_long", op="sparse", B=1, hq=32, hk=8, D=128, fmt="bf16", page=64,
             len_lo=500009, len_hi=500009, keep=64, first=1, last=2),
        # a ragged decode batch on an 8-bit cache
        dict(name="sparse_batch_mxfp8", op="sparse", B=32, hq=32, hk=8, D=128, fmt="mxfp8",
             page=32, len_lo=700, len_hi=65536, keep=64, first=1, last=2),
        # what each cached token was worth to a ragged decode batch
        dict(name="mass_batch_bf16", op="mass", B=32, hq=32, hk=8, D=128, fmt="bf16", page=16,
             len_lo=300, len_hi=8192, window=0),
        # long 4-bit contexts, 16 query heads a key head
        dict(name="mass_long_mxfp4", op="mass", B=16, hq=64, hk=4, D=128, fmt="mxfp4", page=32,
             len_lo=1, len_hi=60000, window=0),
        # a batch that has outgrown its budget by some pages
        dict(name="evict_steady", op="evict", B=64, hk=8, D=128, fmt="bf16", page=32,
             len_lo=2049, len_hi=2176, keep=2048, first=4, recent=256),
        # prompts cut down to the budget on an 8-bit cache, one of them within it
        dict(name="evict_prompts_mxfp8", op="evict", B=8, hk=8, D=128, fmt="mxfp8", page=64,
             len_lo=2000, len_hi=32768, keep=2048, first=4, recent=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["shared", "shared", "bounds", "sparse", "sparse", "mass", "mass", "evict"])
    fmt = rng.choice(["bf16", "bf16", "mxfp8", "mxfp8", "mxfp4", "f32"])
    D = rng.choice([64, 96, 128, 128, 256] + ([80] if fmt in ("bf16", "f32") else []))
    page = rng.choice([16, 16, 32, 48, 64, 128])
    hk = rng.choice([1, 2, 4, 8, 8, 16])
    hq = hk * rng.choice([1, 2, 4, 5, 8, 16])
    c = dict(op=op, hk=hk, D=D, fmt=fmt, page=page)
    row = 2 * hk * D  # numbers of a token in the cache
    if op == "bounds":
        c["pages"] = _log_int(rng, 1, max(2, int(2e9 / (page * row * 2))))
        return c
    B = _log_int(rng, 1, 128)
    most = int(2e9 / (B * row * 2))  # tokens a sequence may have
    if op == "shared":
        hi = max(2, min(_log_int(rng, 8, 2048), most))
        top = min(65536, int(1e9 / row), int(3e8 / (B * hq)), int(4e10 / (B * hq * D)))
        c.update(B=B, hq=hq, prefix=_log_int(rng, 1, max(2, top)))
    elif op == "sparse":
        hi = max(2, min(_log_int(rng, 16, 500000), most, int(3e8 * page / (B * row))))
        first, last = rng.choice([0, 1, 1, 2]), rng.choice([1, 1, 2, 4])
        c.update(B=B, hq=hq, keep=first + last + _log_int(rng, 1, min(128, max(2, hi // page))),
                 first=first, last=last)
    elif op == "mass":
        hi = max(2, min(_log_int(rng, 16, 300000), most))
        c.update(B=B, hq=hq, window=rng.choice([0, 0, 0, _log_int(rng, 1, 4096)]))
    else:
        if fmt == "mxfp4":
            c["fmt"] = "mxfp8"  # 4-bit codes have no tensor type to be returned in
        hi = max(40, min(_log_int(rng, 40, 60000), most // 2))
        first, recent = rng.choice([0, 1, 4]), _log_int(rng, 1, 16)
        c.update(B=B, keep=max(first + recent, _log_int(rng, 20, hi)), first=first, recent=recent)
    c.update(len_lo=rng.choice([0, 1, max(1, hi // 3), hi]), len_hi=hi)
    return c


def _lengths(case):
    """Tokens of each sequence: spread over [len_lo, len_hi], both ends taken (a
    property of the case, not of the seed)."""
    B, lo, hi = case["B"], case["len_lo"], case["len_hi"]
    return [hi if b == 0 else lo if b == 1 else lo + (b * 2654435761 >> 7) % (hi - lo + 1)
            for b in range(B)]


def _fills(case):
    """Tokens in each page of a bounds case: prompts fill them, the last of each
    prompt (or every page, in a decode step of up to 64) only in part."""
    n, page = case["pages"], case["page"]
    return [1 + (i * 40503 >> 3) % page if n <= 64 or i % 61 == 60 else page for i in range(n)]


def work(case):
    op, D, hk, fmt = case["op"], case["D"], case["hk"], case["fmt"]
    row = D * ROW_BYTES[fmt] + (D // 32 if fmt in EMAX else 0)  # one head's key or value
    e = 4 if fmt == "f32" else 2
    if op == "bounds":
        n = sum(_fills(case))
        return {"bytes": n * hk * row + case["pages"] * (2 * hk * D * e + 8),
                "flops": 2 * n * hk * D}
    lens, page, B = _lengths(case), case["page"], case["B"]
    if op == "shared":
        n, q = case["prefix"] + sum(lens), case["hq"] * D
        return {"bytes": n * (2 * hk * row + 4 / page) + B * (2 * q * e + 4 * case["hq"]),
                "flops": 4 * (case["prefix"] * B + sum(lens)) * q}
    pages = [-(-n // page) for n in lens]
    if op == "sparse":
        seen = sum(n if p <= case["keep"] else n - (p - case["keep"]) * page
                   for n, p in zip(lens, pages))
        look = sum(p for p in pages if p > case["keep"])
        q = case["hq"] * D
        return {"bytes": seen * 2 * hk * row + look * (2 * hk * D * e + 4)
                + B * (2 * q * e + 4 * case["hq"] + 4 * hk * case["keep"]),
                "flops": 4 * seen * q + 2 * look * q}
    if op == "mass":
        n = sum(min(x, case["window"]) if case["window"] else x for x in lens)
        return {"bytes": n * hk * (row + 8) + 4 * n / page + B * case["hq"] * (D * e + 4),
                "flops": 2 * n * case["hq"] * D}
    kept = sum(min(n, case["keep"]) for n in lens)
    over = sum(n for n in lens if n > case["keep"])
    return {"bytes": kept * hk * (4 * row + 8 + 4) + over * hk * 4, "flops": over * hk}


# ---- inputs ------------------------------------------------------------------------
def _gen(seed, salt=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + salt)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


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


def _dequantise(code, scale, fmt):
    if fmt == "mxfp8":
        v = code.view(torch.float8_e4m3fn).float()
    else:
        grid = torch.tensor(GRID + tuple(-x for x in GRID), device=code.device)
        v = grid[torch.stack([code & 15, code >> 4], -1).flatten(-2).int()]
    s = (scale.int() << 23).view(torch.float32)  # 2^(scale - 127)
    return (v.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def _pool(case, pages, g):
    """Pools of keys and of values [pages][hk][page][row] with a context's numbers in
    them (some key channels larger than others), scale rows padded to 4 bytes."""
    hk, D, fmt, page = case["hk"], case["D"], case["fmt"], case["page"]
    shape = (pages, hk, page)
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}.get(fmt, torch.uint8)
    cols = D // 2 if fmt == "mxfp4" else D
    state = {n: torch.zeros(*shape, cols, dtype=dt, device="cuda") for n in ("kc", "vc")}
    for n in ("ks", "vs"):
        state[n] = (torch.zeros(*shape, (D // 32 + 3) // 4 * 4, dtype=torch.uint8, device="cuda")
                    if fmt in EMAX else None)
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


def _act(case):
    return torch.float32 if case["fmt"] == "f32" else torch.bfloat16


def _tables(counts, pool, width):
    """int32 [len(counts)][width]: the pool's page numbers in their order, counts[b] of
    them to row b, the rest -1; and how many were taken."""
    table, at = torch.full((len(counts), width), -1, dtype=torch.int32, device="cuda"), 0
    for b, n in enumerate(counts):
        table[b, :n] = pool[at:at + n]
        at += n
    return table, at


def prepare(case, seed):
    g = _gen(seed)
    op, D, hk, page = case["op"], case["D"], case["hk"], case["page"]
    if op == "bounds":
        n = case["pages"]
        state = _pool(case, n + 3, g)
        state.update(case=case,
                     pages=torch.randperm(n + 3, generator=g, device="cuda")[:n].int(),
                     fills=torch.tensor(_fills(case), dtype=torch.int32, device="cuda"),
                     bounds=torch.zeros(n + 3, hk, 2, D, dtype=_act(case), device="cuda"))
        return state
    lens = _lengths(case)
    per = [-(-n // page) for n in lens]
    spare = -(-case.get("prefix", 0) // page)
    if op == "evict":
        spare = case["B"] * -(-case["keep"] // page)
    total = sum(per) + spare + 3
    state = _pool(case, total, g)
    order = torch.randperm(total, generator=g, device="cuda").int()  # pages in no order
    table, at = _tables(per, order, max(1, max(per)))
    state.update(case=case, table=table, spare=order[-1].long(),
                 lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    if op != "evict":
        # q is a slice of the fused projection's output
        qkv = _randn(g, case["B"], (case["hq"] + 2 * hk) * D).to(_act(case))
        state["q"] = qkv[:, :case["hq"] * D].unflatten(-1, (case["hq"], D))
    if op == "shared":
        state["prefix"] = order[at:at + spare].contiguous()
    if op == "sparse":  # what the steps before this one left: bounds of every page
        state["bounds"] = torch.zeros(total, hk, 2, D, dtype=_act(case), device="cuda")
        fills = torch.full((total,), page, device="cuda")
        for b, n in enumerate(lens):
            if n:
                fills[table[b, per[b] - 1]] = n - (per[b] - 1) * page
        step = max(1, (1 << 26) // (hk * page * D))
        for p in range(0, total, step):
            at = torch.arange(p, min(total, p + step), device="cuda")
            state["bounds"][at] = _plain_bounds(state, at, fills[at])
    if op in ("mass", "evict"):  # weights summed over earlier steps: few tokens hold most
        u = torch.rand(total, hk, page, generator=g, device="cuda")
        state["mass"] = 0.02 / (0.001 + u)
    if op == "mass":
        # what attention over the same context returned beside its output
        state["known"] = (state["lens"] - 1).clamp(min=0).int()
        s, seen = _scores(state, state["table"], state["lens"], case["window"])
        state["lse"] = torch.logsumexp(s, -1).reshape(case["B"], case["hq"])
    if op == "evict":
        keep = -(-case["keep"] // page)
        state["into"], _ = _tables([keep] * case["B"], order[at:], keep)
    return state


# ---- one pass ----------------------------------------------------------------------
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _rows_moved(state):
    """The pools as they stand: 8-bit codes as the numbers they are, scale bytes."""
    if state["case"]["fmt"] == "mxfp8":
        return [state["kc"].view(torch.float8_e4m3fn), state["ks"],
                state["vc"].view(torch.float8_e4m3fn), state["vs"], state["mass"]]
    return [state["kc"], state["vc"], state["mass"]]


def _run_own(state):
    import mixture_experts_gb300 as moe
    case = state["case"]
    op = case["op"]
    if "cache" not in state:  # what a program keeps: a view of its pool
        state["cache"] = moe.PagedKVCache(state["kc"], state["vc"], state["ks"], state["vs"],
                                          case["D"])
    cache = state["cache"]
    if op == "shared":
        return cache.attend_shared(state["q"], state["prefix"], case["prefix"], state["table"],
                                   state["lens"], return_lse=True)
    if op == "bounds":
        cache.page_bounds(state["bounds"], state["pages"], state["fills"])
        return state["bounds"]
    if op == "sparse":
        pages, lens = cache.select_pages(state["q"], state["bounds"], state["table"],
                                         state["lens"], case["keep"], first=case["first"],
                                         last=case["last"])
        out, lse = cache.attend_selected(state["q"], pages, lens, return_lse=True)
        return out, lse, pages, lens
    if op == "mass":
        cache.accumulate(state["mass"], state["q"], state["table"], state["lens"], state["lse"],
                         known=state["known"], window=case["window"])
        return state["mass"]
    kept, lens = cache.evict(state["mass"], state["table"], state["lens"], case["keep"],
                             first=case["first"], recent=case["recent"], into=state["into"])
    return [kept, lens] + _rows_moved(state)


def _rows(state, codes, scales, pages):
    """fp32 rows [..][hk][page][D] of whole pages."""
    case = state["case"]
    x = state[codes][pages]
    if case["fmt"] in EMAX:
        return _dequantise(x, state[scales][pages][..., :case["D"] // 32], case["fmt"])
    return x.float()


def _plain_bounds(state, pages, fills):
    """[pages][hk][2][D]: least and largest key of each channel among a page's tokens."""
    k = _rows(state, "kc", "ks", pages)
    dead = torch.arange(k.shape[2], device="cuda") >= fills[:, None]
    dead = dead[:, None, :, None]
    return torch.stack([torch.where(dead, math.inf, k).amin(2),
                        torch.where(dead, -math.inf, k).amax(2)], 2).to(_act(state["case"]))


def _context(state, codes, scales, table):
    """fp32 [B][hk][tokens][D] of whole block tables (entries below 0: any page)."""
    x = _rows(state, codes, scales, table.clamp(min=0).long())  # [B][pages][hk][page][D]
    return x.transpose(1, 2).flatten(2, 3)


def _scores(state, table, lens, window=0):
    """Scaled scores [B][hk][group][tokens] (-inf out of sight) and what is in sight."""
    case = state["case"]
    B, hk, D = case["B"], case["hk"], case["D"]
    q = state["q"].float().reshape(B, hk, -1, D)
    s = torch.matmul(q, _context(state, "kc", "ks", table).transpose(-1, -2)) * D ** -0.5
    j = torch.arange(s.shape[-1], device="cuda")
    last = lens[:, None]
    seen = j < last
    if window:
        seen = seen & (j >= last - window)
    seen = seen[:, None, None]
    return torch.where(seen, s, -math.inf), seen


def _weigh(s, values):
    """Weights exp(s - max) by values: (largest score, sum of weights, weighted sum)."""
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(s - top)
    return top, e.sum(-1, keepdim=True), torch.matmul(e, values)


def _plain_shared(state):
    case = state["case"]
    B, hq, hk, D, n = case["B"], case["hq"], case["hk"], case["D"], case["prefix"]
    # the prefix once, for the queries of all sequences together
    q = state["q"].float().reshape(B, hk, hq // hk, D).transpose(0, 1).reshape(hk, -1, D)
    k, v = (_context(state, c, s, state["prefix"][None])[0, :, :n]
            for c, s in (("kc", "ks"), ("vc", "vs")))
    m0, l0, o0 = (x.unflatten(1, (B, -1)).transpose(0, 1) for x in
                  _weigh(torch.matmul(q, k.transpose(-1, -2)) * D ** -0.5, v))
    # each sequence's own tokens, padded to the longest
    s, _ = _scores(state, state["table"], state["lens"])
    m1, l1, o1 = _weigh(s, _context(state, "vc", "vs", state["table"]))
    m1 = torch.where(l1 > 0, m1, -math.inf)
    top = torch.maximum(m0, m1)
    f0, f1 = torch.exp(m0 - top), torch.exp(m1 - top)
    total = l0 * f0 + l1 * f1
    return (((o0 * f0 + o1 * f1) / total).reshape(B, hq, D).to(state["q"].dtype),
            (torch.log(total) + top).reshape(B, hq))


def _picked(value, count, take, low, high):
    """Places of the `take` largest of value [..][n] among the first count [..] places,
    in rising order (-1 past them): below `low` and from count - high on always; of
    equal values the lower place."""
    n = value.shape[-1]
    j = torch.arange(n, device="cuda")
    value = torch.where(torch.isnan(value), -math.inf, value).double()
    value = torch.where((j < low) | (j >= (count - high)[..., None]), math.inf, value)
    place = torch.sort(value, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(place).scatter_(-1, place, j.expand_as(place))
    # places out of sight are all in the last part, which counts as taken: only those in sight
    more = (n - count)[..., None]
    some = (j < count[..., None]) & ((rank < take + more) | (count[..., None] <= take))
    at = torch.cumsum(some, -1) - 1
    out = torch.full((*value.shape[:-1], take + 1), -1, dtype=torch.int64, device="cuda")
    out.scatter_(-1, torch.where(some, at, take), j.expand_as(at))
    return out[..., :take]


def _plain_sparse(state):
    case = state["case"]
    B, hq, hk, D, page, keep = (case[n] for n in ("B", "hq", "hk", "D", "page", "keep"))
    table, lens = state["table"].clamp(min=0).long(), state["lens"].long()
    # no key of a page scores higher than this; in 64 bits, since pages are ranked by it
    q = state["q"].double().reshape(B, hk, -1, D)
    pages = table.shape[1]
    best = torch.empty(B, hk, pages, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 28) // (B * hk * 2 * D))
    for p in range(0, pages, step):
        b = state["bounds"][table[:, p:p + step]].double()  # [B][pages][hk][2][D]
        b = b.permute(0, 2, 3, 4, 1)                        # [B][hk][2][D][pages]
        best[:, :, p:p + step] = (torch.matmul(q.clamp(max=0), b[:, :, 0]) +
                                  torch.matmul(q.clamp(min=0), b[:, :, 1])).amax(2)
    count = -(-lens // page)
    place = _picked(best, count[:, None].expand(B, hk), keep, case["first"], case["last"])
    chosen = torch.where(place >= 0, table[:, None].expand(B, hk, -1).gather(2, place.clamp(min=0)),
                         -1)
    seen = torch.where(count > keep, lens - (count - keep) * page, lens)
    h = torch.arange(hk, device="cuda")[:, None]
    at = chosen.clamp(min=0)

    def rows(codes, scales):                                # [B][hk][keep][page][D]
        x = state[codes][at, h]
        if case["fmt"] in EMAX:
            x = _dequantise(x, state[scales][at, h][..., :D // 32], case["fmt"])
        return x.float().flatten(2, 3)

    s = torch.matmul(state["q"].float().reshape(B, hk, -1, D),
                     rows("kc", "ks").transpose(-1, -2)) * D ** -0.5
    in_sight = torch.arange(keep * page, device="cuda") < seen[:, None]
    s = torch.where(in_sight[:, None, None], s, -math.inf)
    top, total, o = _weigh(s, rows("vc", "vs"))
    o = o / torch.where(total > 0, total, 1.0)
    return (o.reshape(B, hq, D).to(state["q"].dtype), (torch.log(total) + top).reshape(B, hq),
            chosen.int(), seen.int())


def _places(state, table, n):
    """Flat places [B][hk][n] of the first n tokens in mass [pages][hk][page]."""
    case = state["case"]
    hk, page = case["hk"], case["page"]
    j = torch.arange(n, device="cuda")
    p = table.clamp(min=0).long()[:, j // page]
    return (p[:, None] * hk + torch.arange(hk, device="cuda")[:, None]) * page + j % page


def _plain_mass(state):
    case = state["case"]
    B, hk = case["B"], case["hk"]
    s, seen = _scores(state, state["table"], state["lens"], case["window"])
    lse = state["lse"].reshape(B, hk, -1, 1)
    w = torch.where(seen, torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)), 0.0).sum(2)
    n = w.shape[-1]
    spot = state["spare"] * hk * case["page"]  # a place that no sequence has
    flat = state["mass"].view(-1)
    seen = seen[:, 0].expand_as(w)
    at = torch.where(seen, _places(state, state["table"], n), spot)
    old = torch.arange(n, device="cuda") < state["known"][:, None]
    new = torch.where(old[:, None], flat[at], 0.0) + w
    flat[at] = torch.where(seen, new, flat[spot])
    return state["mass"]


def _plain_evict(state):
    case = state["case"]
    B, hk, page, keep = case["B"], case["hk"], case["page"], case["keep"]
    lens = state["lens"].long()
    flat = state["mass"].view(-1)
    from_ = _places(state, state["table"], state["table"].shape[1] * page)
    kept = _picked(flat[from_], lens[:, None].expand(B, hk), keep, case["first"], case["recent"])
    into = _places(state, state["into"], keep)
    spot = state["spare"] * hk * page  # a place that no sequence has
    some = kept >= 0
    src = torch.where(some, from_.gather(2, kept.clamp(min=0)), spot)
    dst = torch.where(some, into, spot)
    for name in ("kc", "vc", "ks", "vs", "mass"):
        if state[name] is not None:
            rows = state[name].view(-1, *state[name].shape[3:])
            rows[dst] = rows[src]
    return [kept.int(), lens.clamp(max=keep).int()] + _rows_moved(state)


def _run_plain(state):
    op = state["case"]["op"]
    if op == "bounds":
        state["bounds"][state["pages"].long()] = _plain_bounds(state, state["pages"].long(),
                                                              state["fills"])
        return state["bounds"]
    return {"shared": _plain_shared, "sparse": _plain_sparse, "mass": _plain_mass,
            "evict": _plain_evict}[op](state)


# ---- the definition in 64 bits -----------------------------------------------------
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


def _keys64(state, codes, scales, pages, h, n):
    """The first n rows [n][D] of head h of a list of pages."""
    sc = state[scales][pages, h] if state["case"]["fmt"] in EMAX else None
    x = _decode64(state[codes][pages, h], sc, state["case"]["fmt"])
    return x.reshape(-1, x.shape[-1])[:n]


def _largest64(values, take, low, high):
    """Places of the `take` largest of a list of numbers, see the operators."""
    n = len(values)
    if n <= take:
        return list(range(n))
    must = set(range(min(low, n))) | set(range(max(0, n - high), n))
    rest = sorted((j for j in range(n) if j not in must), key=lambda j: (-values[j], j))
    return sorted(list(must) + rest[:take - len(must)])


def exact(case, seed):
    state = prepare(case, seed)
    op, D, hk, fmt, page = (case[n] for n in ("op", "D", "hk", "fmt", "page"))
    if op == "bounds":
        out = state["bounds"].double()
        for p, f in zip(state["pages"].tolist(), state["fills"].tolist()):
            k = _decode64(state["kc"][p], state["ks"][p] if fmt in EMAX else None, fmt)[:, :f]
            out[p, :, 0], out[p, :, 1] = k.min(1).values, k.max(1).values
        return out
    B, lens = case["B"], _lengths(case)
    table = state["table"].tolist()
    if op in ("shared", "sparse", "mass"):
        hq = case["hq"]
        G = hq // hk
        q = state["q"].double()
        out = torch.zeros(B, hq, D, dtype=torch.float64, device="cuda")
        lse = torch.full((B, hq), -math.inf, dtype=torch.float64, device="cuda")
    if op == "shared":
        pre = state["prefix"].long()
        for h in range(hk):
            g = slice(h * G, (h + 1) * G)
            k0 = _keys64(state, "kc", "ks", pre, h, case["prefix"])
            v0 = _keys64(state, "vc", "vs", pre, h, case["prefix"])
            for b in range(B):
                own_pages = torch.tensor(table[b], device="cuda")[:-(-lens[b] // page)]
                s0 = q[b, g] @ k0.T / math.sqrt(D)
                s1 = q[b, g] @ _keys64(state, "kc", "ks", own_pages, h, lens[b]).T / math.sqrt(D)
                lse[b, g] = torch.logsumexp(torch.cat([s0, s1], -1), -1)
                out[b, g] = torch.exp(s0 - lse[b, g, None]) @ v0
                out[b, g] += (torch.exp(s1 - lse[b, g, None]) @
                              _keys64(state, "vc", "vs", own_pages, h, lens[b]))
        return out, lse
    if op == "sparse":
        for b, n in enumerate(lens):
            count = -(-n // page)
            mine = torch.tensor(table[b], device="cuda")[:count]
            seen = n - max(0, count - case["keep"]) * page
            for h in range(hk):
                g = slice(h * G, (h + 1) * G)
                box = state["bounds"][mine, h].double()     # [pages][2][D]
                score = torch.full((count,), -math.inf, dtype=torch.float64, device="cuda")
                for i in range(h * G, (h + 1) * G):
                    one = (torch.where(q[b, i] > 0, box[:, 1], box[:, 0]) * q[b, i]).sum(-1)
                    score = torch.maximum(score, one)
                pick = _largest64(score.tolist(), case["keep"], case["first"], case["last"])
                pages = mine[torch.tensor(pick, dtype=torch.int64, device="cuda")]
                if n == 0:
                    continue
                s = q[b, g] @ _keys64(state, "kc", "ks", pages, h, seen).T / math.sqrt(D)
                lse[b, g] = torch.logsumexp(s, -1)
                out[b, g] = torch.softmax(s, -1) @ _keys64(state, "vc", "vs", pages, h, seen)
        return out, lse, None, None
    if op == "mass":
        mass = state["mass"].double()
        for b, n in enumerate(lens):
            lo = max(0, n - case["window"]) if case["window"] else 0
            if n == 0:
                continue
            mine = torch.tensor(table[b], device="cuda")[:-(-n // page)]
            j = torch.arange(lo, n, device="cuda")
            for h in range(hk):
                g = slice(h * G, (h + 1) * G)
                k = _keys64(state, "kc", "ks", mine, h, n)[lo:]
                w = torch.exp(q[b, g] @ k.T / math.sqrt(D) - state["lse"][b, g, None].double())
                old = mass[mine[j // page], h, j % page]
                mass[mine[j // page], h, j % page] = (torch.where(j < n - 1, old, 0.0) +
                                                      w.sum(0))
        return mass
    moved = {n: state[n].clone() for n in ("kc", "vc", "ks", "vs", "mass")
             if state[n] is not None}
    into = state["into"]
    for b, n in enumerate(lens):
        mine = torch.tensor(table[b], device="cuda")
        for h in range(hk):
            j = torch.arange(n, device="cuda")
            pick = _largest64(state["mass"][mine[j // page], h, j % page].tolist(), case["keep"],
                              case["first"], case["recent"])
            src = torch.tensor(pick, dtype=torch.int64, device="cuda")
            r = torch.arange(len(pick), device="cuda")
            for name, pool in moved.items():
                pool[into[b].long()[r // page], h, r % page] = \
                    state[name][mine[src // page], h, src % page]
    if fmt == "mxfp8":
        return [None, None, _decode64(moved["kc"], torch.full_like(moved["ks"], 127), fmt), None,
                _decode64(moved["vc"], torch.full_like(moved["vs"], 127), fmt), None,
                moved["mass"].double()]
    return [None, None, moved["kc"].double(), moved["vc"].double(), moved["mass"].double()]
