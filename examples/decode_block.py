"""A transformer block at decode time: rotated attention over a paged, quantised
key-value cache, then the sparse MoE layer, step after step.

    python examples/decode_block.py [--format mxfp8] [--batch 8] [--steps 16]

Random weights (there is no checkpoint here). A prompt is written into the cache in one
call, then each step projects one new token a sequence, rotates its query and key on
the way into the cache, attends over the whole context and runs the experts. Prints the time
of a step's parts and, with --check, compares the attention with a plain fp32 one.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixture_experts_gb300 as moe  # noqa: E402

FORMATS = {"bf16": moe.BF16, "mxfp8": moe.MXFP8, "mxfp4": moe.MXFP4}


class Block:
    """Attention and experts of one layer, with the pages of its batch."""

    def __init__(self, batch, context, d=1024, n_heads=16, n_kv_heads=4, head_dim=64, experts=8,
                 top_k=2, d_ff=512, page=32, fmt="mxfp8", seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            w = torch.randn(*shape, generator=g, device="cuda") * shape[-1] ** -0.5
            return w.to(torch.bfloat16)
        self.hq, self.hk, self.D, self.page = n_heads, n_kv_heads, head_dim, page
        self.w_qkv = weight((n_heads + 2 * n_kv_heads) * head_dim, d)
        self.w_o = weight(d, n_heads * head_dim)
        self.layer = moe.MoELayer(d, d_ff, experts, top_k, batch, moe.BF16, moe.BF16, {
            "w_router": weight(experts, d), "b_router": None, "w_gate": weight(experts, d_ff, d),
            "w_up": weight(experts, d_ff, d), "w_down": weight(experts, d, d_ff)})
        self.rotary = moe.Rotary.build(head_dim, context, base=10000.0)
        per = -(-context // page)               # pages a sequence may grow to
        self.cache = moe.PagedKVCache.empty(batch * per, page, n_kv_heads, head_dim, FORMATS[fmt])
        self.table = torch.randperm(batch * per, generator=g, device="cuda").int().reshape(batch, per)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")

    def slots(self, seq, pos):
        """Pool places of position pos of sequence seq."""
        return self.table[seq.long(), (pos // self.page).long()] * self.page + pos % self.page

    def project(self, x):
        qkv = (x @ self.w_qkv.T).unflatten(-1, (-1, self.D))
        return qkv[:, :self.hq], qkv[:, self.hq:self.hq + self.hk], qkv[:, self.hq + self.hk:]

    def prompt(self, x):
        """Writes the keys and values of x [batch][tokens][d] (the cache is empty)."""
        B, n, d = x.shape
        seq = torch.arange(B, device="cuda").repeat_interleave(n)
        pos = torch.arange(n, device="cuda", dtype=torch.int32).repeat(B)
        _, k, v = self.project(x.reshape(-1, d))
        self.cache.append(k, v, self.slots(seq, pos).int(), rotary=self.rotary, positions=pos)
        self.lens += n

    def attention(self, x):
        """One new token a sequence: appends it, then attends over the context with it."""
        q, k, v = self.project(x)
        pos = self.lens.clone()
        place = self.slots(torch.arange(x.shape[0], device="cuda"), pos).int()
        q = self.cache.append(k, v, place, rotary=self.rotary, positions=pos, q=q)
        self.lens += 1
        return q, self.cache.attend(q, self.table, self.lens)

    def step(self, x):
        _, o = self.attention(x)
        x = x + o.flatten(1) @ self.w_o.T
        return x + self.layer(x)


def plain_attention(block, q):
    """fp32 attention over what the cache holds, read back."""
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    for b, n in enumerate(block.lens.tolist()):
        pos = torch.arange(n, device="cuda")
        k, v = block.cache.read(block.slots(torch.full_like(pos, b), pos).int())
        k, v = (x.float().repeat_interleave(block.hq // block.hk, 1) for x in (k, v))
        s = torch.einsum("hd,nhd->hn", q[b].float(), k) / math.sqrt(block.D)
        out[b] = torch.einsum("hn,nhd->hd", torch.softmax(s, -1), v)
    return out


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--format", choices=list(FORMATS), default="mxfp8")
    p.add_argument("--batch", type=int, default=8)
    p.add_argument("--prompt", type=int, default=500)
    p.add_argument("--steps", type=int, default=16)
    p.add_argument("--check", action="store_true")
    a = p.parse_args(argv)
    block = Block(a.batch, a.prompt + a.steps, fmt=a.format)
    g = torch.Generator(device="cuda").manual_seed(1)
    d = block.w_qkv.shape[1]
    block.prompt(torch.randn(a.batch, a.prompt, d, generator=g, device="cuda").bfloat16())
    x = torch.randn(a.batch, d, generator=g, device="cuda").bfloat16()
    worst = 0.0
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(a.steps - 1):
        y = block.step(x)
        x = torch.nn.functional.rms_norm(y.float(), (d,)).bfloat16()
    end.record()
    q, o = block.attention(x)
    if a.check:
        want = plain_attention(block, q)
        worst = float((o.float() - want).norm() / want.norm())
    torch.cuda.synchronize()
    assert moe.coli_device_status() == moe.COLI_OK
    line = f"{a.format}: {a.batch} sequences, {int(block.lens[0])} tokens"
    if a.steps > 1:
        line += f", {begin.elapsed_time(end) / (a.steps - 1):.3f} ms a step"
    print(line + (f", attention off by {worst:.2e}" if a.check else ""))
    return worst


if __name__ == "__main__":
    main()
