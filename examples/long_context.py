"""Long contexts at decode time: a batch of chats behind one shared prompt, attending to
chosen pages of what each said itself, and evicting what was worth least.

    python examples/long_context.py [--format mxfp8] [--batch 16] [--steps 200]

Random weights and projections (there is no checkpoint here). The prompt's pages are written
once and shared by every sequence. Each step appends one token a sequence, attends to the whole
context (the prompt read once for the batch) and adds what each own token weighed to its mass;
every second layer would attend to a few pages only, which the step also does and compares.
When a sequence outgrows its budget, its least heavy tokens leave the cache.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixture_experts_gb300 as moe  # noqa: E402

FORMATS = {"f32": moe.F32, "bf16": moe.BF16, "mxfp8": moe.MXFP8, "mxfp4": moe.MXFP4}


class Chats:
    """The caches of one layer: a shared prompt and pages of each sequence's own."""

    def __init__(self, batch, prompt, budget, n_heads=16, n_kv_heads=4, head_dim=64, page=16,
                 fmt="mxfp8", seed=0):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.hq, self.hk, self.D, self.page = n_heads, n_kv_heads, head_dim, page
        self.budget, self.prompt = budget, prompt
        per = -(-budget // page) + 2          # a sequence grows by up to two pages before a cut
        pre = -(-prompt // page)
        self.cache = moe.PagedKVCache.empty(pre + batch * per, page, n_kv_heads, head_dim,
                                            FORMATS[fmt])
        self.rotary = moe.Rotary.build(head_dim, prompt + 100000)
        self.prefix = torch.arange(pre, dtype=torch.int32, device="cuda")
        self.table = (pre + torch.arange(batch * per, dtype=torch.int32, device="cuda")
                      ).reshape(batch, per)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.longest, self.step_no = 0, 0     # the host knows both: every sequence grows alike
        self.bounds, self.mass = self.cache.new_bounds(), self.cache.new_mass()
        rows = self.project(prompt)
        pos = torch.arange(prompt, dtype=torch.int32, device="cuda")
        self.cache.append(rows[:, n_heads:n_heads + n_kv_heads], rows[:, n_heads + n_kv_heads:],
                          (self.prefix[pos.long() // page] * page + pos % page).int(),
                          rotary=self.rotary, positions=pos)

    def project(self, n):
        """Stands for a fused projection: [n][query, key and value heads][head_dim]."""
        x = torch.randn(n, self.hq + 2 * self.hk, self.D, generator=self.g, device="cuda")
        return x.to(self.cache.act_torch)

    def step(self, keep=4):
        """(attention over everything, over the chosen pages of the own tokens)"""
        B, c = self.table.shape[0], self.cache
        rows = self.project(B)
        at = self.table.gather(1, (self.lens.long() // self.page)[:, None])[:, 0]
        place = self.lens % self.page
        pos = torch.full((B,), self.prompt + self.step_no, dtype=torch.int32, device="cuda")
        q = c.append(rows[:, self.hq:self.hq + self.hk], rows[:, self.hq + self.hk:],
                     at * self.page + place, rotary=self.rotary, positions=pos, q=rows[:, :self.hq])
        c.page_bounds(self.bounds, at, place + 1)
        known = self.lens.clone()
        self.lens += 1
        self.longest += 1
        self.step_no += 1
        out, lse = c.attend_shared(q, self.prefix, self.prompt, self.table, self.lens,
                                   return_lse=True)
        c.accumulate(self.mass, q, self.table, self.lens, lse, known=known)
        pages, held = c.select_pages(q, self.bounds, self.table, self.lens, keep)
        few = c.attend_selected(q, pages, held)
        if self.longest == self.budget + self.page:
            self.cut()
        return out, few

    def cut(self):
        _, self.lens = self.cache.evict(self.mass, self.table, self.lens, self.budget, first=2,
                                        recent=self.budget // 4)
        self.longest = self.budget
        n = -(-self.budget // self.page)      # the pages that hold other tokens now
        fills = torch.full((n,), self.page, dtype=torch.int32, device="cuda")
        fills[-1] = self.budget - (n - 1) * self.page
        self.cache.page_bounds(self.bounds, self.table[:, :n].flatten().contiguous(),
                               fills.repeat(self.table.shape[0]))


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--format", choices=list(FORMATS), default="mxfp8")
    p.add_argument("--batch", type=int, default=16)
    p.add_argument("--prompt", type=int, default=2000)
    p.add_argument("--budget", type=int, default=128)
    p.add_argument("--steps", type=int, default=200)
    a = p.parse_args(argv)
    chats = Chats(a.batch, a.prompt, a.budget, fmt=a.format)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(a.steps):
        out, few = chats.step()
    end.record()
    torch.cuda.synchronize()
    assert moe.coli_device_status() == moe.COLI_OK
    assert torch.isfinite(out.float()).all() and torch.isfinite(few.float()).all()
    print(f"{a.format}: {a.batch} sequences behind {a.prompt} tokens, {int(chats.lens[0])} tokens "
          f"of {a.steps} kept, {begin.elapsed_time(end) / a.steps:.3f} ms a step")
    return chats


if __name__ == "__main__":
    main()
