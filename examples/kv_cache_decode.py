"""One attention layer of a decoder served from low-bit storage: projections
kept as INT4 codes of their rows' RHT (rht_lowbit_gemv), keys and values in a
paged cache (kv_append, kv_attention), 16-bit or INT4.

Several sequences of different lengths get their prompts in one call, then
decode in step.  Every call takes its sizes from the host and its positions,
lengths and tables from device tensors that one copy a step fills.

    python examples/kv_cache_decode.py [--seqs 8 --prompt 700 --steps 32 --page 64]

prints the time of a prompt and of a step with either cache, the bytes that a
cached token takes, and how far the INT4 cache moves the layer's output.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from wht_adapters_amd import whtq  # noqa: E402


class Linear:
    """A weight [rows, n] stored as INT4 codes of its rows' RHT, one scale per 128."""

    def __init__(self, rows, n, signs, gen):
        w = (torch.randn(rows, n, device=gen.device, generator=gen) * n ** -0.5).bfloat16()
        self.signs = signs
        self.codes, self.scales = whtq.rht_quantize_rtn(w, signs, 4, 128)

    def __call__(self, x):
        return whtq.rht_lowbit_gemv(x, self.codes, self.scales, self.signs, 4, 128)


class Pages:
    """Which pages of a cache each sequence owns; page_size slots a page."""

    def __init__(self, pages, page_size, seqs, width):
        self.free, self.page = list(range(pages))[::-1], page_size
        self.table = torch.zeros((seqs, width), dtype=torch.int32)
        self.length = [0] * seqs

    def extend(self, counts):
        """Slots of counts[b] more tokens of each sequence b, sequence by sequence."""
        slots = []
        for b, n in enumerate(counts):
            for j in range(self.length[b], self.length[b] + n):
                if j % self.page == 0:
                    self.table[b, j // self.page] = self.free.pop()
                slots.append(int(self.table[b, j // self.page]) * self.page + j % self.page)
            self.length[b] += n
        return slots


class Attention:
    def __init__(self, hidden=4096, heads=32, kv_heads=8, dim=128, positions=8192, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        bits = lambda n: torch.randint(-2 ** 31, 2 ** 31 - 1, (n // 32,), dtype=torch.int32, device=device, generator=gen)
        self.heads, self.kv_heads, self.dim, self.device = heads, kv_heads, dim, torch.device(device)
        self.cache_signs = bits(dim)
        signs = bits(hidden)
        self.wq = Linear(heads * dim, hidden, signs, gen)
        self.wk = Linear(kv_heads * dim, hidden, signs, gen)
        self.wv = Linear(kv_heads * dim, hidden, signs, gen)
        self.wo = Linear(hidden, heads * dim, bits(heads * dim), gen)
        angle = torch.arange(positions, dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(0, dim, 2, dtype=torch.float64) / dim)
        self.cos, self.sin = angle.cos().float().to(device), angle.sin().float().to(device)

    def cache(self, pages, page_size, int4):
        return whtq.kv_cache_alloc(pages, page_size, self.kv_heads, self.dim, int4=int4,
                                   signs=self.cache_signs if int4 else None, device=self.device)

    def __call__(self, x, cache, pages, counts, seen=None):
        """x: the new tokens' rows, counts[b] of each sequence b.  seen: a list
        to which the rotated queries and the attention's output are added."""
        first = list(pages.length)
        slots = pages.extend(counts)
        put = lambda v, t: torch.tensor(v, dtype=t).to(self.device, non_blocking=True)
        pos = put([first[b] + i for b, n in enumerate(counts) for i in range(n)], torch.int32)
        start = put([sum(counts[:b]) for b in range(len(counts) + 1)], torch.int32)
        length, table = put(pages.length, torch.int32), pages.table.to(self.device, non_blocking=True)

        rows = lambda y, h: y.view(-1, h, self.dim)
        q, k, v = rows(self.wq(x), self.heads), rows(self.wk(x), self.kv_heads), rows(self.wv(x), self.kv_heads)
        q = whtq.kv_append(cache, k, v, put(slots, torch.int64), q=q, q_out=q, cos=self.cos, sin=self.sin, positions=pos)
        o = whtq.kv_attention(cache, q, start, length, table, max_q_len=max(counts), max_kv_len=max(pages.length))
        if seen is not None:
            seen.append((q, o))
        return self.wo(o.view(-1, self.heads * self.dim))


def decode(layer, prompts, steps, page_size, int4, seed=1, seen=None):
    """Prompts of the given lengths, then `steps` tokens of each sequence.
    Returns (outputs of every call, seconds of the prompt, seconds of a step,
    cache, pages)."""
    gen = torch.Generator(device=layer.device).manual_seed(seed)
    hidden = layer.wo.codes.shape[0]
    width = -(-(max(prompts) + steps) // page_size)
    total = sum(-(-(n + steps) // page_size) for n in prompts)
    cache, pages = layer.cache(total, page_size, int4), Pages(total, page_size, len(prompts), width)
    new = lambda n: torch.randn(n, hidden, device=layer.device, generator=gen).bfloat16()
    outs, times = [], []
    for counts in [list(prompts)] + [[1] * len(prompts)] * steps:
        x = new(sum(counts))
        torch.cuda.synchronize()
        t = time.perf_counter()
        outs.append(layer(x, cache, pages, counts, seen))
        torch.cuda.synchronize()
        times.append(time.perf_counter() - t)
    return outs, times[0], sorted(times[1:])[steps // 2] if steps else 0.0, cache, pages


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--seqs", type=int, default=8)
    p.add_argument("--prompt", type=int, default=700, help="the longest prompt; the others are shorter")
    p.add_argument("--steps", type=int, default=32)
    p.add_argument("--page", type=int, default=64)
    a = p.parse_args(argv)
    layer = Attention(positions=a.prompt + a.steps)
    prompts = [max(1, a.prompt - a.prompt * b // (2 * a.seqs)) for b in range(a.seqs)]
    runs = {}
    for int4 in (False, True):
        decode(layer, prompts, 2, a.page, int4)  # first calls load the library's kernels
        outs, first, step, cache, _ = decode(layer, prompts, a.steps, a.page, int4)
        nbytes = sum(t[0].nbytes for t in (cache.k, cache.v, cache.k_scales, cache.v_scales) if t is not None) / a.page
        runs[int4] = torch.cat(outs).double()
        print(f"{'INT4' if int4 else '16-bit'} cache: {nbytes:.0f} bytes a token, prompt of {sum(prompts)} tokens "
              f"{first * 1e3:.2f} ms, step of {a.seqs} sequences {step * 1e6:.0f} us", flush=True)
    moved = (runs[True] - runs[False]).norm() / runs[False].norm()
    print(f"the INT4 cache moves the layer's output by {moved:.1%}")


if __name__ == "__main__":
    main()
