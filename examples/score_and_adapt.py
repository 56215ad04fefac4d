"""A text scored while it streams through a decoder layer, and a training step
of QWHA adapters beside it.

score: a text longer than the window passes in chunks.  Queries and keys are
normed, rotated and cached in one pass (kv_append), each token sees the latest
`window` keys and the first `sinks` (kv_attention), an INT4 head gives logits,
and token_logprobs the log probability of every next token, the entropy and
the likeliest alternatives.  Run with a 16-bit and an INT4 cache, the two
scores say what the cache's 4 bits cost.

adapt: gradients of the values of two adapters on frozen INT4 projections: one
on the head, by the log probabilities of the next tokens (with a bonus for
entropy), and one on the queries, through their norms and rotation, by the
distance to another layer's queries and keys.

    python examples/score_and_adapt.py [--tokens 3000 --chunk 500 --window 1024 --sinks 4]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from kv_cache_decode import Attention, Linear, Pages  # noqa: E402
from wht_adapters_amd import synth, whtq  # noqa: E402


def score(layer, embed, head, tokens, chunk, page, int4, top=3, seen=None):
    """TokenLogprobs of each chunk of tokens (int64 [n]): of every token the next
    one's.  seen: a list to which (rotated queries, attention's output, logits)
    are added."""
    n = tokens.numel()
    pages = Pages(-(-n // page), page, 1, -(-n // page))
    cache = layer.cache(-(-n // page), page, int4)
    results = []
    for at in range(0, n, chunk):
        x, here = embed[tokens[at:at + chunk]], []
        hidden = x + layer(x, cache, pages, [x.shape[0]], here)
        logits = head(hidden)
        following = torch.full((x.shape[0],), -1, dtype=torch.int64, device=x.device)  # the last token has none
        following[:min(chunk, n - at - 1)] = tokens[at + 1:at + 1 + chunk]
        results.append(whtq.token_logprobs(logits, following, top=top))
        if seen is not None:
            seen.append((*here[0], logits, following))
    return results, cache, pages


class Adapter:
    """Sparse values in the Walsh-Hadamard domain beside a frozen projection."""

    def __init__(self, rows, n, entries, seed, device):
        rp, ci, vals = synth.sparse_adapter(seed, rows, n, entries)
        self.row_ptr, self.col_idx = torch.from_numpy(rp).to(device), torch.from_numpy(ci).to(device)
        self.vals, self.rows = vals.to(device), rows

    def __call__(self, x):
        return whtq.qwha_adapter_forward(x, self.row_ptr, self.col_idx, self.vals, self.rows)

    def gradient(self, x, dy):
        return whtq.qwha_adapter_grad_values(x, dy, self.row_ptr, self.col_idx)


def head_step(head, adapter, x, targets, bonus=0.01):
    """(logits, their TokenLogprobs, the gradient of the logits, of the adapter's values) of
    loss = -(mean logprob + bonus * mean entropy) of the rows that have a target."""
    logits = head(x) + adapter(x)
    r = whtq.token_logprobs(logits, targets)
    given = (targets >= 0).float()
    weight = -given / given.sum().clamp(min=1)
    dlogits = whtq.token_logprobs_backward(logits, targets, r, weight, bonus * weight)
    return logits, r, dlogits, adapter.gradient(x, dlogits)


def query_step(layer, adapter, x, positions, other):
    """(q, k, dq, gradients of the adapter's values, of q_norm and k_norm) of half the mean squared distance of the
    rotated queries and keys to `other`'s (q, k)."""
    rows = lambda y, h: y.view(-1, h, layer.dim)  # noqa: E731
    how = dict(layer.norms, cos=layer.cos, sin=layer.sin, positions=positions)
    q, k = rows(layer.wq(x) + adapter(x), layer.heads), rows(layer.wk(x), layer.kv_heads)
    outs = whtq.qk_norm_rope(q, k, **how)
    dq_out, dk_out = ((y - t) / x.shape[0] for y, t in zip(outs, other))
    dq, _, dq_norm, dk_norm = whtq.qk_norm_rope_backward(dq_out, dk_out, q, k, **how)
    return q, k, dq, adapter.gradient(x, dq.view(x.shape[0], -1)), dq_norm, dk_norm


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--tokens", type=int, default=3000)
    p.add_argument("--chunk", type=int, default=500)
    p.add_argument("--window", type=int, default=1024)
    p.add_argument("--sinks", type=int, default=4)
    p.add_argument("--vocab", type=int, default=4096)
    a = p.parse_args(argv)
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(3)
    layer = Attention(positions=a.tokens, norms=True, window=a.window, sinks=a.sinks)
    embed = torch.randn(a.vocab, 4096, device=dev, generator=gen).bfloat16()
    head = Linear(a.vocab, 4096, torch.randint(-2 ** 31, 2 ** 31 - 1, (128,), dtype=torch.int32, device=dev, generator=gen), gen)
    tokens = torch.randint(0, a.vocab, (a.tokens,), device=dev, generator=gen)
    for int4 in (False, True):
        results, _, _ = score(layer, embed, head, tokens, a.chunk, 64, int4)
        lp, ent = (torch.cat([getattr(r, name) for r in results])[:-1].mean().item() for name in ("logprob", "entropy"))
        print(f"{'INT4' if int4 else '16-bit'} cache: mean log probability {lp:.4f}, entropy {ent:.4f}, first alternatives "
              f"{results[0].top_id[0].tolist()}", flush=True)
    x, other = embed[tokens[:256]], Attention(positions=a.tokens, norms=True, seed=1)
    pos = torch.arange(256, dtype=torch.int32, device=dev)
    _, _, _, dc = head_step(head, Adapter(a.vocab, 4096, 65536, 1, dev), x, tokens[1:257])
    rows = lambda y, h: y.view(-1, h, layer.dim)  # noqa: E731
    target = whtq.qk_norm_rope(rows(other.wq(x), layer.heads), rows(other.wk(x), layer.kv_heads), **other.norms, cos=layer.cos,
                               sin=layer.sin, positions=pos)
    *_, dcq, dwq, dwk = query_step(layer, Adapter(4096, 4096, 65536, 2, dev), x, pos, target)
    print(f"gradients of {dc.numel()} values of the head: {dc.norm().item():.3e}, of {dcq.numel()} of the queries: "
          f"{dcq.norm().item():.3e}, of the norms: {dwq.norm().item():.3e} {dwk.norm().item():.3e}")


if __name__ == "__main__":
    main()
