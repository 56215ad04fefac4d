"""examples/score_and_adapt.py: norms, cache, windowed attention with sinks and
log probabilities in one run, and the gradients of a training step, against fp64."""
import os
import sys

import numpy as np
import pytest
import torch

from oracle import hadamard, kv as K, lm, qwha
from tests.gpu_util import DEV, host64

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
U, E32 = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module")
def small():
    """A layer of 32 heads on 8, its window and sinks, an embedding and a head."""
    import kv_cache_decode as D
    gen = torch.Generator(device=DEV).manual_seed(5)
    bits = torch.randint(-2 ** 31, 2 ** 31 - 1, (128,), dtype=torch.int32, device=DEV, generator=gen)
    layer = D.Attention(positions=400, norms=True, window=48, sinks=3)
    embed = torch.randn(1000, 4096, device=DEV, generator=gen).bfloat16()
    return layer, embed, D.Linear(1000, 4096, bits, gen), torch.randint(0, 1000, (211,), device=DEV, generator=gen)


@pytest.mark.parametrize("int4", [False, True])
def test_score(small, int4):
    import score_and_adapt as E
    from wht_adapters_amd import whtq as W
    layer, embed, head, tokens = small
    seen = []
    results, cache, pages = E.score(layer, embed, head, tokens, 50, 16, int4, seen=seen)
    n = tokens.numel()
    assert pages.length == [n] and sum(r.top_id.shape[0] for r in results) == n
    j = np.arange(n)
    slots = pages.table.numpy()[0, j // 16].astype(np.int64) * 16 + j % 16
    k, v = (host64(t) for t in W.kv_gather(cache, torch.from_numpy(slots).to(DEV)))
    if not int4:  # the cached keys are the projection's, normed and rotated: one rounding, fp32 before it
        x = embed[tokens]
        raw = host64(layer.wk(x).view(-1, 8, 128))
        want = lm.norm_rope(raw, host64(layer.norms["k_norm"]), 1e-6, host64(layer.cos)[:n], host64(layer.sin)[:n])
        size = np.abs(raw * lm.rms(raw, 1e-6) * host64(layer.norms["k_norm"])).max(-1, keepdims=True) * 2
        # (the projection's products of another batch may be rounded apart: half a step of bf16 more of the row's size)
        assert np.all(np.abs(k - want) <= U * np.abs(want) + (U + 32 * E32) * size)
    at = 0
    for (q, o, logits, following), r in zip(seen, results):
        m, kv = q.shape[0], at + q.shape[0]
        qq, got = host64(q), host64(o)
        want, _ = K.attention(qq, k[:kv], v[:kv], 128 ** -0.5, True, layer.window, layer.sinks)
        mean, _ = K.attention(qq, k[:kv], np.abs(v[:kv]), 128 ** -0.5, True, layer.window, layer.sinks)
        # as for the layer alone: the probabilities' and the result's rounding, for INT4 what gather rounds, and what
        # fp32 sums (INT4: gather's and the rotated query's rounding) move a score
        heads = [np.abs(qq[:, h]) @ np.abs(k[:kv, h // 4]).T for h in range(32)]
        ds = (E32 * (128 + 8) + (2.0 ** -9 + 2.0 ** -12 if int4 else 0.0)) * 128 ** -0.5 * np.max(heads)
        assert np.linalg.norm(got - want) <= (U * (3 if int4 else 2) + np.expm1(2 * ds)) * np.linalg.norm(mean)
        t = following.cpu().numpy()
        assert t.tolist() == tokens[at + 1:kv + 1].tolist() + ([-1] if kv == n else [])
        ref = lm.logprobs(host64(logits), t, top=3)
        # 1000 logits: two chunks, sums of 8 and 64 terms; exponents below 64
        assert np.all(np.abs(host64(r.logprob) - ref["logprob"]) <= E32 * 512)
        assert np.all(np.abs(host64(r.entropy) - ref["entropy"]) <= E32 * 2048)
        assert np.array_equal(r.top_id.cpu().numpy(), ref["top_id"])
        at = kv
    assert at == n


def test_gradients(small):
    import score_and_adapt as E
    layer, embed, head, tokens = small
    x = embed[tokens[:60]]
    targets = tokens[1:61].clone()
    targets[[4, 17]] = -1
    adapter = E.Adapter(1000, 4096, 9000, 1, DEV)
    logits, r, dlogits, dc = E.head_step(head, adapter, x, targets, 0.1)
    t = targets.cpu().numpy()
    w = -1.0 * (t >= 0) / (t >= 0).sum()
    want = lm.logprobs_backward(host64(logits), t, w, 0.1 * w)
    # one rounding, and fp32 of the probability (64 units: exponents below 16, sums) times its bracket (below 20 |w|)
    p = np.exp(host64(logits) - lm.logprobs(host64(logits), t)["lse"][:, None])
    assert np.all(np.abs(host64(dlogits) - want) <= U * np.abs(want) + 2.0 ** -134 + 128 * E32 * 20 * np.abs(w)[:, None] * p + 8 * E32 * np.abs(want))
    rp, ci = adapter.row_ptr.cpu().numpy(), adapter.col_idx.cpu().numpy()
    x64 = host64(x)
    dc64 = qwha.qwha_grad_values(x64, want, rp, ci)
    mass = qwha.qwha_grad_values(x64, host64(dlogits), rp, ci)
    z = np.abs(hadamard.wht(x64))
    rows = np.repeat(np.arange(1000), np.diff(rp))
    room = np.einsum("te,te->e", np.abs(want)[:, rows], z[:, ci])
    # the gradient's own rounding in every term, the products' fp32 (1e-5 of the sum's mass, as for them alone)
    assert np.all(np.abs(host64(dc) - dc64) <= (U * 1.01 + 1e-5) * room + 1e-5 * np.sqrt(np.mean(mass ** 2)))

    qa = E.Adapter(4096, 4096, 40000, 2, DEV)
    pos = torch.arange(60, dtype=torch.int32, device=DEV)
    other = [torch.randn(60, h, 128, device=DEV).bfloat16() for h in (32, 8)]
    q, k, dq, dcq, dwq, dwk = E.query_step(layer, qa, x, pos, other)
    cos, sin = host64(layer.cos)[:60], host64(layer.sin)[:60]
    from wht_adapters_amd import whtq as W
    outs = W.qk_norm_rope(q, k, **layer.norms, cos=layer.cos, sin=layer.sin, positions=pos)
    for raw, w, y, tgt, dw in ((q, "q_norm", outs[0], other[0], dwq), (k, "k_norm", outs[1], other[1], dwk)):
        dy = host64((y - tgt) / 60)
        dx64, dw64 = lm.norm_rope_backward(dy, host64(raw), host64(layer.norms[w]), 1e-6, cos, sin)
        top = np.abs(dy).max(-1, keepdims=True) * 2
        massw = (top * np.abs(host64(raw)) * lm.rms(host64(raw), 1e-6)).sum((0, 1))
        # as many additions as terms at most, each term off by its turn, its norm and two products
        assert np.all(np.abs(host64(dw) - dw64) <= (dy.shape[0] * dy.shape[1] + 64) * E32 * massw)
        if w == "q_norm":
            r = lm.rms(host64(raw), 1e-6)
            size = r * top * np.abs(host64(layer.norms[w])).max()
            size = size + r ** 3 * np.abs(host64(raw)) * np.mean(np.abs(host64(raw)) * top * 2, -1, keepdims=True)
            assert np.all(np.abs(host64(dq) - dx64) <= U * np.abs(dx64) + 80 * E32 * size)
    dcq64 = qwha.qwha_grad_values(x64, host64(dq).reshape(60, -1), qa.row_ptr.cpu().numpy(), qa.col_idx.cpu().numpy())
    assert np.all(np.abs(host64(dcq) - dcq64) <= 1e-5 * np.abs(dcq64) + 1e-5 * np.sqrt(np.mean(dcq64 ** 2)))


def test_example_runs(capsys):
    import score_and_adapt as E
    E.main(["--tokens", "300", "--chunk", "128", "--window", "64", "--vocab", "1024"])
    text = capsys.readouterr().out
    assert "16-bit cache: mean log probability" in text and "INT4 cache: mean log probability" in text
    assert "gradients of" in text and "nan" not in text
