"""The layer of examples/kv_cache_decode.py: what its prompt and its steps
attend to, against fp64 attention over what the cache stands for."""
import os
import sys

import numpy as np
import pytest
import torch

from oracle import kv as K
from tests.gpu_util import DEV, host64

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("prompts", [[41, 7, 130], [1]])
def test_decode_layer(int4, prompts):
    import kv_cache_decode as E
    from wht_adapters_amd import whtq as W
    layer = E.Attention(positions=max(prompts) + 3)
    seen = []
    outs, _, _, cache, pages = E.decode(layer, prompts, 3, 16, int4, seen=seen)
    assert [o.shape[0] for o in outs] == [sum(prompts)] + [len(prompts)] * 3
    rows = []
    for b, n in enumerate(pages.length):
        j = np.arange(n)
        slots = pages.table.numpy()[b, j // 16].astype(np.int64) * 16 + j % 16
        k, v = W.kv_gather(cache, torch.from_numpy(slots).to(DEV))
        rows.append((host64(k), host64(v)))
    scale = layer.dim ** -0.5
    at = [n for n in prompts]
    for step, (q, o) in enumerate(seen):
        counts = prompts if step == 0 else [1] * len(prompts)
        lo = 0
        for b, n in enumerate(counts):
            kl = at[b] if step == 0 else at[b] + step
            qq, got = host64(q)[lo:lo + n], host64(o)[lo:lo + n]
            k, v = (t[:kl] for t in rows[b])
            want, _ = K.attention(qq, k, v, scale, True, 0)
            mean, _ = K.attention(qq, k, np.abs(v), scale, True, 0)
            # relative to the mean of |v|, 2^-8 each: the probabilities' rounding, the result's, and for INT4 what
            # gather rounds of v; a score is off by fp32 sums, for INT4 also by gather's rounding of k (2^-9 of a
            # value) and the rotated query's (2^-12), and a probability by twice the largest
            heads = [np.abs(qq[:, h]) @ np.abs(k[:, h // (layer.heads // layer.kv_heads)]).T for h in range(layer.heads)]
            ds = (2.0 ** -24 * (layer.dim + 8) + (2.0 ** -9 + 2.0 ** -12 if int4 else 0.0)) * scale * np.max(heads)
            bound = (2.0 ** -8 * (3 if int4 else 2) + np.expm1(2 * ds)) * np.linalg.norm(mean)
            assert np.linalg.norm(got - want) <= bound, (step, b)
            lo += n


def test_example_runs(capsys):
    import kv_cache_decode as E
    E.main(["--seqs", "2", "--prompt", "40", "--steps", "3", "--page", "16"])
    text = capsys.readouterr().out
    assert "16-bit cache: 4096 bytes a token" in text and "INT4 cache: 1056 bytes a token" in text
