"""kv_attention under a window with a few first keys that stay visible, against
fp64 over what the cache stands for."""
import math

import numpy as np
import pytest
import torch

from oracle import kv as K
from tests.gpu_util import DEV, host64
from tests.test_gpu_kv import DTS, E32, U, fill, new_cache, randn

# (infinities are subtracted in the bounds and then left out)
pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore:invalid value encountered")]


@pytest.fixture(scope="module")
def W():
    from wht_adapters_amd import whtq
    return whtq


def ints(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x), dtype=dtype).to(DEV)


def starts(counts):
    return ints(np.cumsum([0] + list(counts)))


def seen(n, kv, causal, window, sinks):
    p, j = kv - n + np.arange(n)[:, None], np.arange(kv)
    return ((j <= p) | (not causal)) & ((j > p - window) | (window == 0) | (j < sinks))


def check(got, gl, q, k, v, scale, causal, window, sinks, dtype, int4):
    """got [n, heads, d], gl [n, heads] of one sequence.  A score is off by ds = (E32 (d + 8) + low) scale |q| |k| (norms
    bound sums of products in any rotated basis; low: a bf16 row's rotated query rounded to fp16), a probability by the
    relative 2 ds + its own rounding + 2^-20 (exp2, sums); fp16 probabilities vanish below 2^-33, rounded by 2^-25; one
    rounding of the result."""
    n, heads, d = q.shape
    group = heads // k.shape[1]
    um = 2.0 ** -11 if int4 else U[dtype]
    low = 2.0 ** -11 if int4 and dtype == torch.bfloat16 else 0.0
    m = seen(n, len(k), causal, window, sinks)
    any_key = m.any(0)
    for h in range(heads):
        kk, vv = (np.where(any_key[:, None], t[:, h // group], 0.0) for t in (k, v))  # what no query sees may be anything
        s = np.where(m, scale * (q[:, h] @ kk.T), -np.inf)
        top = s.max(-1, initial=-np.inf)
        none = ~np.isfinite(top)
        w = np.exp(s - np.where(none, 0, top)[:, None])
        total = np.where(none, 1, w.sum(-1))
        p = w / total[:, None]
        want, lse = p @ vv, np.where(none, -np.inf, top + np.log(total))
        assert (got[none, h] == 0).all() and (gl[none, h] == -np.inf).all()
        ds = (E32 * (d + 8) + low) * abs(scale) * np.linalg.norm(q[:, h], axis=-1) * np.linalg.norm(kk, axis=-1).max(initial=0)
        tiny = 0.0 if um > 2.0 ** -9 else m.sum(-1) * 2.0 ** -25 * np.abs(vv).max(initial=0) * math.sqrt(d)
        bound = (np.expm1(2 * ds) + um + 2.0 ** -20) * (p @ np.linalg.norm(vv, axis=-1)) + tiny + \
            U[dtype] * np.linalg.norm(want, axis=-1) + 2.0 ** -24 * math.sqrt(d)
        err = np.linalg.norm(got[:, h] - want, axis=-1)
        assert (err <= bound).all(), (h, np.argmax(err - bound), err.max(), bound.max())
        assert (np.abs(gl[:, h] - lse) <= ds + 2.0 ** -20 + 4 * E32 * np.abs(lse))[~none].all(), h


def test_the_mask_is_the_oracle_s():
    for n, kv, causal, window, sinks in ((3, 9, True, 2, 3), (2, 5, False, 1, 1), (4, 2, True, 3, 1), (1, 7, True, 9, 2)):
        m = seen(n, kv, causal, window, sinks)
        assert all(m[i, j] == K.sees(kv, n, i, j, causal, window, sinks) for i in range(n) for j in range(kv))


CASES = [
    # heads, kv heads, dim, page, (new, keys) of each sequence, causal, window, sinks
    (4, 2, 128, 16, [(1, 1)], True, 1, 1),
    (4, 4, 64, 16, [(1, 700), (1, 0), (1, 64), (1, 3)], True, 64, 4),
    (8, 1, 128, 32, [(1, 2000), (1, 31), (1, 129)], True, 33, 1),
    (6, 2, 64, 64, [(1, 900)], False, 100, 7),
    (16, 1, 64, 16, [(1, 1095)], True, 17, 64),              # sinks of whole tiles
    (8, 2, 128, 16, [(1, 1095), (1, 130)], True, 17, 65),    # sinks that end one key into a tile
    (17, 1, 128, 16, [(1, 70), (1, 900)], True, 40, 5),
    (4, 2, 128, 16, [(3, 5), (0, 9), (4, 2), (2, 640)], True, 3, 2),
    (8, 2, 64, 16, [(5, 1000), (1, 7)], True, 6, 3),
    (4, 2, 128, 16, [(2, 300), (1, 96), (3, 97)], True, 20, 70),   # sinks that reach the window's tile, or the window
    (4, 1, 64, 16, [(2, 300), (1, 50)], True, 20, 5000),     # sinks beyond the keys: all is seen
    (4, 2, 128, 16, [(70, 70), (3, 900), (33, 34)], True, 30, 4),
    (2, 2, 64, 64, [(130, 1900)], True, 200, 9),
    (3, 1, 128, 16, [(90, 1333)], True, 50, 130),
    (5, 5, 64, 16, [(65, 64), (40, 0)], True, 7, 3),
    (8, 2, 128, 128, [(64, 1290)], False, 31, 33),
    (14, 2, 64, 32, [(20, 1500), (1, 3), (75, 76)], True, 64, 20),
    (1, 1, 128, 16, [(200, 1000)], True, 64, 64),
    (2, 1, 64, 16, [(300, 700), (33, 640)], True, 100, 191),
]


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(W, case, dtype, int4):
    """Step and chunk kernel, split and unsplit keys.  The keys that no query sees are NaN, infinite, or (INT4) of huge
    scales, and pages that hold no other keys are gone from the table."""
    heads, hk, d, page, seqs, causal, window, sinks = CASES[case]
    rng = np.random.default_rng(500 + case)
    kls = [b for _, b in seqs]
    cache, sg = new_cache(W, rng, sum(-(-n // page) for n in kls) + 3, page, hk, d, dtype, int4, "token" if case % 2 else "head")
    table, slots, kvs = fill(W, rng, cache, sg, kls, hk, d, dtype, int4, page, 1.5)
    for b, (n, kv) in enumerate(seqs):
        hidden = np.flatnonzero(~seen(n, kv, causal, window, sinks).any(0)) if n else np.arange(0)
        s = slots[b][hidden]
        at = (ints(s // page, torch.int64), slice(None), ints(s % page, torch.int64))
        fill_with = ints(np.resize([np.nan, np.inf, -np.inf, 60000.0], len(s)), torch.float32)
        for t in ((cache.k_scales, cache.v_scales) if int4 else (cache.k, cache.v)):
            t[at] = fill_with.to(t.dtype).reshape(-1, *([1] * (t.dim() - 2))).expand(len(s), *t.shape[1:2], *t.shape[3:])
        for pg in range(kv // page):
            if np.isin(np.arange(pg * page, (pg + 1) * page), hidden).all():
                table[b, pg] = (-1, 1 << 30)[pg % 2]
    n = sum(a for a, _ in seqs)
    q = randn(rng, n, heads, d, dtype=dtype, scale=1.5)
    qst = np.cumsum([0] + [a for a, _ in seqs])
    scale = 0.9 / math.sqrt(d)
    lse = torch.empty((n, heads), device=DEV)
    most_q = max(a for a, _ in seqs)
    for mq, mk in ((most_q, max(kls)), (most_q, 1 << 16), (most_q, 0), (4096, max(kls)), (4096, 64)):
        lse.fill_(9.0)
        out = W.kv_attention(cache, q.to(DEV), ints(qst), ints(kls), ints(table), max_q_len=mq, max_kv_len=mk, scale=scale,
                             causal=causal, window=window, sinks=sinks, lse=lse)
        got, gl = host64(out), host64(lse)
        for b, (k, v) in enumerate(kvs):
            a, e = qst[b], qst[b + 1]
            check(got[a:e], gl[a:e], host64(q)[a:e], k, v, scale, causal, window, sinks, dtype, int4)


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("top,group", [(1, 2), (4, 2), (4, 5)])
def test_runs_over_many_sequences(W, d, dtype, int4, top, group):
    """70 ragged sequences on 32 key heads: runs of blocks go through sinks, gaps and windows of many of them."""
    rng = np.random.default_rng(92)
    hk, heads, page, seqs, window, sinks = 32, 32 * group, 16, 70, 70, 5
    counts = [0 if b % 11 == 10 else 1 + b % top for b in range(seqs)]
    lens = [int(x) for x in rng.integers(1, 90, seqs)]
    lens[3], lens[30], lens[31], lens[66], lens[68] = 1700, 0, 900, 2, 1100
    cache, sg = new_cache(W, rng, sum(-(-n // page) for n in lens) + 3, page, hk, d, dtype, int4)
    table, _, kvs = fill(W, rng, cache, sg, lens, hk, d, dtype, int4, page)
    q = randn(rng, sum(counts), heads, d, dtype=dtype)
    lse = torch.empty(sum(counts), heads, device=DEV)
    call = lambda: W.kv_attention(cache, q.to(DEV), starts(counts), ints(lens), ints(table), max_q_len=top,  # noqa: E731
                                  max_kv_len=max(lens), scale=0.1, window=window, sinks=sinks, lse=lse)
    out = call()
    got, gl, q64, at = host64(out), host64(lse), host64(q), 0
    for b, n in enumerate(counts):
        check(got[at:at + n], gl[at:at + n], q64[at:at + n], *kvs[b], 0.1, True, window, sinks, dtype, int4)
        at += n
    assert torch.equal(call(), out)


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("n", [1, 3, 80])
def test_special_sinks(W, n, int4):
    """No sinks, or no window: the bytes of the call without them.  Sinks or a window beyond the keys: what no mask gives."""
    rng = np.random.default_rng(93)
    dtype, hk, heads, d, page, kv = torch.float16, 2, 8, 64, 16, 500
    cache, sg = new_cache(W, rng, 40, page, hk, d, dtype, int4)
    table, _, kvs = fill(W, rng, cache, sg, [kv], hk, d, dtype, int4, page)
    q = randn(rng, n, heads, d, dtype=dtype)
    lse = torch.empty(n, heads, device=DEV)

    def call(**kw):
        return W.kv_attention(cache, q.to(DEV), ints([0, n]), ints([kv]), ints(table), max_q_len=n, max_kv_len=kv, scale=0.1,
                              lse=lse, **kw)
    assert torch.equal(call(window=60, sinks=0), call(window=60))
    assert torch.equal(call(sinks=7), call())
    for kw in (dict(window=60, sinks=kv), dict(window=60, sinks=2 ** 40), dict(window=2 ** 62, sinks=4), dict(window=kv, sinks=1)):
        out = call(**kw)
        check(host64(out), host64(lse), host64(q), *kvs[0], 0.1, True, 0, 0, dtype, int4)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("d,n", [(64, 5), (128, 3), (128, 90), (64, 90)])
def test_values_not_finite_reach_only_who_sees_them(W, bad, dtype, d, n):
    """One in the sinks (every query sees it), one that only the first queries' windows reach."""
    rng = np.random.default_rng(94)
    hk, heads, page, kv, window, sinks = 2, 4, 16, 600, 40, 6
    cache, _ = new_cache(W, rng, 40, page, hk, d, dtype, False)
    table, slots, kvs = fill(W, rng, cache, None, [kv], hk, d, dtype, False, page)
    k64, v64 = kvs[0]
    for j, col in ((3, 5), (kv - n - window + 2, 9)):
        s = slots[0][j]
        cache.v[s // page, 1, s % page, col] = bad
        v64[j, 1, col] = bad
    q = randn(rng, n, heads, d, dtype=dtype)
    with np.errstate(invalid="ignore"):
        want, _ = K.attention(host64(q), k64, v64, 0.1, True, window, sinks)
    for mq in (n, 4096):
        out = host64(W.kv_attention(cache, q.to(DEV), ints([0, n]), ints([kv]), ints(table), max_q_len=mq, max_kv_len=kv,
                                    scale=0.1, window=window, sinks=sinks))
        assert np.array_equal(np.isfinite(want), np.isfinite(out))
        fine = np.isfinite(want)
        assert np.all(np.abs(out - np.where(fine, want, 0))[fine] <= 4 * U[dtype])  # means of values of size about 1


def test_captured_and_replayed(W):
    """One workspace, lengths that grow between replays: the gap appears and moves."""
    rng = np.random.default_rng(95)
    dtype, hk, heads, d, page, kv, window, sinks = torch.bfloat16, 2, 8, 128, 16, 4000, 100, 4
    cache, sg = new_cache(W, rng, kv // page + 3, page, hk, d, dtype, False)
    table, _, kvs = fill(W, rng, cache, sg, [kv], hk, d, dtype, False, page)
    q, length, start, tb = randn(rng, 1, heads, d, dtype=dtype).to(DEV), ints([1]), ints([0, 1]), ints(table)
    ws = torch.empty(W.kv_attention_workspace_bytes(cache, 1, heads, 1, 1, kv, window, sinks), dtype=torch.uint8, device=DEV)
    lse = torch.empty(1, heads, device=DEV)
    call = lambda: W.kv_attention(cache, q, start, length, tb, max_q_len=1, max_kv_len=kv, scale=0.1, window=window,  # noqa: E731
                                  sinks=sinks, lse=lse, workspace=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for n in (1, 3, 103, 104, 140, 3999, 4000, 0):
        length.fill_(n)
        graph.replay()
        torch.cuda.synchronize()
        check(host64(out), host64(lse), host64(q), *(t[:n] for t in kvs[0]), 0.1, True, window, sinks, dtype, False)
        kept = out.clone()
        assert torch.equal(call(), kept)


def test_refusals(W):
    cache = W.kv_cache_alloc(4, 16, 2, 64, device=DEV)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(W.WhtqError):
        W.kv_attention(cache, q, ints([0, 1]), ints([1]), ints([[0]]), max_q_len=1, max_kv_len=1, window=4, sinks=-1)
    assert W.kv_attention_workspace_bytes(cache, 1, 4, 1, 1, 64, 4, -1) == -1
