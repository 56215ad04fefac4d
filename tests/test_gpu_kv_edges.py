"""The paged key/value cache at its edges, against fp64: runs that cross
sequences, values and scales that are not finite, tiny queries, tiny
probabilities, lengths and grids out of the ordinary."""
import math

import numpy as np
import pytest
import torch

from oracle import rtn
from tests.gpu_util import DEV, host64
from tests.test_gpu_kv import DTS, E32, U, check, fill, new_cache, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def W():
    from wht_adapters_amd import whtq
    return whtq


def ints(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x), dtype=dtype).to(DEV)


def starts(counts):
    return ints(np.cumsum([0] + list(counts)))


def stored(cache, sg, slots, d):
    """fp64 (k, v) [slots, kv_heads, d] of an INT4 cache, from its codes and scales."""
    page, out = cache.page_size, []
    for codes, scales in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
        c = codes.cpu().numpy()[slots // page, :, slots % page]
        s = scales.cpu().numpy()[slots // page, :, slots % page]
        out.append(rtn.dequantize_inverse(c.reshape(-1, d // 2), s.reshape(-1, 1), sg, 4, d, d).reshape(*s.shape, d))
    return out


def reference(q, k, v, scale, window, low):
    """out, lse [n, heads, ..] in fp64, causal, and a bound on the 2-norm of an output row's error.  Norms bound sums of
    products in any rotated basis: a score is off by ds = (E32 (d + 8) + low) scale |q| |k|, low for a rotated query's
    rounding to fp16; u is the probabilities' rounding."""
    n, heads, d = q.shape
    group = heads // k.shape[1]
    kk, vv = (np.repeat(t, group, 1) for t in (k, v))
    s = scale * np.einsum("ihd,jhd->ihj", q, kk)
    p, j = len(k) - n + np.arange(n)[:, None, None], np.arange(len(k))
    s = np.where((j <= p) & ((j > p - window) | (window == 0)), s, -np.inf)
    top = np.where(np.isfinite(s.max(-1, initial=-np.inf)), s.max(-1, initial=-np.inf), 0.0)
    w = np.exp(s - top[..., None])
    total = w.sum(-1)
    w /= np.where(total == 0, 1.0, total)[..., None]
    with np.errstate(divide="ignore"):
        lse = top + np.log(total)
    norm = lambda t: np.linalg.norm(t, axis=-1)  # noqa: E731
    ds = (E32 * (d + 8) + low) * scale * norm(q).max(-1, initial=0) * norm(kk).max(initial=0)
    mean = np.einsum("ihj,jh->ih", w, norm(vv))
    return np.einsum("ihj,jhd->ihd", w, vv), lse, ds, mean


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,int4,top,window,poison,group", [
    (dtype, int4, *rest) for dtype in DTS for int4 in (False, True)
    for rest in ((1, 0, False, 2), (4, 0, False, 2), (4, 50, False, 2), (4, 0, True, 2), (4, 0, False, 5))
    if not (rest[2] if int4 else rest[3] > 4)])  # 20 rows a key head: INT4 alone has a step kernel for them
def test_runs_over_many_sequences(W, d, dtype, int4, top, window, poison, group):
    """70 ragged sequences on 32 key heads (a few blocks a head): a block's run of keys goes through many sequences, the
    runs are of two lengths, some begin after the 64th sequence, and long sequences reach over several.  Poisoned: the
    last value of every second sequence is not finite on every head, which only its last query sees."""
    rng = np.random.default_rng(91)
    hk, heads, page, seqs = 32, 32 * group, 16, 70
    counts = [0 if b % 11 == 10 else 1 + b % top for b in range(seqs)]
    lens = [int(x) for x in rng.integers(1, 60, seqs)]
    lens[3], lens[30], lens[31], lens[66], lens[68] = 1700, 0, 900, 2, 1100
    cache, sg = new_cache(W, rng, sum(-(-n // page) for n in lens) + 3, page, hk, d, dtype, int4)
    table, slots, kvs = fill(W, rng, cache, sg, lens, hk, d, dtype, int4, page)
    bad = [b for b in range(0, seqs, 2) if poison and lens[b] > 4 and counts[b] > 1]
    for b in bad:
        s = int(slots[b][-1])
        cache.v[s // page, :, s % page, :] = (float("nan"), float("inf"))[b % 8 // 4]
    q = randn(rng, sum(counts), heads, d, dtype=dtype)
    lse = torch.empty(sum(counts), heads, device=DEV)
    args = (q.to(DEV), starts(counts), ints(lens), ints(table))
    out = W.kv_attention(cache, *args, max_q_len=top, max_kv_len=max(lens), scale=0.1, window=window, lse=lse)
    got, gl, q64, at = host64(out), host64(lse), host64(q), 0
    um, low = (2.0 ** -11 if int4 else U[dtype]), (2.0 ** -11 if int4 and dtype == torch.bfloat16 else 0.0)
    for b, n in enumerate(counts):
        want, wl, ds, mean = reference(q64[at:at + n], *kvs[b], 0.1, window, low)
        tiny = 0.0 if um > 2.0 ** -9 else lens[b] * 2.0 ** -25
        bound = ((np.expm1(2 * ds)[:, None] + um + 2.0 ** -20) * mean + tiny * np.abs(kvs[b][1]).max(initial=0) * math.sqrt(d) +
                 U[dtype] * np.linalg.norm(want, axis=-1) + 2.0 ** -24 * math.sqrt(d))
        err = np.linalg.norm(got[at:at + n] - want, axis=-1)
        sees = np.ones(n, bool)
        if b in bad:
            sees[-1] = False
            assert not np.isfinite(got[at + n - 1]).any(), b
        assert (err <= bound)[sees].all(), (b, err.max(), bound.max())
        fine = np.isfinite(wl)
        assert np.array_equal(np.isfinite(gl[at:at + n]), fine)
        gl0, wl0 = (np.where(fine, t, 0.0) for t in (gl[at:at + n], wl))
        assert (np.abs(gl0 - wl0) <= ds[:, None] + 2.0 ** -20 + 4 * E32 * np.abs(wl0)).all(), b
        at += n
    if not poison:  # the same bytes again
        again = W.kv_attention(cache, *args, max_q_len=top, max_kv_len=max(lens), scale=0.1, window=window)
        assert torch.equal(again, out)


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("mq,most", [(4, 64), (4, 1 << 16), (4096, 64), (4096, 1 << 16)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 5), (False, 7)])
def test_lengths_are_held_to_the_table(W, int4, mq, most, causal, window):
    """Lengths below 0 count as 0, lengths beyond the table as its width."""
    rng = np.random.default_rng(81)
    hk, heads, d, page, width = 2, 4, 64, 16, 3
    dtype = torch.bfloat16
    cache, sg = new_cache(W, rng, 9, page, hk, d, dtype, int4)
    table, _, kvs = fill(W, rng, cache, sg, [48, 48], hk, d, dtype, int4, page)
    table = np.concatenate([table[:, :width], np.zeros((4, width), np.int32)])
    lens = [48, 2 ** 31 - 1, -1, -2 ** 31, -2 ** 31 + 2, 0]
    none = (np.zeros((0, hk, d)),) * 2
    counts = [4, 3, 2, 4, 1, 3]
    q = randn(rng, sum(counts), heads, d, dtype=dtype)
    lse = torch.empty(sum(counts), heads, device=DEV)
    out = W.kv_attention(cache, q.to(DEV), starts(counts), ints(lens), ints(table), max_q_len=mq, max_kv_len=most,
                         scale=0.1, causal=causal, window=window, lse=lse)
    cut = np.cumsum([0] + counts)
    check(out, lse, [host64(q)[a:b] for a, b in zip(cut[:-1], cut[1:])], kvs + [none] * 4, 0.1, dtype, int4, sg, causal,
          window, hk)


def test_more_threads_than_one_launch_takes(W):
    """2^29 and more rows of 8 lanes: several launches, all of them there."""
    n, hk, d = (1 << 26) + 3, 4, 128
    cache = W.kv_cache_alloc(1, 16, hk, d, device=DEV)
    k, v = (torch.randn(1, hk, d, device=DEV).bfloat16() for _ in range(2))
    slots = torch.full((n,), -1, dtype=torch.int64, device=DEV)
    at = [0, (1 << 25) - 1, 1 << 25, n - 1]
    slots[at] = torch.arange(4, device=DEV)
    W.kv_append(cache, k.expand(n, hk, d), v.expand(n, hk, d), slots)
    for c, x in ((cache.k, k), (cache.v, v)):
        assert torch.equal(c[0, :, :4], x[0][:, None].expand(hk, 4, d)) and not c[0, :, 4:].any()
    cache = W.kv_cache_alloc(1, 16, 8, d, device=DEV)
    out = [torch.ones(1, 8, d, device=DEV).bfloat16().expand(n, 8, d) for _ in range(2)]
    slots.fill_(-1)
    W.kv_gather(cache, slots, k_out=out[0], v_out=out[1])
    assert not out[0][0].any() and not out[1][0].any()


@pytest.mark.parametrize("mq", [1, 4096])
def test_more_sequences_than_one_launch_takes(W, mq):
    """2^21 sequences on 8 key heads, nearly all of them empty: more blocks than one launch has threads for, of the
    kernel that joins the split keys of a step and of the chunk kernel."""
    rng = np.random.default_rng(71)
    seqs, hk, d, page = (1 << 21) + 5, 8, 64, 2048
    where, lens = [0, 7, 1 << 20, seqs - 1], [2000, 3, 900, 1500]
    cache, _ = new_cache(W, rng, 5, page, hk, d, torch.bfloat16, False)
    small, _, kvs = fill(W, rng, cache, None, lens, hk, d, torch.bfloat16, False, page)
    count = np.zeros(seqs, np.int64)
    count[where] = 1
    kv = np.zeros(seqs, np.int32)
    kv[where] = lens
    table = np.zeros((seqs, 1), np.int32)
    table[where, 0] = small[:, 0]
    q = randn(rng, 4, hk, d, dtype=torch.bfloat16)
    lse = torch.empty(4, hk, device=DEV)
    out = W.kv_attention(cache, q.to(DEV), starts(count), ints(kv), ints(table), max_q_len=mq, max_kv_len=2000,
                         scale=0.125, lse=lse)
    check(out, lse, [host64(q)[i:i + 1] for i in range(4)], kvs, 0.125, torch.bfloat16, False, None, True, 0, hk)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("d,n,kv,window", [(64, 5, 50, 0), (128, 5, 700, 0), (64, 1, 700, 0), (128, 90, 150, 0),
                                           (64, 90, 600, 40)])
def test_rows_not_finite_in_int4_pages(W, bad, dtype, d, n, kv, window):
    """A key or value with one value that is not finite: what its entry stands for is NaN all over (the transform
    spreads it), for gather and for the queries that see it, and for nobody else."""
    rng = np.random.default_rng(41)
    hk, heads, page = 2, 4, 16
    cache, sg = new_cache(W, rng, -(-kv // page) + 2, page, hk, d, dtype, True)
    table, slots, _ = fill(W, rng, cache, sg, [kv], hk, d, dtype, True, page)
    slots = slots[0]
    q = randn(rng, n, heads, d, dtype=dtype)
    args = (starts([n]), ints([kv]), ints(table))

    def run(mq, most):
        lse = torch.empty(n, heads, device=DEV)
        out = W.kv_attention(cache, q.to(DEV), *args, max_q_len=mq, max_kv_len=most, scale=0.1, window=window, lse=lse)
        return host64(out), host64(lse)

    calls = [(n, kv), (4096, kv), (n, 0), (4096, 1 << 16)]
    clean = [run(*c) for c in calls]
    before = [host64(t) for t in W.kv_gather(cache, ints(slots, torch.int64), dtype=dtype)]
    j = kv - n // 2 - 1  # in the middle of the chunk (its last key where that is one token)
    rows = ints(slots[j:j + 1], torch.int64)
    for side in (0, 1):
        kept = [t.clone() for t in (cache.k, cache.v, cache.k_scales, cache.v_scales)]
        x = [t.to(dtype).to(DEV) for t in (randn(rng, 1, hk, d), randn(rng, 1, hk, d))]
        x[side][0, 1, d // 2 + 3] = bad
        W.kv_append(cache, x[0], x[1], rows)
        assert not torch.isfinite((cache.k_scales, cache.v_scales)[side][slots[j] // page, 1, slots[j] % page])
        got = host64(W.kv_gather(cache, ints(slots, torch.int64), dtype=dtype)[side])
        assert np.isnan(got[j, 1]).all() and np.isfinite(got[j, 0]).all()
        assert np.array_equal(np.delete(got, j, 0), np.delete(before[side], j, 0))
        # as it was, with the entry not finite: key head 0's row must not have changed either
        for new, old in zip((cache.k, cache.v, cache.k_scales, cache.v_scales), kept):
            new[slots[j] // page, 0, slots[j] % page] = old[slots[j] // page, 0, slots[j] % page]
            if new.data_ptr() not in ((cache.k, cache.v)[side].data_ptr(), (cache.k_scales, cache.v_scales)[side].data_ptr()):
                new.copy_(old)
        p = kv - n + np.arange(n)
        hit = np.zeros((n, heads), bool)
        hit[:, 2:] = ((p >= j) & ((p - window < j) | (window == 0)))[:, None]
        for c, (out0, lse0) in zip(calls, clean):
            out, lse = run(*c)
            assert not np.isfinite(out[hit]).any(), (side, c)
            # two results of the same sums, each good to 2 U of values of size about 1
            assert np.all(np.abs(out - out0)[~hit] <= 4 * U[dtype]), (side, c)
            if side == 0:
                assert np.isnan(lse[hit]).all()
            assert np.abs(lse - lse0)[~hit].max(initial=0) <= 2.0 ** -18
        for new, old in zip((cache.k, cache.v, cache.k_scales, cache.v_scales), kept):
            new.copy_(old)


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("most", [0, 1 << 16])
@pytest.mark.parametrize("n,mq", [(1, 1), (5, 5), (5, 4096)])
@pytest.mark.parametrize("dtype,size,scale", [(torch.bfloat16, 1e-37, 0.1), (torch.bfloat16, 1e-9, 0.0),
                                              (torch.bfloat16, 1e-20, 1e-20), (torch.bfloat16, 1e-20, 0.0),
                                              (torch.bfloat16, 2e-38, 1e-30), (torch.float16, 1e-7, 0.0),
                                              (torch.float16, 1e-7, 1e-38)])
def test_tiny_queries_give_the_mean(W, int4, n, mq, most, dtype, size, scale):
    """Scores that are all but 0: the mean of the values seen, lse the logarithm of their number."""
    rng = np.random.default_rng(31)
    d, hk, page, kv = 64, 1, 16, 700
    cache, sg = new_cache(W, rng, 46, page, hk, d, dtype, int4)
    table, _, kvs = fill(W, rng, cache, sg, [kv], hk, d, dtype, int4, page)
    q = (randn(rng, n, 2, d) * size).to(dtype)
    lse = torch.empty(n, 2, device=DEV)
    out = W.kv_attention(cache, q.to(DEV), starts([n]), ints([kv]), ints(table), max_q_len=mq, max_kv_len=most,
                         scale=scale, lse=lse)
    check(out, lse, [host64(q)], kvs, scale, dtype, int4, sg, True, 0, hk)


@pytest.mark.parametrize("most", [0, 1 << 16])
def test_zero_values_beside_large_ones_out_of_sight(W, most):
    """The first tile in the window holds values of 0 and, before the window, large ones; the weight lies on keys of the
    same wave whose values are the least that INT4 scales hold.  What is out of sight leaves their bits alone."""
    rng = np.random.default_rng(61)
    d, page, kv, window, dtype = 64, 64, 1280, 1034, torch.bfloat16
    cache, sg = new_cache(W, rng, 20, page, 1, d, dtype, True)
    j = np.arange(kv)
    # tiles of 64 keys; the window begins inside tile 3; the weight is on the wave's next ones
    heavy = np.isin(j // 64, [7, 11, 15, 19])
    q = randn(rng, 1, 4, d, dtype=dtype)
    k = randn(rng, kv, 1, d)
    k[~heavy] -= 8.0 * q[0].sum(0)
    v = randn(rng, kv, 1, d) * 2.0 ** -21
    v[j < kv - window] = 1e4
    v[(j >= kv - window) & (j < 256)] = 0.0
    W.kv_append(cache, k.to(dtype).to(DEV), v.to(dtype).to(DEV), torch.arange(kv, device=DEV))
    kvs = [stored(cache, sg, j, d)]
    lse = torch.empty(1, 4, device=DEV)
    out = W.kv_attention(cache, q.to(DEV), starts([1]), ints([kv]), ints(np.arange(20)[None]), max_q_len=1,
                         max_kv_len=most, scale=0.125, window=window, lse=lse)
    # relative to the output: 2^-8 for its rounding and 2^-11 for the probabilities' (keys of one size, so their errors
    # add up as their values do), 2^-11 |q| |k| / 8 = 0.004 for the rotated query's; together below 0.01, held to 0.03
    want = check_rel(host64(q), kvs[0], 0.125, kv - window)
    err = np.linalg.norm(host64(out)[0] - want, axis=-1) / np.linalg.norm(want, axis=-1)
    assert err.max() <= 0.03, err


def check_rel(q, kv, scale, first):
    k, v = (t[first:, 0] for t in kv)
    s = scale * (q[0] @ k.T)
    p = np.exp(s - s.max(-1, keepdims=True))
    return (p @ v) / p.sum(-1, keepdims=True)


@pytest.mark.parametrize("mq", [1, 4096])
@pytest.mark.parametrize("dtype,int4", [(torch.float16, False), (torch.float16, True), (torch.bfloat16, True),
                                        (torch.bfloat16, False)])
def test_many_tiny_probabilities(W, dtype, int4, mq):
    """Eight keys (one in the first tile of each wave) with value 0 take nearly all the weight; 131064 others, 2^-25.1
    of theirs each, make the whole result.  A probability has a rounding of u and, in fp16, an absolute one of 2^-25
    beside a largest one that may stand at 2^8.  A lane adds up to half the keys to its fp32 sum."""
    rng = np.random.default_rng(51)
    d, page, kv, lead = 64, 65536, 131072, 64 * np.arange(8)
    cache, sg = new_cache(W, rng, 2, page, 1, d, dtype, int4)
    k, v = torch.zeros(kv, 1, d), torch.ones(kv, 1, d)
    k[lead], v[lead] = 1.0, 0.0
    W.kv_append(cache, k.to(dtype).to(DEV), v.to(dtype).to(DEV), torch.arange(kv, device=DEV))
    k64, v64 = stored(cache, sg, np.arange(kv), d) if int4 else (k.double().numpy(), v.double().numpy())
    gap = float(np.float32(25.1 * math.log(2) / k64[0].sum()))
    q = torch.ones(1, 1, d, dtype=dtype)
    lse = torch.empty(1, 1, device=DEV)
    out = W.kv_attention(cache, q.to(DEV), starts([1]), ints([kv]), ints([[0, 1]]), max_q_len=mq, max_kv_len=64,
                         scale=gap, lse=lse)
    s = gap * k64[:, 0].sum(-1)
    w = np.exp(s - s.max())
    want = (w @ v64[:, 0]) / w.sum()
    um = 2.0 ** -11 if int4 else U[dtype]
    # scores: fp32 sums of d products and the scale's product with log2(e), the rotated query's fp16 rounding
    ds = (E32 * (d + 8) + (2.0 ** -11 if int4 else 0.0)) * s.max()
    sums = kv / 2 * E32
    rel = np.expm1(2 * ds) + um + sums + U[dtype]
    tiny = 0.0 if dtype == torch.bfloat16 and not int4 else kv * 2.0 ** -25 * 2.0 ** -8 / w.sum() * 1.25
    assert np.all(np.abs(host64(out)[0, 0] - want) <= rel * np.abs(want).max() + tiny)
    assert abs(float(lse) - (s.max() + math.log(w.sum()))) <= ds + sums


def test_a_window_beyond_all_keys_plans_like_none(W):
    cache = W.kv_cache_alloc(2, 16, 1, 64, device=DEV)
    for n in (1, 64):
        want = W.kv_attention_workspace_bytes(cache, n, 8, 1, n, 8000)
        assert want > 0
        for window in (8000, 1 << 40, 2 ** 63 - 1):
            assert W.kv_attention_workspace_bytes(cache, n, 8, 1, n, 8000, window) == want
