"""Paged key/value cache on the GPU (kv_append, kv_gather, kv_attention)
against oracle/kv.py and oracle/rtn.py in fp64."""
import math

import numpy as np
import pytest
import torch

from oracle import hadamard as H, kv as K, rtn
from tests.gpu_util import DEV, host64, mask_dev

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # unit roundoff
E32 = 2.0 ** -24
DTS = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def W():
    from wht_adapters_amd import whtq
    return whtq


def randn(rng, *shape, dtype=torch.float32, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(dtype)


def tables(top, rot):
    ang = np.arange(top)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return torch.from_numpy(np.cos(ang).astype(np.float32)), torch.from_numpy(np.sin(ang).astype(np.float32))


def sign_words(rng, d):
    return rng.integers(0, 2 ** 32, d // 32, dtype=np.uint32)


def new_cache(W, rng, pages, page, hk, d, dtype, int4, layout="head"):
    """A cache full of NaN (16-bit) or stale codes: nothing may leak from it."""
    if int4:
        signs = sign_words(rng, d)
        c = W.kv_cache_alloc(pages, page, hk, d, int4=True, signs=mask_dev(signs), device=DEV)
        for t in (c.k, c.v):
            t.copy_(torch.from_numpy(rng.integers(0, 256, t.shape, dtype=np.uint8)))
        c.k_scales.fill_(float("nan"))
        c.v_scales.fill_(float("inf"))
        return c, H.signs_from_bits(signs, d)
    shape = (pages, hk, page, d) if layout == "head" else (pages, page, hk, d)
    k, v = (torch.full(shape, float("nan"), dtype=dtype, device=DEV) for _ in range(2))
    if layout != "head":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    return W.KVCache(k, v), None


# ------------------------------------------------------------------ append, gather

@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("d,rot,inter", [(128, 128, False), (128, 128, True), (64, 64, False), (64, 32, False),
                                         (128, 48, True), (128, 96, False), (64, 16, True)])
@pytest.mark.parametrize("layout", ["head", "token"])
def test_append_dense(W, dtype, d, rot, inter, layout):
    rng = np.random.default_rng(d + rot + inter)
    n, hk, hq, page, pages = 37, 3, 5, 16, 4
    cache, _ = new_cache(W, rng, pages, page, hk, d, dtype, False, layout)
    # rows inside wider storage: odd strides that keep 16-byte alignment
    k = randn(rng, n, hk + 1, d + 8, dtype=dtype, scale=3)[:, :hk, :d]
    v = randn(rng, n, hk, d, dtype=dtype)
    q = randn(rng, n, hq, d, dtype=dtype)
    cos, sin = tables(500, rot)
    pos = rng.integers(0, 500, n).astype(np.int32)
    slots = rng.permutation(pages * page)[:n].astype(np.int64)
    slots[[3, 5, 7]] = -1, pages * page, 2 ** 40
    pos[[9, 11]] = -1, 500
    kd = torch.empty(n, hk + 1, d + 8, dtype=dtype, device=DEV)[:, :hk, :d]
    kd.copy_(k)
    qd = q.to(DEV)
    sentinel = torch.full((n, hq, d), 7.0, dtype=dtype, device=DEV)
    got_q = W.kv_append(cache, kd, v.to(DEV), torch.from_numpy(slots).to(DEV), q=qd, cos=cos.to(DEV), sin=sin.to(DEV),
                        positions=torch.from_numpy(pos).to(DEV), interleaved=inter, q_out=sentinel)
    c64, s64 = cos.double().numpy(), sin.double().numpy()
    gone = {9, 11}
    ck, cv, gq = host64(cache.k), host64(cache.v), host64(got_q)
    written = np.zeros((pages, page), bool)
    for t in range(n):
        if t in gone:
            assert (gq[t] == 7.0).all()
            continue
        cs, sn = c64[pos[t]], s64[pos[t]]
        for x, y in ((host64(q)[t], gq[t]),) + (() if not 0 <= slots[t] < pages * page else (
                (host64(k)[t], ck[slots[t] // page, :, slots[t] % page]),)):
            want = K.rotate(x, cs, sn, inter)
            # two products and a sum in fp32 (three roundings of at most |a| + |b|), one rounding to the type
            size = np.abs(x).max() * 2
            assert np.all(np.abs(y - want) <= U[dtype] * np.abs(want) + (3 * E32) * size + 2.0 ** -25)
        if 0 <= slots[t] < pages * page:
            p, o = divmod(int(slots[t]), page)
            written[p, o] = True
            assert np.array_equal(cv[p, :, o], host64(v)[t])
    left = ~written
    assert np.isnan(ck.transpose(0, 2, 1, 3)[left]).all() and np.isnan(cv.transpose(0, 2, 1, 3)[left]).all()
    # read back, slots outside the cache included
    gk, gv = W.kv_gather(cache, torch.from_numpy(slots).to(DEV))
    for t in range(n):
        if not 0 <= slots[t] < pages * page:
            assert (host64(gk)[t] == 0).all() and (host64(gv)[t] == 0).all()
        elif t not in gone:
            p, o = divmod(int(slots[t]), page)
            assert np.array_equal(host64(gk)[t], ck[p, :, o]) and np.array_equal(host64(gv)[t], cv[p, :, o])


def test_append_in_place_and_without_rotation(W):
    rng = np.random.default_rng(3)
    cache, _ = new_cache(W, rng, 2, 16, 2, 64, torch.bfloat16, False)
    k, v, q = (randn(rng, 5, h, 64, dtype=torch.bfloat16).to(DEV) for h in (2, 2, 4))
    slots = torch.arange(5, dtype=torch.int64, device=DEV)
    cos, sin = (t.to(DEV) for t in tables(64, 32))
    pos = torch.arange(5, dtype=torch.int32, device=DEV)
    want = W.kv_append(cache, k, v, slots, q=q, cos=cos, sin=sin, positions=pos)
    q2 = q.clone()
    assert W.kv_append(cache, k, v, slots, q=q2, q_out=q2, cos=cos, sin=sin, positions=pos) is q2
    assert torch.equal(q2, want)
    assert torch.equal(W.kv_append(cache, k, v, slots, q=q), q)
    assert W.kv_append(cache, k, v, slots) is None
    gk, gv = W.kv_gather(cache, slots)
    assert torch.equal(gk, k) and torch.equal(gv, v)
    for n in (0,):
        W.kv_append(cache, k[:n], v[:n], slots[:n])
        assert W.kv_gather(cache, slots[:n])[0].shape == (0, 2, 64)


@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("signed", [True, False])
def test_append_int4(W, dtype, d, signed):
    rng = np.random.default_rng(11 + d)
    n, hk, page, pages = 41, 3, 32, 2
    words = sign_words(rng, d)
    cache = W.kv_cache_alloc(pages, page, hk, d, int4=True, signs=mask_dev(words) if signed else None, device=DEV)
    sg = H.signs_from_bits(words, d) if signed else np.ones(d)
    k = randn(rng, n, hk, d, dtype=dtype, scale=2.0)
    k[4] *= 100.0           # large, tiny and zero rows; an outlier channel
    k[5] *= 1e-4
    k[6] = 0
    k[7, :, 3] = 300.0
    v = randn(rng, n, hk, d, dtype=dtype)
    cos, sin = tables(300, d)
    pos = rng.integers(0, 300, n).astype(np.int32)
    slots = rng.permutation(pages * page)[:n].astype(np.int64)
    q = randn(rng, n, 6, d, dtype=dtype).to(DEV)
    W.kv_append(cache, k.to(DEV), v.to(DEV), torch.from_numpy(slots).to(DEV), q=q, cos=cos.to(DEV), sin=sin.to(DEV),
                positions=torch.from_numpy(pos).to(DEV))
    rot = np.stack([K.rotate(host64(k)[t], cos.double().numpy()[pos[t]], sin.double().numpy()[pos[t]]) for t in range(n)])
    for codes, scales, x in ((cache.k, cache.k_scales, rot), (cache.v, cache.v_scales, host64(v))):
        y = H.rht(x.reshape(-1, d), sg)
        # fp32 error of a transformed value: 3 roundings of the rotation, log2 d additions and 1 product, each at
        # most E32 of a partial sum of |x|, over sqrt(d)
        dy = (3 + math.log2(d) + 2) * E32 * np.abs(x.reshape(-1, d)).sum(-1) * 2 / math.sqrt(d)
        got = rtn.unpack_codes(codes.cpu().numpy()[slots // page, :, slots % page].reshape(-1, d // 2), 4, d)
        s = scales.cpu().numpy()[slots // page, :, slots % page].reshape(-1).astype(np.float64)
        top = np.abs(y).max(-1) / 7
        # half an ulp of fp16 (2^-11 relative, 2^-25 among subnormals) and the error of the maximum
        assert np.all(np.abs(s - top) <= np.maximum(2.0 ** -11 * top, 2.0 ** -25) + dy / 7 + E32 * top)
        with np.errstate(divide="ignore", invalid="ignore"):
            val = np.where(s[:, None] > 0, y / s[:, None], 0.0)
            slack = np.where(s > 0, dy / s, 0.0)[:, None] + 4 * E32 * np.abs(val)
        # the code is a nearest whole number, but for values within the error of a tie
        assert np.all(np.abs(np.clip(val, -7, 7) - got) <= 0.5 + slack)
    # what the cache stands for, by the library's own inverse and by gather
    for codes, scales, out in zip((cache.k, cache.v), (cache.k_scales, cache.v_scales),
                                  W.kv_gather(cache, torch.from_numpy(slots).to(DEV), dtype=dtype)):
        c = codes.cpu().numpy()[slots // page, :, slots % page].reshape(-1, d // 2)
        s = scales.cpu().numpy()[slots // page, :, slots % page].reshape(-1, 1)
        want = rtn.dequantize_inverse(c, s, sg, 4, d, d).reshape(n, hk, d)
        size = np.abs(rtn.unpack_codes(c, 4, d) * s.astype(np.float64)).sum(-1).reshape(n, hk, 1) / math.sqrt(d)
        err = (math.log2(d) + 2) * E32 * size
        assert np.all(np.abs(host64(out) - want) <= U[dtype] * np.abs(want) + err + 2.0 ** -25)
        lib = W.rht_dequantize_inverse(torch.from_numpy(c).to(DEV), torch.from_numpy(s.copy()).to(DEV),
                                       mask_dev(words) if signed else None, 4, d, d, out_dtype=torch.float32)
        assert np.all(np.abs(host64(lib).reshape(n, hk, d) - host64(out)) <= U[dtype] * np.abs(want) + 2 * err + 2.0 ** -25)


# ------------------------------------------------------------------ attention

def fill(W, rng, cache, sg, kls, hk, d, dtype, int4, page, scale_k=1.0):
    """Random keys / values for sequences of kls keys through kv_append; returns the
    table, and per sequence what the cache stands for (fp64)."""
    width = max(1, -(-max(kls) // page)) + 1
    pages = cache.k.shape[0]
    order = rng.permutation(pages).astype(np.int32)
    table = rng.choice(np.array([-1, 2 ** 30, pages], np.int32), (len(kls), width))  # unused entries: outside the cache
    at, slots = 0, []
    for b, n in enumerate(kls):
        m = -(-n // page)
        table[b, :m] = order[at:at + m]
        at += m
        j = np.arange(n)
        slots.append(table[b, j // page].astype(np.int64) * page + j % page)
    assert at <= pages
    alls = np.concatenate(slots) if slots else np.zeros(0, np.int64)
    k = randn(rng, len(alls), hk, d, dtype=dtype, scale=scale_k)
    v = randn(rng, len(alls), hk, d, dtype=dtype)
    W.kv_append(cache, k.to(DEV), v.to(DEV), torch.from_numpy(alls).to(DEV))
    if int4:
        side = []
        for codes, scales in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
            c = codes.cpu().numpy()[alls // page, :, alls % page].reshape(-1, d // 2)
            s = scales.cpu().numpy()[alls // page, :, alls % page].reshape(-1, 1)
            side.append(rtn.dequantize_inverse(c, s, sg, 4, d, d).reshape(len(alls), hk, d))
        k64, v64 = side
    else:
        k64, v64 = host64(k), host64(v)
    cut = np.cumsum([0] + [len(s) for s in slots])
    return table, slots, [(k64[a:b], v64[a:b]) for a, b in zip(cut[:-1], cut[1:])]


def check(out, lse, qs, kvs, scale, dtype, int4, sg, causal, window, hk):
    """Row 2-norm bound.  With u the roundoff of the products' type: the score of key j is off by at most
    ds_j = E32 (D + 4) scale sum|q k| (INT4: + 2^-11 scale sum|q' k'| for the rotated query's fp16 rounding, u its
    type), a probability by the relative 2 ds + u + 2^-20 (exp2, sums), so the mean by that of the mean of |v|; then
    one rounding of the result.  fp16 probabilities below 2^-14 lose up to 2^-25 each (INT4: of the largest scale's
    values)."""
    at = 0
    for q, (k, v) in zip(qs, kvs):
        n, heads, d = q.shape
        want, wl = K.attention(q, k, v, scale, causal, window)
        got, gl = host64(out[at:at + n]), host64(lse[at:at + n])
        um = 2.0 ** -11 if int4 else U[dtype]
        for i in range(n):
            js = [j for j in range(len(k)) if K.sees(len(k), n, i, j, causal, window)]
            for h in range(heads):
                if not js:
                    assert (got[i, h] == 0).all() and gl[i, h] == -np.inf
                    continue
                g = h // (heads // hk)
                kk, vv, qq = k[js, g], v[js, g], q[i, h]
                if int4:
                    kk, vv, qq = H.rht(kk, sg), H.rht(vv, sg), H.rht(qq[None], sg)[0]
                size = scale * (np.abs(kk) @ np.abs(qq))
                ds = (E32 * (d + 4) * size + (2.0 ** -11 * size if int4 else 0) + 4 * E32 * np.abs(size)).max()
                p = np.exp(scale * (kk @ qq) - wl[i, h])
                rel = np.expm1(2 * ds) + um + 2.0 ** -20
                mean = np.linalg.norm(p @ np.abs(vv)) * rel
                tiny = 0.0 if (dtype == torch.bfloat16 and not int4) else \
                    len(js) * 2.0 ** -25 * np.linalg.norm(np.abs(vv).max(0)) * min(1.0, p.max())
                bound = mean + tiny + U[dtype] * np.linalg.norm(want[i, h]) + 2.0 ** -24 * math.sqrt(d)
                err = np.linalg.norm(got[i, h] - want[i, h])
                assert err <= bound, (at, i, h, err, bound)
                assert abs(gl[i, h] - wl[i, h]) <= ds + 2.0 ** -20 + 4 * E32 * abs(wl[i, h]), (i, h, gl[i, h], wl[i, h])
        at += n


CASES = [
    # heads, kv heads, dim, page, (new, keys) of each sequence, causal, window
    (4, 2, 128, 16, [(1, 1)], True, 0),
    (4, 4, 64, 16, [(1, 33), (1, 0), (1, 64), (1, 1)], True, 0),
    (8, 1, 128, 32, [(1, 257), (1, 31), (1, 129)], True, 0),
    (6, 2, 64, 64, [(1, 300)], False, 0),
    (16, 1, 64, 16, [(1, 95)], True, 17),
    (17, 1, 128, 16, [(1, 70), (1, 300)], True, 0),          # 17 rows: two column blocks
    (40, 1, 64, 16, [(1, 70)], True, 0),                     # more rows than the step kernel takes
    (4, 2, 128, 16, [(3, 5), (0, 9), (4, 2), (2, 40)], True, 0),   # a chunk longer than its keys: rows that see nothing
    (8, 2, 64, 16, [(5, 100), (1, 7)], True, 6),
    (6, 2, 128, 32, [(7, 80)], False, 0),
    (4, 2, 128, 16, [(70, 70), (3, 200), (33, 34)], True, 0),
    (2, 2, 64, 64, [(130, 190)], True, 0),
    (3, 1, 128, 16, [(90, 333)], True, 50),
    (5, 5, 64, 16, [(65, 64), (40, 0)], True, 0),
    (8, 2, 128, 128, [(64, 129)], False, 31),
    (14, 2, 64, 32, [(20, 500), (1, 3), (75, 76)], True, 64),
]


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(W, case, dtype, int4):
    heads, hk, d, page, seqs, causal, window = CASES[case]
    rng = np.random.default_rng(100 + case)
    kls = [b for _, b in seqs]
    pages = sum(-(-n // page) for n in kls) + 3
    layout = "token" if case % 2 else "head"
    cache, sg = new_cache(W, rng, pages, page, hk, d, dtype, int4, layout)
    table, _, kvs = fill(W, rng, cache, sg, kls, hk, d, dtype, int4, page, 1.5)
    n = sum(a for a, _ in seqs)
    q = randn(rng, n, heads + 1, d + 8, dtype=dtype, scale=1.5)[:, :heads, :d]
    qd = torch.empty(n, heads + 1, d + 8, dtype=dtype, device=DEV)[:, :heads, :d]
    qd.copy_(q)
    qst = np.cumsum([0] + [a for a, _ in seqs]).astype(np.int32)
    scale = 0.7 / math.sqrt(d) * 1.3
    lse = torch.full((n, heads), 9.0, device=DEV)
    out = torch.full((n, heads, d + 16), 9.0, dtype=dtype, device=DEV)[:, :, :d]
    args = (torch.from_numpy(qst).to(DEV), torch.tensor(kls, dtype=torch.int32, device=DEV),
            torch.from_numpy(table).to(DEV))
    kw = dict(max_q_len=max(a for a, _ in seqs), max_kv_len=max(kls), scale=scale, causal=causal, window=window)
    W.kv_attention(cache, qd, *args, out=out, lse=lse, **kw)
    qs = [host64(q)[a:b] for a, b in zip(qst[:-1], qst[1:])]
    check(out, lse, qs, kvs, scale, dtype, int4, sg, causal, window, hk)
    # a bound on the keys that splits them, and one that is far too small, give the same within the same bound
    for most in (1 << 16, 0):
        o2 = W.kv_attention(cache, qd, *args, lse=lse, **dict(kw, max_kv_len=most))
        check(o2, lse, qs, kvs, scale, dtype, int4, sg, causal, window, hk)
    # the chunk kernel on the same rows
    o3 = W.kv_attention(cache, qd, *args, lse=lse, **dict(kw, max_q_len=4096))
    check(o3, lse, qs, kvs, scale, dtype, int4, sg, causal, window, hk)


LONG = [
    (4, 2, 128, 32, [(260, 1400), (1, 900), (70, 70)], True, 0),
    (3, 1, 64, 64, [(130, 1100)], False, 0),
    (4, 1, 128, 16, [(200, 1000)], True, 300),
    (2, 1, 64, 16, [(300, 700), (33, 640)], True, 0),
]


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("case", range(len(LONG)))
def test_attention_long(W, case, dtype, int4):
    """Many whole tiles between the masked ones, with and without a split of the keys."""
    heads, hk, d, page, seqs, causal, window = LONG[case]
    rng = np.random.default_rng(200 + case)
    kls = [b for _, b in seqs]
    cache, sg = new_cache(W, rng, sum(-(-n // page) for n in kls) + 3, page, hk, d, dtype, int4)
    table, _, kvs = fill(W, rng, cache, sg, kls, hk, d, dtype, int4, page, 1.5)
    n = sum(a for a, _ in seqs)
    q = randn(rng, n, heads, d, dtype=dtype, scale=1.5)
    qst = np.cumsum([0] + [a for a, _ in seqs]).astype(np.int32)
    args = (torch.from_numpy(qst).to(DEV), torch.tensor(kls, dtype=torch.int32, device=DEV),
            torch.from_numpy(table).to(DEV))
    qs = [host64(q)[a:b] for a, b in zip(qst[:-1], qst[1:])]
    lse = torch.full((n, heads), 9.0, device=DEV)
    for most in (64, max(kls)):
        out = W.kv_attention(cache, q.to(DEV), *args, lse=lse, max_q_len=max(a for a, _ in seqs), max_kv_len=most,
                             scale=-0.1, causal=causal, window=window)
        check(out, lse, [-x for x in qs], kvs, 0.1, dtype, int4, sg, causal, window, hk)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,hk", [(1, 4), (5, 2), (40, 1), (150, 4)])
def test_int4_fp16_keeps_the_precision_of_its_outputs(W, d, n, hk):
    """Scores of deviation 3: rounding the rotated query to fp16 alone would leave an error of 3 2^-11 / sqrt(3) and more
    in the probabilities.  What may stay is one rounding of each probability's product with its value scale and one of
    the result, each at most 2^-10 / sqrt(12) of its value in the root mean square, independent of each other; 10 % for
    the sample (about 2000 values or more), and fp32 sums far below."""
    rng = np.random.default_rng(17 + d + n)
    heads, page, kls = 8, 16, [700, 331]
    cache, sg = new_cache(W, rng, sum(-(-m // page) for m in kls) + 3, page, hk, d, torch.float16, True)
    table, _, kvs = fill(W, rng, cache, sg, kls, hk, d, torch.float16, True, page)
    q = randn(rng, 2 * n, heads, d, dtype=torch.float16, scale=3.0)
    args = (torch.tensor([0, n, 2 * n], dtype=torch.int32, device=DEV), torch.tensor(kls, dtype=torch.int32, device=DEV),
            torch.from_numpy(table).to(DEV))
    lse = torch.empty(2 * n, heads, device=DEV)
    got = host64(W.kv_attention(cache, q.to(DEV), *args, lse=lse, max_q_len=n, max_kv_len=max(kls), scale=d ** -0.5))
    pairs = [K.attention(host64(q)[b * n:b * n + n], k, v, d ** -0.5, True, 0) for b, (k, v) in enumerate(kvs)]
    want, wl = (np.concatenate([p[i] for p in pairs]) for i in (0, 1))
    assert np.linalg.norm(got - want) <= 1.1 * math.sqrt(2) * 2.0 ** -10 / math.sqrt(12) * np.linalg.norm(want)
    # sums of d products in fp32, the two parts of the query good to 2^-22 of its largest value
    size = d ** -0.5 * 3 * 4.5 * d
    assert np.abs(host64(lse) - wl).max() <= (E32 * (d + 4) + 2.0 ** -22) * size + 2.0 ** -20 + 4 * E32 * np.abs(wl).max()


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("d,n,kv,window", [(64, 5, 50, 0), (128, 5, 50, 0), (128, 90, 150, 0), (64, 90, 150, 40), (128, 6, 200, 9)])
def test_values_not_finite_reach_only_who_sees_them(W, bad, dtype, d, n, kv, window):
    rng = np.random.default_rng(5)
    hk, heads, page = 2, 4, 16
    cache, _ = new_cache(W, rng, 14, page, hk, d, dtype, False)
    table, slots, kvs = fill(W, rng, cache, None, [kv], hk, d, dtype, False, page)
    k64, v64 = kvs[0]
    # the last key's value, one in the middle of the chunk, and one that a window drops
    for j in (kv - 1, kv - n // 2) + ((kv - n - 3,) if window else ()):
        s = slots[0][j]
        cache.v[s // page, 1, s % page, d // 2 + 1] = bad
        v64[j, 1, d // 2 + 1] = bad
    q = randn(rng, n, heads, d, dtype=dtype)
    lse = torch.empty(n, heads, device=DEV)
    with np.errstate(invalid="ignore"):
        want, _ = K.attention(host64(q), k64, v64, 0.1, True, window)
    for mq in (n, 4096):
        out = host64(W.kv_attention(cache, q.to(DEV), torch.tensor([0, n], dtype=torch.int32, device=DEV),
                                    torch.tensor([kv], dtype=torch.int32, device=DEV), torch.from_numpy(table).to(DEV),
                                    max_q_len=mq, max_kv_len=kv, scale=0.1, window=window, lse=lse))
        assert np.array_equal(np.isnan(want), np.isnan(out))
        assert np.array_equal(np.isinf(want), np.isinf(out))
        fine = np.isfinite(want)
        assert np.all(np.abs(out - np.where(fine, want, 0))[fine] <= 4 * U[dtype])  # means of values of size about 1


def test_scores_not_finite(W):
    """A key of +inf / NaN makes the rows that see it NaN and no other; -inf scores drop out."""
    rng = np.random.default_rng(6)
    cache, _ = new_cache(W, rng, 4, 16, 1, 64, torch.float16, False)
    table, slots, kvs = fill(W, rng, cache, None, [40], 1, 64, torch.float16, False, 16)
    s = slots[0][38]
    cache.k[s // 16, 0, s % 16, 5] = float("nan")
    q = randn(rng, 4, 2, 64, dtype=torch.float16)
    out = host64(W.kv_attention(cache, q.to(DEV), torch.tensor([0, 4], dtype=torch.int32, device=DEV),
                                torch.tensor([40], dtype=torch.int32, device=DEV), torch.from_numpy(table).to(DEV),
                                max_q_len=4, max_kv_len=40))
    assert np.isnan(out[2:]).all() and np.isfinite(out[:2]).all()


@pytest.mark.parametrize("int4", [False, True])
def test_extreme_scores_and_scales(W, int4):
    """Scores that grow along the keys (the maximum keeps moving) and values of very different size."""
    rng = np.random.default_rng(8)
    d, hk, page, kv = 64, 1, 16, 400
    cache, sg = new_cache(W, rng, 26, page, hk, d, torch.float16, int4)
    table, slots, kvs = fill(W, rng, cache, sg, [kv], hk, d, torch.float16, int4, page)
    q = randn(rng, 3, 2, d, dtype=torch.float16, scale=8.0)
    base = randn(rng, kv, hk, d, dtype=torch.float16) * 0.2 + torch.linspace(-4, 4, kv)[:, None, None] * q[0, 0].sign()
    v = randn(rng, kv, hk, d) * torch.exp(torch.linspace(-9, 6, kv))[:, None, None]
    k, v = base.half(), v.half()
    W.kv_append(cache, k.to(DEV), v.to(DEV), torch.from_numpy(slots[0]).to(DEV))
    if int4:
        gk = []
        for codes, scales in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
            c = codes.cpu().numpy()[slots[0] // page, :, slots[0] % page].reshape(-1, d // 2)
            s = scales.cpu().numpy()[slots[0] // page, :, slots[0] % page].reshape(-1, 1)
            gk.append(rtn.dequantize_inverse(c, s, sg, 4, d, d).reshape(kv, hk, d))
    else:
        gk = [host64(k), host64(v)]
    for mq in (3, 4096):
        lse = torch.empty(3, 2, device=DEV)
        out = W.kv_attention(cache, q.to(DEV), torch.tensor([0, 3], dtype=torch.int32, device=DEV),
                             torch.tensor([kv], dtype=torch.int32, device=DEV), torch.from_numpy(table).to(DEV),
                             max_q_len=mq, max_kv_len=kv, lse=lse)
        check(out, lse, [host64(q)], [tuple(gk)], d ** -0.5, torch.float16, int4, sg, True, 0, hk)


def test_cache_beyond_4_gib(W):
    """Pages whose offsets pass 2^32 bytes and 2^31 elements."""
    rng = np.random.default_rng(9)
    d, hk, page, pages = 128, 8, 64, 44000
    k, v = (torch.empty(pages, hk, page, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    assert k.numel() * 2 > 5 * 2 ** 30
    cache = W.KVCache(k, v)
    kv, n = 150, 40
    table = np.array([[pages - 1, 5, pages - 2]], np.int32)
    j = np.arange(kv)
    slots = table[0, j // page].astype(np.int64) * page + j % page
    kk, vv = (randn(rng, kv, hk, d, dtype=torch.bfloat16) for _ in range(2))
    W.kv_append(cache, kk.to(DEV), vv.to(DEV), torch.from_numpy(slots).to(DEV))
    gk, gv = W.kv_gather(cache, torch.from_numpy(slots).to(DEV))
    assert torch.equal(gk.cpu(), kk) and torch.equal(gv.cpu(), vv)
    q = randn(rng, n, hk, d, dtype=torch.bfloat16)
    for take in (1, n):
        lse = torch.empty(take, hk, device=DEV)
        out = W.kv_attention(cache, q[:take].to(DEV), torch.tensor([0, take], dtype=torch.int32, device=DEV),
                             torch.tensor([kv], dtype=torch.int32, device=DEV), torch.from_numpy(table).to(DEV),
                             max_q_len=take, max_kv_len=kv, lse=lse)
        check(out, lse, [host64(q)[:take]], [(host64(kk), host64(vv))], d ** -0.5, torch.bfloat16, False, None, True, 0, hk)


@pytest.mark.parametrize("int4", [False, True])
def test_side_stream_graph_and_repeat(W, int4):
    """A decode step captured once and replayed with new lengths; the same bytes each time and on another stream."""
    rng = np.random.default_rng(10)
    d, hk, heads, page, b, most = 128, 2, 8, 16, 3, 2000
    cache, sg = new_cache(W, rng, 3 * 126, page, hk, d, torch.bfloat16, int4)
    table, slots, _ = fill(W, rng, cache, sg, [most] * b, hk, d, torch.bfloat16, int4, page)
    table = torch.from_numpy(table).to(DEV)
    q = randn(rng, b, heads, d, dtype=torch.bfloat16).to(DEV)
    knew, vnew = (randn(rng, b, hk, d, dtype=torch.bfloat16).to(DEV) for _ in range(2))
    qst = torch.arange(b + 1, dtype=torch.int32, device=DEV)
    lens = torch.tensor([1500, 77, 2000], dtype=torch.int32, device=DEV)
    slot = torch.zeros(b, dtype=torch.int64, device=DEV)
    cos, sin = (t.to(DEV) for t in tables(most, d))
    out, qr = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(max(16, W.kv_attention_workspace_bytes(cache, b, heads, b, 1, most)), dtype=torch.uint8, device=DEV)

    def step():
        W.kv_append(cache, knew, vnew, slot, q=q, q_out=qr, cos=cos, sin=sin, positions=lens - 1)
        W.kv_attention(cache, qr, qst, lens, table, max_q_len=1, max_kv_len=most, out=out, workspace=ws)

    pos = torch.empty_like(lens)

    def captured():
        W.kv_append(cache, knew, vnew, slot, q=q, q_out=qr, cos=cos, sin=sin, positions=pos)
        W.kv_attention(cache, qr, qst, lens, table, max_q_len=1, max_kv_len=most, out=out, workspace=ws)

    def setup(ls):
        lens.copy_(torch.tensor(ls, dtype=torch.int32))
        pos.copy_(lens - 1)
        slot.copy_(torch.tensor([int(slots[i][n - 1]) for i, n in enumerate(ls)]))

    setup([1500, 77, 2000])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        captured()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured()
    for ls in ([1500, 77, 2000], [1, 2, 3], [1999, 640, 16], [1500, 77, 2000]):
        setup(ls)
        step()
        torch.cuda.synchronize()
        want, wq = out.clone(), qr.clone()
        out.zero_()
        qr.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(qr, wq)
        with torch.cuda.stream(side):
            out.zero_()
            captured()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_refusals(W):
    bf = dict(dtype=torch.bfloat16, device=DEV)
    cache = W.kv_cache_alloc(2, 16, 2, 64, device=DEV)
    k = torch.zeros(3, 2, 64, **bf)
    slots = torch.zeros(3, dtype=torch.int64, device=DEV)
    for bad in (lambda: W.kv_append(cache, k[:, :1], k, slots), lambda: W.kv_append(cache, k, k, slots.int()),
                lambda: W.kv_append(cache, k.half(), k.half(), slots), lambda: W.kv_append(cache, k, k, slots[:2]),
                lambda: W.kv_append(cache, k, k, slots, cos=torch.zeros(4, 32, device=DEV)),
                lambda: W.kv_append(cache, k, k, slots, q_out=k), lambda: W.kv_append(cache, k.cpu(), k, slots),
                lambda: W.kv_gather(cache, slots, dtype=torch.float16),
                lambda: W.KVCache(cache.k, cache.v[:1]), lambda: W.KVCache(cache.k.float(), cache.v.float()),
                lambda: W.KVCache(cache.k, cache.v, signs=slots),
                lambda: W.KVCache(cache.k.view(torch.uint8), cache.v.view(torch.uint8))):
        with pytest.raises(ValueError):
            bad()
    q = torch.zeros(1, 4, 64, **bf)
    one = torch.ones(1, dtype=torch.int32, device=DEV)
    qst = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    tab = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    kw = dict(max_q_len=1, max_kv_len=1)
    for bad in (lambda: W.kv_attention(cache, q[:, :3], qst, one, tab, **kw),
                lambda: W.kv_attention(cache, q, qst[:1], one, tab, **kw),
                lambda: W.kv_attention(cache, q, qst, one.long(), tab, **kw),
                lambda: W.kv_attention(cache, q, qst, one, tab[0], **kw),
                lambda: W.kv_attention(cache, q, qst, one, tab, lse=torch.zeros(1, 4, 2, device=DEV), **kw)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(W.WhtqError) as e:  # the call's own workspace rule
        W.kv_attention(cache, q, qst, one, tab, max_q_len=1, max_kv_len=1 << 20,
                       workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == 1
    with pytest.raises(W.WhtqError) as e:  # rows that are not 16-byte aligned
        W.kv_append(cache, torch.zeros(3, 2, 65, **bf)[:, :, 1:], k, slots)
    assert e.value.status == 3
    with pytest.raises(W.WhtqError) as e:
        c = W.kv_cache_alloc(2, 16, 2, 96, device=DEV)
        W.kv_gather(c, slots)
    assert e.value.status == 2
    with pytest.raises(W.WhtqError) as e:
        c = W.kv_cache_alloc(2, 24, 2, 64, device=DEV)
        W.kv_gather(c, slots)
    assert e.value.status == 2
