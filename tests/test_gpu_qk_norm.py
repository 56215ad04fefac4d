"""Norms and positions of queries and keys on the GPU (kv_append with norms,
qk_norm_rope and its backward pass) against oracle/lm.py in fp64."""
import numpy as np
import pytest
import torch

from oracle import hadamard as H, kv as K, lm, rtn
from tests.gpu_util import DEV, host64, mask_dev

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # unit roundoff
TINY = 2.0 ** -25  # half of fp16's least step
E32 = 2.0 ** -24
DTS = [torch.bfloat16, torch.float16]
EPS = 1e-5


@pytest.fixture(scope="module")
def W():
    from wht_adapters_amd import whtq
    return whtq


def randn(rng, *shape, dtype=torch.float32, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(dtype)


def tables(top, rot):
    ang = np.arange(top)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return torch.from_numpy(np.cos(ang).astype(np.float32)), torch.from_numpy(np.sin(ang).astype(np.float32))


def weights(rng, heads, d, per_head, dtype):
    return randn(rng, *((heads, d) if per_head else (d,)), scale=0.3).add(1).to(dtype)


# r: 16 products of a lane and 3 sums over lanes (each relative to the sum of squares, halved by the root), the
# mean, eps, the root (2 units): below 14 units; two products; three roundings of a rotation of two such values
NORM = 14 + 2
TURN = 3


def norm_bound(x, w, dtype, want):
    size = np.abs(x * lm.rms(x, EPS) * w).max(-1, keepdims=True) * 2
    return U[dtype] * np.abs(want) + (NORM + TURN) * E32 * size + TINY


LAYOUTS = [(128, 128, False), (128, 128, True), (64, 64, False), (64, 32, False), (128, 48, True), (128, 96, False),
           (64, 0, False)]


@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("d,rot,inter", LAYOUTS)
@pytest.mark.parametrize("per_head,wdt", [(False, torch.float32), (True, None)])
def test_append(W, dtype, d, rot, inter, per_head, wdt):
    rng = np.random.default_rng(d + rot)
    n, hk, hq, page, pages = 37, 3, 5, 16, 4
    qkv = randn(rng, n, hq + 2 * hk, d, dtype=dtype, scale=3)  # one projection's output
    qkv[4] = 0
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    qn, kn = weights(rng, hq, d, per_head, wdt or dtype), weights(rng, hk, d, per_head, wdt or dtype)
    cache = W.KVCache(*(torch.full((pages, hk, page, d), float("nan"), dtype=dtype, device=DEV) for _ in range(2)))
    dev = qkv.to(DEV)
    qd, kd, vd = dev[:, :hq], dev[:, hq:hq + hk], dev[:, hq + hk:]
    slots = rng.permutation(pages * page)[:n].astype(np.int64)
    slots[[3, 5]] = -1, pages * page
    kw, c64, s64 = {}, None, None
    pos = rng.integers(0, 500, n).astype(np.int32)
    gone = []
    if rot:
        cos, sin = tables(500, rot)
        pos[[9, 11]] = -1, 500
        gone = [9, 11]
        kw = dict(cos=cos.to(DEV), sin=sin.to(DEV), positions=torch.from_numpy(pos).to(DEV), interleaved=inter)
        c64, s64 = cos.double().numpy()[pos % 500], sin.double().numpy()[pos % 500]
    out = torch.full((n, hq, d), 7.0, dtype=dtype, device=DEV)
    W.kv_append(cache, kd, vd, torch.from_numpy(slots).to(DEV), q=qd, q_out=out, q_norm=qn.to(DEV), k_norm=kn.to(DEV),
                norm_eps=EPS, **kw)
    assert torch.equal(dev.cpu(), qkv)
    keep = np.array([t not in gone for t in range(n)])
    wq = lm.norm_rope(host64(q), host64(qn), EPS, c64, s64, inter)
    wk = lm.norm_rope(host64(k), host64(kn), EPS, c64, s64, inter)
    got = host64(out)
    assert (got[~keep] == 7).all()
    assert np.all(np.abs(got - wq)[keep] <= norm_bound(host64(q), host64(qn), dtype, wq)[keep])
    ck, cv = (host64(t).transpose(0, 2, 1, 3).reshape(pages * page, hk, d) for t in (cache.k, cache.v))
    there = keep & (slots >= 0) & (slots < pages * page)
    at = slots[there]
    assert np.all(np.abs(ck[at] - wk[there]) <= norm_bound(host64(k), host64(kn), dtype, wk)[there])
    assert np.array_equal(cv[at], host64(v)[there])
    left = np.setdiff1d(np.arange(pages * page), at)
    assert np.isnan(ck[left]).all() and np.isnan(cv[left]).all()


@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("d", [64, 128])
def test_append_one_side(W, dtype, d):
    """Only keys, or only queries, normed; the other side as without norms, bit for bit; in place."""
    rng = np.random.default_rng(d)
    q, k, v = (randn(rng, 21, h, d, dtype=dtype).to(DEV) for h in (4, 2, 2))
    qn, kn = randn(rng, d).to(DEV), randn(rng, d).to(DEV)
    cos, sin = (t.to(DEV) for t in tables(64, d))
    slots = torch.arange(21, device=DEV)
    kw = dict(cos=cos, sin=sin, positions=torch.arange(21, dtype=torch.int32, device=DEV))

    def call(**more):
        c = W.kv_cache_alloc(2, 16, 2, d, dtype=dtype, device=DEV)
        return W.kv_append(c, k, v, slots, q=q.clone(), **kw, **more), c.k
    bare, both = call(), call(q_norm=qn, k_norm=kn)
    only_q, only_k = call(q_norm=qn), call(k_norm=kn)
    assert torch.equal(only_q[0], both[0]) and torch.equal(only_q[1], bare[1])
    assert torch.equal(only_k[0], bare[0]) and torch.equal(only_k[1], both[1])
    c = W.kv_cache_alloc(2, 16, 2, d, dtype=dtype, device=DEV)
    inplace = q.clone()
    assert W.kv_append(c, k, v, slots, q=inplace, q_out=inplace, q_norm=qn, k_norm=kn, **kw) is inplace
    assert torch.equal(inplace, both[0])
    W.kv_append(c, k, v, slots, k_norm=kn, **kw)
    assert torch.equal(c.k, both[1])


@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("d", [64, 128])
def test_append_int4(W, dtype, d):
    """The codes are those of the unrounded normed key: within the step of 1 / 2 and fp32's error of it."""
    rng = np.random.default_rng(3 + d)
    n, hk, page, pages = 41, 3, 32, 2
    words = rng.integers(0, 2 ** 32, d // 32, dtype=np.uint32)
    cache = W.kv_cache_alloc(pages, page, hk, d, int4=True, signs=mask_dev(words), device=DEV)
    sg = H.signs_from_bits(words, d)
    k, v = randn(rng, n, hk, d, dtype=dtype, scale=2.0), randn(rng, n, hk, d, dtype=dtype)
    kn = weights(rng, hk, d, False, dtype)
    cos, sin = tables(100, d)
    pos = rng.integers(0, 100, n).astype(np.int32)
    slots = torch.from_numpy(rng.permutation(pages * page)[:n].astype(np.int64)).to(DEV)
    W.kv_append(cache, k.to(DEV), v.to(DEV), slots, k_norm=kn.to(DEV), norm_eps=EPS, cos=cos.to(DEV), sin=sin.to(DEV),
                positions=torch.from_numpy(pos).to(DEV))
    gk, _ = W.kv_gather(cache, slots, dtype=torch.float16)
    want = lm.norm_rope(host64(k), host64(kn), EPS, cos.double().numpy()[pos], sin.double().numpy()[pos])
    y = H.rht(want.reshape(-1, d), sg).reshape(n, hk, d)
    scale = (np.abs(y).max(-1, keepdims=True) / 7).astype(np.float16).astype(np.float64)
    got = host64(gk)
    # in the transformed domain: half a step (the top of the range may lie a rounding of the scale beyond 7), another
    # scale's rounding of up to 8 codes, fp16's rounding of the gathered row spread over the transform
    err = np.abs(H.rht(got.reshape(-1, d), sg).reshape(n, hk, d) - y)
    assert np.all(err <= scale * (0.5 + 8 * 2 * 2.0 ** -11) + np.linalg.norm(got, axis=-1, keepdims=True) * 2.0 ** -11
                  + np.abs(want).max(-1, keepdims=True) * d ** 0.5 * 40 * E32)


@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("d,rot,inter", LAYOUTS)
@pytest.mark.parametrize("n,hq,hk,ph", [(1, 1, 1, False), (37, 5, 3, True), (300, 8, 2, False), (65, 7, 1, True)])
def test_dense_and_gradients(W, dtype, d, rot, inter, n, hq, hk, ph):
    rng = np.random.default_rng(n + d + rot)
    qkv = randn(rng, n, hq + hk + 1, d, dtype=dtype, scale=2).to(DEV)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    dqo, dko = (randn(rng, n, h, d + 8, dtype=dtype).to(DEV)[..., :d] for h in (hq, hk))
    qn, kn = weights(rng, hq, d, ph, torch.float32).to(DEV), weights(rng, hk, d, ph, torch.float32).to(DEV)
    kw, c64, s64 = dict(q_norm=qn, k_norm=kn, norm_eps=EPS), None, None
    if rot:
        cos, sin = tables(400, rot)
        pos = rng.integers(0, 400, n)
        kw.update(cos=cos.to(DEV), sin=sin.to(DEV), positions=torch.from_numpy(pos.astype(np.int32)).to(DEV), interleaved=inter)
        c64, s64 = cos.double().numpy()[pos], sin.double().numpy()[pos]
    outs = W.qk_norm_rope(q, k, **kw)
    grads = W.qk_norm_rope_backward(dqo, dko, q, k, **kw)
    for i, (x, w, dy) in enumerate(((q, qn, dqo), (k, kn, dko))):
        x, w, dy = host64(x), host64(w), host64(dy)
        want = lm.norm_rope(x, w, EPS, c64, s64, inter)
        assert np.all(np.abs(host64(outs[i]) - want) <= norm_bound(x, w, dtype, want))
        dx, dw = lm.norm_rope_backward(dy, x, w, EPS, c64, s64, inter)
        r = lm.rms(x, EPS)
        top = np.abs(dy).max(-1, keepdims=True) * 2 * np.abs(w).max()
        # u: turn and weight (4 units of its size); the mean: 19 sums; r thrice, products: below 80 units of both terms' sizes
        size = r * top + r ** 3 * np.abs(x) * np.mean(np.abs(x) * top, -1, keepdims=True)
        assert np.all(np.abs(host64(grads[i]) - dx) <= U[dtype] * np.abs(dx) + 80 * E32 * size + TINY)
        # a sum of n heads terms, each off by its turn, r and two products; no more additions in a row than terms and 40
        axis = 0 if ph else (0, 1)
        g = np.abs(dy).max(-1, keepdims=True) * 2
        mass = (g * np.abs(x) * r).sum(axis)
        terms = n * (1 if ph else x.shape[1])
        assert grads[2 + i].dtype is torch.float32 and grads[2 + i].shape == (qn, kn)[i].shape
        assert np.all(np.abs(host64(grads[2 + i]) - dw) <= (terms + 40 + NORM + TURN + 2) * E32 * mass)


def test_gradient_against_differences(W):
    """d loss / d x by differences of the fp64 oracle, at points of the kernel's own inputs."""
    rng = np.random.default_rng(7)
    q, k = (randn(rng, 2, 1, 64, dtype=torch.float16) for _ in range(2))
    dqo, dko = (randn(rng, 2, 1, 64, dtype=torch.float16) for _ in range(2))
    w = randn(rng, 64)
    dq, dk, dwq, _ = W.qk_norm_rope_backward(*(t.to(DEV) for t in (dqo, dko, q, k)), q_norm=w.to(DEV), k_norm=w.to(DEV),
                                             norm_eps=EPS)
    x, step = host64(q), 1e-5
    f = lambda x, w: (lm.norm_rope(x, w, EPS) * host64(dqo)).sum()
    for i in (0, 17, 63):
        a, b = x.copy(), x.copy()
        a[1, 0, i] += step
        b[1, 0, i] -= step
        slope = (f(a, host64(w)) - f(b, host64(w))) / (2 * step)
        assert abs(slope - host64(dq)[1, 0, i]) <= 2.0 ** -11 * abs(slope) + 1e-4
        a, b = host64(w), host64(w)
        a[i] += step
        b[i] -= step
        assert abs((f(x, a) - f(x, b)) / (2 * step) - host64(dwq)[i]) <= 1e-4


@pytest.mark.parametrize("dtype", DTS)
def test_many_rows(W, dtype):
    """More rows than blocks walk at once; every block's partial sum is joined; the same bytes every time."""
    rng = np.random.default_rng(12)
    n, hq, hk, d = 9001, 6, 2, 64
    q, k, dqo, dko = (randn(rng, n, h, d, dtype=dtype).to(DEV) for h in (hq, hk, hq, hk))
    qn, kn = randn(rng, d).to(DEV), randn(rng, hk, d).to(DEV)  # one shared, one a head
    a = W.qk_norm_rope_backward(dqo, dko, q, k, q_norm=qn, k_norm=kn, norm_eps=EPS)
    b = W.qk_norm_rope_backward(dqo, dko, q, k, q_norm=qn, k_norm=kn, norm_eps=EPS)
    for u, v in zip(a, b):
        assert torch.equal(u, v)
    for x, dy, w, dx, dw in ((q, dqo, qn, a[0], a[2]), (k, dko, kn, a[1], a[3])):
        x, dy, w = host64(x), host64(dy), host64(w)
        want, wdw = lm.norm_rope_backward(dy, x, w, EPS)
        r = lm.rms(x, EPS)
        size = r * np.abs(dy * w).max(-1, keepdims=True) * (1 + r ** 2 * np.abs(x) * np.mean(np.abs(x), -1, keepdims=True))
        assert np.all(np.abs(host64(dx) - want) <= U[dtype] * np.abs(want) + 80 * E32 * size + TINY)
        mass = np.abs(dy * x * r).sum(0 if w.ndim == 2 else (0, 1))
        # a lane walks rows / (blocks * rows of a block) of them, below 400 here, and the joins add 60
        assert np.all(np.abs(host64(dw) - wdw) <= (400 + 60 + NORM + 2) * E32 * mass)


@pytest.mark.parametrize("dtype", DTS)
def test_in_place_and_positions_outside(W, dtype):
    rng = np.random.default_rng(13)
    n, d = 33, 128
    q, k, dqo, dko = (randn(rng, n, h, d, dtype=dtype).to(DEV) for h in (4, 2, 4, 2))
    w = randn(rng, d).to(DEV)
    cos, sin = (t.to(DEV) for t in tables(50, 64))
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    pos[5], pos[7] = -1, 50
    kw = dict(q_norm=w, k_norm=w, cos=cos, sin=sin, positions=pos)
    filled = lambda t: torch.full_like(t, 3.0)
    yq, yk = W.qk_norm_rope(q, k, q_out=filled(q), k_out=filled(k), **kw)
    dq, dk, wq, wk = W.qk_norm_rope_backward(dqo, dko, q, k, dq=filled(q), dk=filled(k), **kw)
    for t in (yq, yk, dq, dk):
        assert (t[[5, 7]] == 3).all() and not (t[[4, 6, 8]] == 3).all()
    keep = torch.tensor([i for i in range(n) if i not in (5, 7)], device=DEV)
    part = dict(kw, positions=pos[keep])
    *_, wq2, wk2 = W.qk_norm_rope_backward(dqo[keep], dko[keep], q[keep], k[keep], **part)
    assert torch.allclose(wq, wq2, rtol=1e-4, atol=1e-4) and torch.allclose(wk, wk2, rtol=1e-4, atol=1e-4)
    a, b = dqo.clone(), dko.clone()
    W.qk_norm_rope_backward(a, b, q, k, dq=a, dk=b, **kw)
    assert torch.equal(a[keep], dq[keep]) and torch.equal(b[keep], dk[keep]) and torch.equal(a[5], dqo[5])
    a, b = q.clone(), k.clone()
    W.qk_norm_rope_backward(dqo, dko, a, b, dq=a, dk=b, **kw)
    assert torch.equal(a[keep], dq[keep]) and torch.equal(b[keep], dk[keep])
    a, b = q.clone(), k.clone()
    W.qk_norm_rope(a, b, q_out=a, k_out=b, **kw)
    assert torch.equal(a[keep], yq[keep]) and torch.equal(b[keep], yk[keep]) and torch.equal(a[7], q[7])


@pytest.mark.parametrize("dtype", DTS)
def test_rows_that_are_not_finite(W, dtype):
    """A NaN or infinity stays in its own row (and, backward, in the weights' gradient that it is part of)."""
    q, k = torch.randn(6, 2, 64, device=DEV).to(dtype), torch.randn(6, 1, 64, device=DEV).to(dtype)
    w = torch.ones(64, device=DEV)
    want = W.qk_norm_rope(q, k, q_norm=w, k_norm=w)[0]
    q2 = q.clone()
    q2[2, 1, 5], q2[4, 0, 9] = float("nan"), float("inf")
    got = W.qk_norm_rope(q2, k, q_norm=w, k_norm=w)[0]
    assert got[2, 1].isnan().all() and got[4, 0, 9].isnan()
    got[2, 1], got[4, 0] = want[2, 1], want[4, 0]
    assert torch.equal(got, want)
    zero = torch.zeros(3, 2, 64, dtype=dtype, device=DEV)
    assert (W.qk_norm_rope(zero, zero, q_norm=w, k_norm=w)[0] == 0).all()


def test_no_tokens(W):
    q, k = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, device=DEV)
    assert W.qk_norm_rope(q, k, q_norm=w, k_norm=w)[0].shape == q.shape
    *_, a, b = W.qk_norm_rope_backward(q, k, q, k, q_norm=w, k_norm=w)
    assert (a == 0).all() and (b == 0).all()


def test_captured_and_replayed(W):
    rng = np.random.default_rng(14)
    q, k, dqo, dko = (torch.zeros(70, h, 128, dtype=torch.bfloat16, device=DEV) for h in (8, 2, 8, 2))
    w = torch.ones(128, device=DEV)
    cos, sin = (t.to(DEV) for t in tables(70, 128))
    kw = dict(q_norm=w, k_norm=w, cos=cos, sin=sin, positions=torch.arange(70, dtype=torch.int32, device=DEV))
    step = lambda: (*W.qk_norm_rope(q, k, **kw), *W.qk_norm_rope_backward(dqo, dko, q, k, **kw))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for _ in range(3):
        for t in (q, k, dqo, dko):
            t.copy_(randn(rng, *t.shape))
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip(kept, step()):
            assert torch.equal(u, v)


def test_refusals(W):
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, device=DEV)
    ok = dict(q_norm=w, k_norm=w)
    for bad in (dict(q_norm=w), dict(ok, q_norm=w[:32]), dict(ok, q_norm=w.double()), dict(ok, q_norm=w.half()),
                dict(ok, k_norm=w.expand(3, 64)), dict(ok, q_norm=w.cpu()), dict(ok, cos=w)):
        with pytest.raises((ValueError, TypeError)):
            W.qk_norm_rope(q, k, **{"k_norm": None, **bad})
    with pytest.raises(ValueError):
        W.qk_norm_rope(q, k.half(), **ok)
    with pytest.raises(ValueError):
        W.qk_norm_rope(q.float(), k.float(), **ok)
    with pytest.raises(W.WhtqError):
        W.qk_norm_rope(q[..., :32].contiguous(), k[..., :32].contiguous(), q_norm=w[:32], k_norm=w[:32])
    with pytest.raises(W.WhtqError):
        W.qk_norm_rope(q, k, norm_eps=-1.0, **ok)
    with pytest.raises(ValueError):  # one vector seen as four: its gradient would be one vector
        W.qk_norm_rope_backward(q, k, q, k, q_norm=w.expand(4, 64), k_norm=w)
    big = [torch.zeros(3000, h, 64, dtype=torch.bfloat16, device=DEV) for h in (4, 2)]
    assert W.qk_norm_rope_backward_workspace_bytes(*big, **ok) > 0
    with pytest.raises(W.WhtqError):
        W.qk_norm_rope_backward(*big, *big, workspace=torch.empty(16, dtype=torch.uint8, device=DEV), **ok)
    cache = W.kv_cache_alloc(2, 16, 2, 64, device=DEV)
    with pytest.raises(ValueError):
        W.kv_append(cache, k, k, torch.arange(3, device=DEV), q_norm=w)
