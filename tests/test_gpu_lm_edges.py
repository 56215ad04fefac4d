"""Norms and log probabilities at calls that their documentation allows, or
refuses, beside those of test_gpu_qk_norm.py and test_gpu_logprob.py."""
import ctypes
import os
import sys

import numpy as np
import pytest
import torch

from oracle import lm
from tests.gpu_util import DEV, host64
from tests.test_gpu_logprob import DTS, check, make

# (infinities are subtracted in the bounds and then left out)
pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore:invalid value encountered")]
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def W():
    from wht_adapters_amd import whtq
    return whtq


def test_gradient_of_rows_whose_squares_overflow(W):
    """Such a row gives 0 (r is 0), and 0 is its gradient; other rows and the weights' gradient do without it."""
    rng = np.random.default_rng(31)
    x, dy = (torch.from_numpy(rng.standard_normal((6, 2, 64)).astype(np.float32)).bfloat16().to(DEV) for _ in range(2))
    w = torch.from_numpy(rng.standard_normal(64).astype(np.float32)).to(DEV)
    want = W.qk_norm_rope_backward(dy, dy[:, :1], x, x[:, :1], q_norm=w, k_norm=w)
    big = x.clone()
    big[2, 1] = 3e38 * x[2, 1].sign()   # sums of its products overflow as well
    big[4, 0] = 1e20 * x[4, 0].sign()
    y, _ = W.qk_norm_rope(big, x[:, :1], q_norm=w, k_norm=w)
    assert (y[2, 1] == 0).all() and (y[4, 0] == 0).all()
    dq, dk, dwq, dwk = W.qk_norm_rope_backward(dy, dy[:, :1], big, x[:, :1], q_norm=w, k_norm=w)
    assert (dq[2, 1] == 0).all() and (dq[4, 0] == 0).all()
    dq[2, 1], dq[4, 0] = want[0][2, 1], want[0][4, 0]
    assert torch.equal(dq, want[0]) and torch.equal(dk, want[1]) and torch.equal(dwk, want[3])
    keep = np.array([[(t, h) not in ((2, 1), (4, 0)) for h in range(2)] for t in range(6)])
    x64, dy64 = host64(x), host64(dy) * keep[..., None]
    _, dw = lm.norm_rope_backward(dy64, x64, host64(w), 1e-6)
    mass = np.abs(dy64 * x64 * lm.rms(x64, 1e-6)).sum((0, 1))
    assert np.all(np.abs(host64(dwq) - dw) <= (12 + 40 + 14 + 2) * 2.0 ** -24 * mass)  # (as for ordinary rows)


def test_rows_outside_the_positions(W):
    """A padded batch: rows that were not given are 0 there, forward and backward (whatever the memory held), and an
    adapter's gradient, summed over all rows, is that of the tokens alone.  Rows that were given stay as they were."""
    rng = np.random.default_rng(32)
    n, d = 70, 128
    q, k, dqo, dko = (torch.from_numpy(rng.standard_normal((n, h, d)).astype(np.float32)).bfloat16().to(DEV)
                      for h in (8, 2, 8, 2))
    w = torch.from_numpy(rng.standard_normal(d).astype(np.float32)).to(DEV)
    angle = np.arange(50)[:, None] * 10000.0 ** (-np.arange(0, d, 2) / d)
    cos, sin = (torch.from_numpy(f(angle).astype(np.float32)).to(DEV) for f in (np.cos, np.sin))
    pos = torch.arange(n, dtype=torch.int32, device=DEV) % 50
    gone = [0, 13, 14, 69]
    pos[gone] = torch.tensor([-1, 50, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    keep = torch.tensor([t for t in range(n) if t not in gone], device=DEV)
    for kw in (dict(), dict(rot_dim=48), dict(interleaved=True)):
        kw.update(q_norm=w, k_norm=w, cos=cos, sin=sin)
        for _ in range(3):  # freed memory of NaN is what the next allocations get
            torch.full((2 ** 22,), float("nan"), dtype=torch.bfloat16, device=DEV)
            held = [torch.full_like(t, float("nan")) for t in (q, k, q, k)]
            del held
            outs = W.qk_norm_rope(q, k, positions=pos, **kw)
            grads = W.qk_norm_rope_backward(dqo, dko, q, k, positions=pos, **kw)
            assert all((t[gone] == 0).all() for t in (*outs, *grads[:2]))
        part = [t[keep] for t in (dqo, dko, q, k)]
        want = (*W.qk_norm_rope(*part[2:], positions=pos[keep], **kw),
                *W.qk_norm_rope_backward(*part, positions=pos[keep], **kw)[:2])
        assert all(torch.equal(a[keep], b) for a, b in zip((*outs, *grads[:2]), want))
        three = torch.full_like(q, 3.0)
        yq, yk = W.qk_norm_rope(q, k, positions=pos, q_out=three, **kw)
        assert (yq[gone] == 3).all() and (yk[gone] == 0).all()
        three = torch.full_like(k, 3.0)
        dq, dk, *_ = W.qk_norm_rope_backward(dqo, dko, q, k, positions=pos, dk=three, **kw)
        assert (dq[gone] == 0).all() and (dk[gone] == 3).all()


@pytest.mark.parametrize("normed", [True, False])
@pytest.mark.parametrize("clear", [True, False])
def test_append_clears_queries(W, normed, clear):
    """The library's append may be asked to clear the queries of tokens outside the positions; the cache has none of them."""
    rng = np.random.default_rng(34)
    n, d, hq, hk = 21, 64, 4, 2
    q, k, v = (torch.from_numpy(rng.standard_normal((n, h, d)).astype(np.float32)).bfloat16().to(DEV) for h in (hq, hk, hk))
    w, table = torch.ones(d, device=DEV), torch.ones((30, d // 2), device=DEV)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    pos[[2, 20]] = torch.tensor([-1, 30], dtype=torch.int32, device=DEV)
    slots = torch.arange(n, device=DEV)
    caches = [W.kv_cache_alloc(2, 16, hk, d, device=DEV) for _ in range(2)]
    out, want = (torch.full_like(q, 3.0) for _ in range(2))
    rope = dict(cos=table, sin=table, positions=pos)
    W.kv_append(caches[0], k, v, slots, q=q, q_out=want, **rope, **(dict(q_norm=w, k_norm=w) if normed else {}))
    assert (want[[2, 20]] == 3).all()
    p, st = (lambda t: t.data_ptr()), lambda h: (ctypes.c_int64 * 2)(h * d, d)  # noqa: E731
    norm = W._Norm(p(w) if normed else 0, p(w) if normed else 0, 0, 0, W.F32 | (W._CLEAR_Q if clear else 0), 1e-6)
    turn = W._Rope(p(table), p(table), p(pos), d // 2, 30, d, 0)
    assert W.raw().kv_append_norm(caches[1]._c, p(k), st(hk), p(v), st(hk), W.BF16, n, p(slots), norm, turn, p(q), st(hq), hq,
                                  p(out), st(hq), torch.cuda.current_stream().cuda_stream) == 0
    if clear:
        want[[2, 20]] = 0
    assert torch.equal(out, want)
    assert torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v, caches[1].v)
    assert (caches[1].k[0, :, 2] == 0).all() and (caches[1].v[1, :, 4] == 0).all()


@pytest.mark.parametrize("n", [60, 3000])
@pytest.mark.parametrize("queries", [True, False])
def test_one_side_alone(W, n, queries):
    """The library's call for queries or keys alone (3000 tokens: partial sums are joined): rows as beside the other side."""
    rng = np.random.default_rng(33)
    heads, d = 3, 64
    x, dy = (torch.from_numpy(rng.standard_normal((n, heads, d)).astype(np.float32)).bfloat16().to(DEV) for _ in range(2))
    w = torch.from_numpy(rng.standard_normal(d).astype(np.float32)).to(DEV)
    both = (W.qk_norm_rope(x, x, q_norm=w, k_norm=w)[1 - queries],
            W.qk_norm_rope_backward(dy, dy, x, x, q_norm=w, k_norm=w)[1 - queries])
    lib, st = W.raw(), (ctypes.c_int64 * 2)(heads * d, d)
    p = lambda t: t.data_ptr()  # noqa: E731
    norm = W._Norm(p(w) if queries else 0, 0 if queries else p(w), 0, 0, W.F32, 1e-6)

    def sides(*own):  # pointer, stride and count where they stand, for either side
        gone = tuple(0 if v == heads else None for v in own)
        return (*own, *gone) if queries else (*gone, *own)
    y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(d, device=DEV)
    s = torch.cuda.current_stream().cuda_stream
    assert lib.qk_norm_rope(*sides(p(x), st, heads), W.BF16, d, n, norm, None, *sides(p(y), st), s) == 0
    need = lib.qk_norm_rope_backward_workspace_bytes(*((heads, 0) if queries else (0, heads)), d, n, norm)
    assert (need > 0) == (n == 3000)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    assert lib.qk_norm_rope_backward(*sides(p(dy), st, p(x), st, heads), W.BF16, d, n, norm, None, *sides(p(dx), st),
                                     p(dw) if queries else None, None if queries else p(dw), p(ws), need, s) == 0
    assert torch.equal(y, both[0]) and torch.equal(dx, both[1])
    x64, dy64 = host64(x), host64(dy)
    _, want = lm.norm_rope_backward(dy64, x64, host64(w), 1e-6)
    # a term: r (14 units) and a product (2); no more additions in a row than a lane's turns (6 at 3000 tokens) and 60 joins
    assert np.all(np.abs(host64(dw) - want) <= (6 + 60 + 16) * 2.0 ** -24 * np.abs(dy64 * x64 * lm.rms(x64, 1e-6)).sum((0, 1)))


def test_results_keep_no_scratch(W):
    """Few long rows have far more scratch than results: it is not the results' to hold."""
    x = torch.zeros((5, 2 ** 19), dtype=torch.bfloat16, device=DEV)
    t = torch.zeros(5, dtype=torch.int64, device=DEV)
    need = W.token_logprobs_workspace_bytes(5, 2 ** 19, 20)
    assert need > 20000
    r = W.token_logprobs(x, t, top=20)
    assert r.logprob.untyped_storage().nbytes() <= 1024
    assert r.top_id[0].tolist() == list(range(20))


def test_gradient_refuses_another_s_result(W):
    """A result of another vocabulary or scale would give wrong numbers without an error."""
    x = torch.randn(3, 100, device=DEV)
    t = torch.zeros(3, dtype=torch.int64, device=DEV)
    g = torch.ones(3, device=DEV)
    r = W.token_logprobs(x, t, scale=0.7)
    want = W.token_logprobs_backward(x, t, r, g, g, scale=0.7)
    assert torch.equal(W.token_logprobs_backward(x.double().float(), t, r, g, g, scale=0.7), want)
    with pytest.raises(ValueError):
        W.token_logprobs_backward(x, t, r, g, g)
    with pytest.raises(ValueError):
        W.token_logprobs_backward(x[:, :99], t, r, g, g, scale=0.7)
    with pytest.raises(ValueError):
        W.token_logprobs_backward(x[:2], t[:2], r, g[:2], g[:2], scale=0.7)


def test_too_many_of_the_likeliest(W):
    """More than the library holds is not supported; more than there are is not valid."""
    x = torch.zeros((2, 100), device=DEV)
    with pytest.raises(W.WhtqError) as e:
        W.token_logprobs(x, top=33)
    assert e.value.status == 2
    for top in (101, -1):
        with pytest.raises(W.WhtqError) as e:
            W.token_logprobs(x, top=top)
        assert e.value.status == 1


@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("rows,vocab,offset", [
    (2, 4096, 1), (3, 4095, 7), (2, 32761, 7), (2, 32762, 0), (3, 32762, 7), (2, 32767, 1), (2, 32768, 0), (5, 32768, 3),
    (2, 262144, 3), (650, 32768, 7)])
def test_at_the_borders_of_the_rules(W, dtype, rows, vocab, offset):
    """Either side of the lengths from which rows are split and groups of logits get longer; rows that begin inside 16
    bytes have one group more than the same row aligned, which may be more than are picked from at once."""
    rng = np.random.default_rng(rows + vocab + offset)
    x, xd = make(rng, min(rows, 5), vocab, dtype, offset)
    if rows > 5:  # the same few again and again
        storage = torch.empty((rows, vocab + offset + 3), dtype=dtype, device=DEV)
        storage[:, offset:offset + vocab] = x.to(DEV).repeat(rows // 5, 1)
        xd = storage[:, offset:offset + vocab]
    t = rng.integers(0, vocab, min(rows, 5))
    r = W.token_logprobs(xd, torch.from_numpy(t).to(DEV).repeat(max(1, rows // 5)), top=32)
    if rows > 5:
        names = ("logprob", "lse", "entropy", "row_ref", "row_sum", "top_logprob", "top_id")
        r = type("Last", (), {n: getattr(r, n)[-5:] for n in names})
    check(r, host64(x), t, 1.0, 32)


def test_example_without_targets():
    """A batch of nothing but padding has a gradient of 0, with the bonus for entropy too."""
    import score_and_adapt as E
    from kv_cache_decode import Linear
    gen = torch.Generator(device=DEV).manual_seed(6)
    bits = torch.randint(-2 ** 31, 2 ** 31 - 1, (128,), dtype=torch.int32, device=DEV, generator=gen)
    head, adapter = Linear(256, 4096, bits, gen), E.Adapter(256, 4096, 4000, 1, DEV)
    x = torch.randn(4, 4096, device=DEV, generator=gen).bfloat16()
    *_, dlogits, dc = E.head_step(head, adapter, x, torch.full((4,), -1, dtype=torch.int64, device=DEV), 0.1)
    assert (dlogits == 0).all() and (dc == 0).all()
