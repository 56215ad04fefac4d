"""token_logprobs and its gradient on the GPU against oracle/lm.py in fp64."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from oracle import lm
from tests.gpu_util import DEV, host64

# (infinities are subtracted in the oracle's bounds and then left out)
pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore:invalid value encountered")]

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}  # unit roundoff
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}  # half the least step
E32 = 2.0 ** -24
DTS = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def W():
    from wht_adapters_amd import whtq
    return whtq


def make(rng, rows, vocab, dtype, offset=0, spread=3.0):
    """Logits [rows, vocab] inside wider storage that starts `offset` elements in, with -inf among them."""
    x = torch.from_numpy((rng.standard_normal((rows, vocab)) * spread).astype(np.float32)).to(dtype)
    x[torch.from_numpy(rng.random((rows, vocab)) < 0.05)] = -float("inf")
    x[torch.arange(rows), torch.from_numpy(rng.integers(0, vocab, rows))] = 4.0
    if not offset:
        return x, x.to(DEV)
    wide = torch.full((rows, vocab + offset + 3), float("nan"), dtype=dtype, device=DEV)
    wide[:, offset:offset + vocab] = x.to(DEV)
    return x, wide[:, offset:offset + vocab]


def parts(r):
    return r.logprob, r.lse, r.entropy, r.row_ref, r.row_sum, r.top_logprob, r.top_id


def slack(x, scale):
    """Bounds of fp32 over a row: of the sum S (relative), and the mean of |z - max| under p."""
    z = x * scale
    m = z.max(-1, keepdims=True)
    p = np.exp(z - m)
    p /= p.sum(-1, keepdims=True)
    bar = (p * np.where(p > 0, m - z, 0)).sum(-1)
    # a term's exponent: three roundings relative to |z - m'|, m' within 2^6 of the maximum (6 log 2 < 5), and
    # exp2's own (2 units); the sum: 8 terms of every fourth chunk a lane, then 6 + 2 + 6 + 2 joins of 4 operations
    chunks = -(-x.shape[1] // 512)
    return E32 * (3 * (bar + 5) + 4 + 8 * -(-chunks // 4) + 64), bar


def check(r, x, t, scale, top):
    want = lm.logprobs(x, t, scale, top)
    rel, bar = slack(np.where(np.isnan(x), 0, x), scale)
    lse, lp, ent = host64(r.lse), host64(r.logprob), host64(r.entropy)
    fine = np.isfinite(want["lse"])
    assert np.array_equal(lse[~fine], want["lse"][~fine], equal_nan=True)
    assert np.array_equal(ent[~fine], want["entropy"][~fine], equal_nan=True)
    assert np.array_equal(lp[~np.isfinite(want["logprob"])], want["logprob"][~np.isfinite(want["logprob"])], equal_nan=True)
    # log S moves by rel, its logarithm and the sum with m by 4 units of what they add up
    size = np.abs(x[np.arange(len(t)), np.clip(t, 0, x.shape[1] - 1)] * scale)
    m = np.nanmax(np.where(np.isfinite(x), x, -1e30), -1) * scale
    for got, ref in ((lse, want["lse"]), (lp, want["logprob"])):
        ok = np.isfinite(ref)
        bound = rel + 4 * E32 * (np.abs(m) + size + np.abs(want["lse"]) + 20)
        assert np.all(np.abs(got - ref)[ok] <= bound[ok])
    # what the gradient takes: a logit near the largest, and the sum relative to it
    ref, total = host64(r.row_ref), host64(r.row_sum)
    assert np.all(np.abs(ref * scale - m)[fine] <= 6 * np.log(2) + 1e-6)
    assert np.all(np.abs(ref * scale + np.log(np.where(fine, total, 1)) - want["lse"])[fine] <= (rel + 2 * E32)[fine])
    # log S - T / S, T relative like S with one rounding more a term
    assert np.all(np.abs(ent - want["entropy"])[fine] <= ((2 * rel + 8 * E32) * (1 + bar + 5 + np.abs(want["lse"] - m)))[fine])
    if top:
        assert np.array_equal(r.top_id.cpu().numpy(), want["top_id"])
        tl, wl = host64(r.top_logprob), want["top_logprob"]
        ok = np.isfinite(wl)
        assert np.array_equal(tl[~ok], wl[~ok], equal_nan=True)
        bound = np.broadcast_to((rel + 4 * E32 * (np.abs(m) + np.abs(want["lse"]) + 20))[:, None], wl.shape)
        assert np.all(np.abs(tl - wl)[ok] <= (bound + 4 * E32 * np.abs(wl))[ok])


@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("rows,vocab,top,offset", [
    (1, 1, 1, 0), (3, 2, 2, 1), (5, 7, 7, 3), (2, 31, 31, 0), (4, 513, 20, 5), (7, 1000, 32, 1), (1, 4096, 5, 0),
    (3, 4097, 32, 1), (2, 30001, 32, 7), (2, 32769, 20, 1), (1, 131072, 20, 0), (600, 5003, 3, 1), (300, 40000, 0, 0)])
def test_rows(W, dtype, rows, vocab, top, offset):
    rng = np.random.default_rng(rows + vocab)
    x, xd = make(rng, rows, vocab, dtype, offset)
    t = rng.integers(0, vocab, rows)
    t[rng.random(rows) < 0.2] = -1
    if rows > 2:
        t[1] = vocab
    for scale in (1.0, 0.7):
        r = W.token_logprobs(xd, torch.from_numpy(t).to(DEV), top=top, scale=scale)
        check(r, host64(x), t, scale, top)


@pytest.mark.parametrize("more", [-1, 0])
def test_one_block_a_row_or_several(W, more):
    """On either side of the number of rows from which a block has a row to itself, and the largest vocabulary either way."""
    rows = -(-5 * torch.cuda.get_device_properties(0).multi_processor_count // 2) + more
    rng = np.random.default_rng(21)
    x, xd = make(rng, rows, 33001, torch.bfloat16, 1)
    t = rng.integers(0, 33001, rows)
    assert (W.token_logprobs_workspace_bytes(rows, 33001, 2) == 0) == (more == 0)
    check(W.token_logprobs(xd, torch.from_numpy(t).to(DEV), top=2), host64(x), t, 1.0, 2)
    vocab, few = 2 ** 20, 2
    x, xd = make(rng, few, vocab, torch.float16)
    t = rng.integers(0, vocab, few)
    if more < 0:
        return check(W.token_logprobs(xd, torch.from_numpy(t).to(DEV), top=32), host64(x), t, 1.0, 32)
    long = xd.repeat(rows // few, 1)  # (whatever its size: each row by a block of its own)
    r = W.token_logprobs(long, torch.from_numpy(t).to(DEV).repeat(rows // few), top=32)
    names = ("logprob", "lse", "entropy", "row_ref", "row_sum", "top_logprob", "top_id")
    last = SimpleNamespace(**{n: v[-few:] for n, v in zip(names, parts(r))})
    check(last, host64(x), t, 1.0, 32)


@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("vocab", [300, 5000, 70000])
@pytest.mark.parametrize("values", [1, 2, 40])
def test_ties_go_to_the_lower_index(W, dtype, vocab, values):
    """Few different values (one: every logit ties, the candidates overflow), zeros of both signs among them."""
    rng = np.random.default_rng(vocab + values)
    x = rng.integers(0, values, (5, vocab)).astype(np.float32) - values // 2
    x[:, ::3] *= np.where(x[:, ::3] == 0, -1.0, 1.0)
    x[4] = -np.inf
    x[4, vocab // 2] = 1.0
    x = torch.from_numpy(x).to(dtype)
    t = np.array([0, 1, 2, -1, 5])
    r = W.token_logprobs(x.to(DEV), torch.from_numpy(t).to(DEV), top=32)
    check(r, host64(x), t, 1.0, 32)


@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("vocab", [9, 777, 40000])
def test_rows_that_are_not_finite(W, dtype, vocab):
    inf, nan = float("inf"), float("nan")
    rng = np.random.default_rng(vocab)
    x = torch.from_numpy(rng.standard_normal((7, vocab)).astype(np.float32)).to(dtype)
    x[0] = -inf
    x[1, vocab // 2] = nan
    x[2] = nan
    x[3, vocab - 1] = inf
    x[4, 1:] = -inf
    x[5, 0] = -inf
    t = np.array([3, 0, 1, vocab - 1, 0, 0, -7])
    td = torch.from_numpy(t).to(DEV)
    for top in (0, 4):
        r = W.token_logprobs(x.to(DEV), td, top=top)
        check(r, host64(x), t, 1.0, top)
    ones = torch.ones(7, device=DEV)
    d = host64(W.token_logprobs_backward(x.to(DEV), td, r, ones, ones))
    assert (d[0] == 0).all() and np.isnan(d[1]).any() and np.isnan(d[2]).all() and np.isnan(d[3]).any()
    assert np.isfinite(d[4:]).all() and (d[4] == 0).all()  # one token left: p = 1, and no way to move it


@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("rows,vocab,offset", [(1, 1, 0), (3, 2, 1), (5, 13, 0), (4, 1001, 3), (2, 8193, 1), (3, 50257, 0),
                                               (200, 3001, 5)])
def test_gradient(W, dtype, rows, vocab, offset):
    rng = np.random.default_rng(rows * vocab)
    x, xd = make(rng, rows, vocab, dtype, offset)
    t = rng.integers(0, vocab, rows)
    t[rng.random(rows) < 0.2] = -1
    g, h = (torch.from_numpy(rng.standard_normal(rows).astype(np.float32)) for _ in range(2))
    junk = g.clone()
    junk[torch.from_numpy(t < 0)] = float("nan")  # of no account without a target
    td = torch.from_numpy(t).to(DEV)
    x64 = host64(x)
    for scale, gg, hh in ((1.0, g, None), (0.7, None, h), (1.3, g, h)):
        r = W.token_logprobs(xd, td, scale=scale)
        got = host64(W.token_logprobs_backward(xd, td, r, None if gg is None else junk.to(DEV),
                                               None if hh is None else hh.to(DEV), scale=scale))
        g64 = np.zeros(rows) if gg is None else host64(gg)
        h64 = np.zeros(rows) if hh is None else host64(hh)
        want = lm.logprobs_backward(x64, t, g64, h64, scale)
        o = lm.logprobs(x64, t, scale)
        rel, bar = slack(x64, scale)
        lp = x64 * scale - o["lse"][:, None]
        p = np.exp(lp)
        lp = np.where(p > 0, lp, 0)
        # p: the exponent's roundings (4 of |lp| and of log S) and S's; the bracket: its terms' roundings and the entropy's error
        m = np.where(np.isfinite(x64), x64, -1e30).max(-1) * scale
        ep = rel[:, None] + 4 * E32 * (np.abs(lp) + np.abs(o["lse"] - m)[:, None] + 10)
        inner = np.abs(g64)[:, None] + np.abs(h64)[:, None] * (np.abs(lp) + o["entropy"][:, None])
        ent = (2 * rel + 8 * E32) * (1 + bar + 5 + np.abs(o["lse"] - m))
        bound = U[dtype] * np.abs(want) + TINY[dtype] + scale * (
            p * (inner * (ep + 8 * E32) + np.abs(h64)[:, None] * (ep + ent[:, None])) + 4 * E32 * (np.abs(g64)[:, None] * (t == np.arange(vocab)[:, None]).T if gg is not None else 0))
        assert np.all(np.abs(got - want) <= bound * (1 + 1e-6))


def test_gradient_of_large_logits(W):
    """Logits around 3000: lse is good to 2^-13 there, the gradient does not go by it."""
    rng = np.random.default_rng(5)
    x = torch.from_numpy((rng.standard_normal((3, 2000)) * 2 + 3000).astype(np.float32))
    t = np.array([4, 5, 1999])
    td, ones = torch.from_numpy(t).to(DEV), torch.ones(3, device=DEV)
    r = W.token_logprobs(x.to(DEV), td)
    got = host64(W.token_logprobs_backward(x.to(DEV), td, r, ones))
    want = lm.logprobs_backward(host64(x), t, np.ones(3), np.zeros(3))
    rel, _ = slack(host64(x), 1.0)
    p = np.exp(host64(x) - lm.logprobs(host64(x), t)["lse"][:, None])
    assert np.all(np.abs(got - want) <= p * (rel[:, None] + 4 * E32 * 40) + 4 * E32)


@pytest.mark.parametrize("dtype", DTS)
def test_in_place_and_other_strides(W, dtype):
    rng = np.random.default_rng(8)
    x, xd = make(rng, 6, 3001, dtype, 1)
    t = torch.from_numpy(rng.integers(0, 3001, 6)).to(DEV)
    g = torch.randn(6, device=DEV)
    r = W.token_logprobs(xd, t)
    want = W.token_logprobs_backward(xd, t, r, g, g)
    wide = torch.full((6, 3010), 7.0, dtype=dtype, device=DEV)
    assert W.token_logprobs_backward(xd, t, r, g, g, out=wide[:, 2:3003]) is not None
    assert torch.equal(wide[:, 2:3003], want) and (wide[:, :2] == 7).all() and (wide[:, 3003:] == 7).all()
    W.token_logprobs_backward(xd, t, r, g, g, out=xd)
    assert torch.equal(xd, want)


def test_rows_do_not_depend_on_the_call(W):
    """A row of a long batch, alone: another split of its logits, the same tokens; the same call twice: the same bytes."""
    rng = np.random.default_rng(9)
    x, xd = make(rng, 2100, 9001, torch.bfloat16)
    t = torch.from_numpy(rng.integers(0, 9001, 2100)).to(DEV)
    a, b = W.token_logprobs(xd, t, top=6), W.token_logprobs(xd, t, top=6)
    for u, v in zip(parts(a), parts(b)):
        assert torch.equal(u, v)
    one = W.token_logprobs(xd[77:78], t[77:78], top=6)
    assert torch.equal(one.top_id[0], a.top_id[77])
    rel, _ = slack(host64(x)[77:78], 1.0)
    assert abs(float(one.logprob[0]) - float(a.logprob[77])) <= 2 * rel[0] + 64 * E32


@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("scale", [1.0, 0.5, 2.0])
def test_masks_of_the_lowest_value(W, dtype, scale):
    """Rows masked with the type's lowest value, in part, but for one token, and whole (uniform, like any row of equals)."""
    rng = np.random.default_rng(11)
    low = torch.finfo(dtype).min
    x = torch.from_numpy(rng.standard_normal((4, 1500)).astype(np.float32)).to(dtype)
    x[0, ::2] = low
    x[1] = low
    x[1, 77] = 1.0
    x[2] = low
    x[3, :-1] = -float("inf")
    x[3, -1] = low
    t = np.array([1, 77, 5, 1499])
    td, ones = torch.from_numpy(t).to(DEV), torch.ones(4, device=DEV)
    r = W.token_logprobs(x.to(DEV), td, top=3, scale=scale)
    with np.errstate(over="ignore"):
        # (in fp64 the lowest value is as good as -inf next to others, and a row of it alone as good as a row of 0)
        y = host64(x)
    y = np.where(y <= float(low), -np.inf, y)
    y[2], y[3, -1] = 0.0, 0.0
    want = lm.logprobs(y, t, scale, 3)
    rel, _ = slack(y, scale)
    # (twice the lowest bf16 or fp32 value is beyond fp32, which lse is given in: -inf there)
    with np.errstate(over="ignore"):
        assert float(r.lse[2]) == pytest.approx(float(np.float32(float(low) * scale + np.log(1500))), rel=2 * E32)
    assert np.all(np.abs(host64(r.logprob) - want["logprob"]) <= rel + 64 * E32)
    assert np.all(np.abs(host64(r.entropy) - want["entropy"]) <= (2 * rel + 8 * E32) * 24)
    ids = r.top_id.cpu().numpy()
    assert ids[0].tolist() == want["top_id"][0].tolist() and ids[1].tolist() == [77, 0, 1] and ids[2].tolist() == [0, 1, 2]
    assert ids[3].tolist() == [1499, 0, 1]
    got = host64(W.token_logprobs_backward(x.to(DEV), td, r, ones, ones, scale=scale))
    wg = lm.logprobs_backward(y, t, np.ones(4), np.ones(4), scale)
    assert np.all(np.abs(got - wg) <= U[dtype] * np.abs(wg) + TINY[dtype] + scale * (4 * rel[:, None] + 400 * E32) * (np.exp(np.maximum(y * scale - want["lse"][:, None], -700)) * 12 + E32))


def test_nothing_to_do(W):
    x = torch.zeros((0, 100), device=DEV)
    t = torch.zeros(0, dtype=torch.int64, device=DEV)
    r = W.token_logprobs(x, t, top=3)
    assert r.top_id.shape == (0, 3) and r.logprob.shape == (0,)
    assert W.token_logprobs_backward(x, t, r, torch.zeros(0, device=DEV)).shape == (0, 100)
    x = torch.randn(4, 50, device=DEV)
    r = W.token_logprobs(x)
    assert r.logprob is None and r.top_id is None
    assert torch.equal(W.token_logprobs_backward(x, None, r, None, torch.zeros(4, device=DEV)), torch.zeros_like(x))


def test_captured_and_replayed(W):
    rng = np.random.default_rng(10)
    x = torch.zeros((5, 33000), dtype=torch.bfloat16, device=DEV)
    t = torch.zeros(5, dtype=torch.int64, device=DEV)
    g = torch.ones(5, device=DEV)
    ws = torch.empty(W.token_logprobs_workspace_bytes(5, 33000, 4), dtype=torch.uint8, device=DEV)

    def step():
        r = W.token_logprobs(x, t, top=4, workspace=ws)
        return r, W.token_logprobs_backward(x, t, r, g, g)
    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept, dx = step()
    for _ in range(3):
        x.copy_(torch.from_numpy(rng.standard_normal((5, 33000)).astype(np.float32)))
        t.copy_(torch.from_numpy(rng.integers(0, 33000, 5)))
        graph.replay()
        torch.cuda.synchronize()
        r, d = step()
        for u, v in zip(parts(kept), parts(r)):
            assert torch.equal(u, v)
        assert torch.equal(dx, d)


def test_refusals(W):
    x = torch.zeros((2, 10), device=DEV)
    t = torch.zeros(2, dtype=torch.int64, device=DEV)
    for bad in (x.double(), x[0], x.t().contiguous().t(), x.cpu()):
        with pytest.raises(ValueError):
            W.token_logprobs(bad, t)
    with pytest.raises(ValueError):
        W.token_logprobs(x, t.int())
    with pytest.raises(ValueError):
        W.token_logprobs(x, t[:1])
    for kw in (dict(top=11), dict(top=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan"))):
        with pytest.raises(W.WhtqError):
            W.token_logprobs(x, t, **kw)
    long = torch.zeros((2, 50000), device=DEV)  # few long rows are split over blocks
    assert W.token_logprobs_workspace_bytes(2, 50000, 3) > 16
    with pytest.raises(W.WhtqError):
        W.token_logprobs(long, t, top=3, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    r = W.token_logprobs(x, t)
    g = torch.zeros(2, device=DEV)
    with pytest.raises(W.WhtqError):
        W.token_logprobs_backward(x, t, r)
    with pytest.raises(W.WhtqError):
        W.token_logprobs_backward(x, None, r, g)
    for kw in (dict(dlogprob=g.double()), dict(dlogprob=g[:1]), dict(dlogprob=g, out=x.half()),
               dict(dlogprob=g, out=torch.zeros((2, 9), device=DEV))):
        with pytest.raises(ValueError):
            W.token_logprobs_backward(x, t, r, **kw)
