"""Argument checks of the norms and log probabilities (no GPU: every check runs before any HIP call)."""
import ctypes

import pytest

from wht_adapters_amd import whtq as W

from tests.test_abi_kv import EALIGN, EINVAL, EUNSUP, L, OK, P, cache, rope, st


def norm(**kw):
    n = W._Norm(P, 2 * P, 0, 0, W.F32, 1e-6)
    for k, v in kw.items():
        setattr(n, k, v)
    return n


def append(nm=None, c=None, q=P, qo=P, n=3, rp=None, heads=4):
    s = st(256, 64)
    return L.kv_append_norm(c or cache(), P, s, P, s, W.BF16, n, P, nm, rp, q, s, heads, qo, s, None)


def dense(nm=None, q=P, heads=4, k=2 * P, kv_heads=2, dt=W.BF16, dim=64, n=3, rp=None, qo=3 * P, ko=4 * P, qs=st(256, 64),
          qos=st(256, 64), ks=st(128, 64), kos=st(128, 64)):
    return L.qk_norm_rope(q, qs, heads, k, ks, kv_heads, dt, dim, n, nm or norm(), rp, qo, qos, ko, kos, None)


def back(nm=None, q=P, heads=4, k=2 * P, kv_heads=2, dt=W.BF16, dim=64, n=3, rp=None, dqo=3 * P, dko=4 * P, dq=5 * P, dk=6 * P,
         dwq=7 * P, dwk=8 * P, s=st(256, 64), dqs=st(256, 64), ws=None, wb=0):
    return L.qk_norm_rope_backward(dqo, s, q, s, heads, dko, s, k, s, kv_heads, dt, dim, n, nm or norm(), rp, dq, dqs, dk, s,
                                   dwq, dwk, ws, wb, None)


@pytest.mark.parametrize("call", [append, dense, back])
def test_norm_rules(call):
    assert call(norm(dtype=W.I8)) == EINVAL
    assert call(norm(eps=-1.0)) == EINVAL
    assert call(norm(eps=float("nan"))) == EINVAL
    assert call(norm(q_head=-64)) == EINVAL
    assert call(norm(q=P + 8)) == EALIGN
    assert call(norm(k=P + 2)) == EALIGN
    assert call(norm(k_head=66, dtype=W.BF16)) == EALIGN
    assert call(rp=rope(rot_dim=80)) == EINVAL
    assert call(rp=rope(cos=0)) == EINVAL
    assert call(rp=rope(ld=33)) == EALIGN


def test_append_norm_rules():
    assert append(norm(), q=None, qo=None) == EINVAL   # weights of queries without queries
    assert append(norm(), n=-1) == EINVAL
    assert append(norm(), c=cache(dim=96)) == EUNSUP
    assert append(norm(), n=0) == OK
    assert append(norm(q=0), q=None, qo=None, n=0) == OK
    assert append(None, n=0) == OK


@pytest.mark.parametrize("call", [dense, back])
def test_dense_rules(call):
    assert call(heads=-1) == EINVAL
    assert call(heads=0) == EINVAL              # pointers of a side that is absent
    assert call(kv_heads=0) == EINVAL
    assert call(n=-1) == EINVAL
    assert call(dt=W.F32) == EINVAL
    assert call(q=None) == EINVAL
    assert call(norm(k=0)) == EINVAL
    assert call(dim=96) == EUNSUP
    assert call(n=(1 << 30) + 1) == EUNSUP
    assert call(heads=65536) == EUNSUP
    assert call(q=P + 2) == EALIGN


def test_dense_aliases():
    assert dense(qo=P, qos=st(512, 64)) == EINVAL
    assert dense(qs=st(-256, 64)) == EINVAL
    assert dense(qo=None) == EINVAL
    assert dense(qos=st(256, 63)) == EALIGN
    assert dense(n=0) == OK
    assert dense(norm(q=0), q=None, qo=None, heads=0, n=0) == OK
    assert back(dq=P, dqs=st(512, 64)) == EINVAL
    assert back(dq=3 * P, dqs=st(512, 64)) == EINVAL
    assert back(dq=None) == EINVAL
    assert back(dwq=None) == EINVAL
    assert back(wb=-1) == EINVAL
    assert back(dwk=P + 2) == EALIGN
    assert back(ws=P + 4) == EALIGN


def test_backward_workspace_refuses():
    bytes_ = L.qk_norm_rope_backward_workspace_bytes
    assert bytes_(4, 2, 96, 3, norm()) == -1
    assert bytes_(0, 0, 64, 3, norm()) == -1
    assert bytes_(4, 2, 64, -1, norm()) == -1
    assert bytes_(4, 2, 64, 3, None) == -1


def logp(x=P, dt=W.BF16, rows=2, vocab=100, ld=100, scale=1.0, t=P, lp=P, top=0, tl=None, ti=None, ws=None, wb=0, ent=P, ref=P):
    return L.token_logprobs(x, dt, rows, vocab, ld, scale, t, lp, P, ref, P, ent, top, tl, ti, ws, wb, None)


def grad(x=P, dt=W.BF16, rows=2, vocab=100, ld=100, scale=1.0, t=P, ref=P, ent=P, g=P, h=P, dx=2 * P, ldd=100):
    return L.token_logprobs_backward(x, dt, rows, vocab, ld, scale, t, ref, P, ent, g, h, dx, ldd, None)


@pytest.mark.parametrize("call", [logp, grad])
def test_logits_rules(call):
    assert call(dt=W.I8) == EINVAL
    assert call(rows=-1) == EINVAL
    assert call(vocab=0) == EINVAL
    assert call(ld=99) == EINVAL
    for scale in (0.0, -1.0, float("nan"), float("inf"), 3e38):
        assert call(scale=scale) == EINVAL
    assert call(x=None) == EINVAL
    assert call(vocab=(1 << 20) + 1, ld=1 << 21, **({"ldd": 1 << 21} if call is grad else {})) == EUNSUP
    assert call(rows=(1 << 30) + 1) == EUNSUP
    assert call(x=P + 1) == EALIGN
    assert call(x=P + 2, dt=W.F32) == EALIGN
    assert call(t=P + 4) == EALIGN
    assert call(ent=P + 2) == EALIGN
    assert call(rows=0) == OK
    assert call(rows=0, x=None) == OK


def test_logprob_rules():
    assert logp(t=None) == EINVAL               # a place for it, and no targets
    assert logp(lp=None) == EINVAL
    assert logp(ref=None) == EINVAL             # one of the gradient's two without the other
    assert logp(top=-1) == EINVAL
    assert logp(top=101, tl=P, ti=P) == EINVAL
    assert logp(top=33, tl=P, ti=P) == EUNSUP
    assert logp(top=3) == EINVAL
    assert logp(top=3, tl=P, ti=P + 4) == EALIGN
    assert logp(wb=-1) == EINVAL
    assert logp(ws=P + 8) == EALIGN
    assert logp(x=P + 2, t=None, lp=None, rows=0) == OK
    bytes_ = L.token_logprobs_workspace_bytes
    assert bytes_(2, 100, 33) == bytes_(2, 10, 11) == bytes_(-1, 10, 1) == bytes_(2, 0, 0) == bytes_(2, 10, -1) == -1


def test_logprob_gradient_rules():
    assert grad(g=None, h=None) == EINVAL
    assert grad(t=None) == EINVAL
    assert grad(ent=None) == EINVAL
    assert grad(ref=None) == EINVAL
    assert grad(ref=P + 2) == EALIGN
    assert grad(dx=None) == EINVAL
    assert grad(ldd=99) == EINVAL
    assert grad(dx=P, ldd=101) == EINVAL        # in place with another stride
    assert grad(dx=P + 1) == EALIGN
    assert grad(g=P + 2) == EALIGN
    assert grad(t=None, g=None, rows=0) == OK


def test_sinks_rules():
    def attend(sinks, window=4, ws=None, wb=0, out=2 * P, n=3):
        return L.kv_attention_sinks(cache(), P, st(256, 64), W.BF16, n, 4, 1, P, P, P, 8, 8, 3, 100, 0.1, 1, window, sinks, out,
                                    st(256, 64), None, ws, wb, None)
    assert attend(-1) == EINVAL
    assert attend(4, window=-1) == EINVAL
    assert attend(4, out=P) == EINVAL
    assert attend(4, ws=P + 8) == EALIGN
    assert attend(4, n=0) == OK
    assert L.kv_attention_sinks_workspace_bytes(cache(), 3, 4, 1, 3, 100, 4, -1) == -1
