"""Argument checks of kv_append, kv_gather and kv_attention (no GPU: every check runs before any HIP call)."""
import ctypes

import pytest

from wht_adapters_amd import whtq as W

OK, EINVAL, EUNSUP, EALIGN, EHIP = 0, 1, 2, 3, 4
P = 1 << 20  # stands for an aligned device address; never touched
L = W.raw()


def cache(fmt=0, **kw):
    c = W._Cache()
    c.k, c.v = P, 2 * P
    c.num_pages, c.page_size, c.kv_heads, c.dim = 10, 16, 2, 64
    row = 64 if fmt == 0 else 32
    c.k_stride[:] = c.v_stride[:] = (32 * row, 16 * row, row)
    c.format, c.dtype = fmt, W.BF16
    if fmt == 1:
        c.k_scales, c.v_scales = 3 * P, 4 * P
        c.ks_stride[:] = c.vs_stride[:] = (32, 16)
    for k, v in kw.items():
        if isinstance(v, tuple):
            getattr(c, k)[:] = v
        else:
            setattr(c, k, v)
    return c


def st(a, b):
    return (ctypes.c_int64 * 2)(a, b)


def rope(**kw):
    r = W._Rope(P, 2 * P, 3 * P, 32, 100, 64, 0)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def append(c=None, k=P, ks=st(128, 64), v=P, vs=st(128, 64), dt=W.BF16, n=3, slots=P, rp=None, q=None, qs=st(256, 64),
           heads=4, qo=None, qos=st(256, 64)):
    return L.kv_append(c or cache(), k, ks, v, vs, dt, n, slots, rp, q, qs, heads, qo, qos, None)


def gather(c=None, n=3, slots=P, k=P, ks=st(128, 64), v=P, vs=st(128, 64), dt=W.BF16):
    return L.kv_gather(c or cache(), n, slots, k, ks, v, vs, dt, None)


def attend(c=None, q=P, qs=st(256, 64), dt=W.BF16, n=3, heads=4, seqs=1, start=P, kv=P, table=P, ts=8, tw=8, mq=3,
           mk=100, scale=0.1, causal=1, window=0, out=2 * P, os=st(256, 64), lse=None, ws=None, wb=0):
    return L.kv_attention(c or cache(), q, qs, dt, n, heads, seqs, start, kv, table, ts, tw, mq, mk, scale, causal,
                          window, out, os, lse, ws, wb, None)


@pytest.mark.parametrize("call", [append, gather, attend])
def test_cache_rules(call):
    assert call(cache(format=2)) == EINVAL
    assert call(cache(dtype=W.F32)) == EINVAL
    assert call(cache(k=0)) == EINVAL
    assert call(cache(num_pages=0)) == EINVAL
    assert call(cache(k_stride=(-64, 64, 64))) == EINVAL
    assert call(cache(1, k_scales=0)) == EINVAL
    assert call(cache(1, vs_stride=(-16, 16))) == EINVAL
    assert call(cache(dim=96)) == EUNSUP
    assert call(cache(page_size=24)) == EUNSUP
    assert call(cache(page_size=8)) == EUNSUP
    assert call(cache(num_pages=1 << 31)) == EUNSUP
    assert call(cache(v=P + 8)) == EALIGN
    assert call(cache(v_stride=(2048, 1024, 66))) == EALIGN
    assert call(cache(1, k_scales=P + 2)) == EALIGN
    assert call(cache(1, ks_stride=(32, 17))) == EALIGN
    assert call(cache(1, sign_bits=P + 1)) == EALIGN


def test_append_rules():
    assert append(dt=W.F32) == EINVAL
    assert append(dt=W.F16) == EINVAL            # not the cache's type
    assert append(n=-1) == EINVAL
    assert append(k=None) == EINVAL
    assert append(slots=None) == EINVAL
    assert append(ks=st(-1, 64)) == EINVAL
    assert append(q=P) == EINVAL                 # no q_out
    assert append(q=P, qo=P, heads=0) == EINVAL
    assert append(q=P, qo=P, qos=st(512, 64)) == EINVAL   # in place with other strides
    assert append(rp=rope(rot_dim=24)) == EINVAL
    assert append(rp=rope(rot_dim=80)) == EINVAL
    assert append(rp=rope(interleaved=2)) == EINVAL
    assert append(rp=rope(max_position=0)) == EINVAL
    assert append(rp=rope(ld=16)) == EINVAL
    assert append(rp=rope(cos=0)) == EINVAL
    assert append(n=(1 << 30) + 1) == EUNSUP
    assert append(k=P + 2) == EALIGN
    assert append(vs=st(128, 66)) == EALIGN
    assert append(q=P + 8, qo=P) == EALIGN
    assert append(slots=P + 4) == EALIGN
    assert append(rp=rope(ld=33)) == EALIGN
    assert append(rp=rope(sin=P + 4)) == EALIGN
    assert append(n=0) == OK
    assert append(cache(1), n=0, dt=W.F16, rp=rope(), q=P, qo=P) == OK


def test_gather_rules():
    assert gather(dt=W.F16) == EINVAL
    assert gather(n=-1) == EINVAL
    assert gather(slots=None) == EINVAL
    assert gather(k=None, v=None) == EINVAL
    assert gather(ks=st(-1, 0)) == EINVAL
    assert gather(k=P + 2) == EALIGN
    assert gather(vs=st(100, 64)) == EALIGN
    assert gather(slots=P + 4) == EALIGN
    assert gather(n=0) == OK


def test_attention_rules():
    assert attend(dt=W.F16) == EINVAL
    assert attend(n=-1) == EINVAL
    assert attend(heads=3) == EINVAL             # not a multiple of the cache's heads
    assert attend(seqs=-1) == EINVAL
    assert attend(mq=-1) == EINVAL
    assert attend(causal=2) == EINVAL
    assert attend(window=-1) == EINVAL
    assert attend(scale=float("nan")) == EINVAL
    assert attend(scale=float("inf")) == EINVAL
    assert attend(ts=4) == EINVAL                # rows of the table overlap
    assert attend(tw=-1) == EINVAL
    assert attend(q=None) == EINVAL
    assert attend(kv=None) == EINVAL
    assert attend(table=None) == EINVAL
    assert attend(out=P) == EINVAL               # out over q
    assert attend(wb=-1) == EINVAL
    assert attend(n=(1 << 30) + 1) == EUNSUP
    assert attend(mk=(1 << 30) + 1) == EUNSUP
    assert attend(q=P + 4) == EALIGN
    assert attend(os=st(256, 60)) == EALIGN
    assert attend(lse=P + 2) == EALIGN
    assert attend(ws=P + 8, wb=64) == EALIGN
    assert attend(start=P + 1) == EALIGN
    assert attend(n=0) == OK
    assert attend(seqs=0) == OK


def test_workspace_of_invalid_sizes():
    f = L.kv_attention_workspace_bytes
    assert f(cache(dim=96), 1, 4, 1, 1, 1, 0) == -1
    assert f(cache(), 1, 3, 1, 1, 1, 0) == -1
    assert f(cache(), -1, 4, 1, 1, 1, 0) == -1


def test_null_cache():
    assert L.kv_append(None, P, st(0, 0), P, st(0, 0), W.BF16, 1, P, None, None, None, 0, None, None, None) == EINVAL
    assert L.kv_gather(None, 1, P, P, st(0, 0), P, st(0, 0), W.BF16, None) == EINVAL


@pytest.mark.parametrize("heads", [2, 8])
@pytest.mark.parametrize("mk", [0, 100, 1 << 20])
def test_a_chunk_bound_of_zero_is_refused(heads, mk):
    """Tokens under a bound of no tokens would leave the joining kernel nothing to read but a workspace nobody wrote."""
    f = L.kv_attention_workspace_bytes
    for fmt in (0, 1):
        assert attend(cache(fmt), heads=heads, mq=0, mk=mk) == EINVAL
        assert attend(cache(fmt), heads=heads, mq=0, mk=mk, ws=P, wb=1 << 40) == EINVAL
        assert f(cache(fmt), 3, heads, 1, 0, mk, 0) == -1
        assert attend(cache(fmt), heads=heads, n=0, mq=0, mk=mk) == OK
        assert attend(cache(fmt), heads=heads, seqs=0, mq=0, mk=mk) == OK


@pytest.mark.parametrize("call", [append, gather, attend])
def test_offsets_inside_a_page_stay_below_2_31(call):
    """Strides whose product with the element's size or the page's would pass 64 bits too."""
    for fmt in (0, 1):
        for far in (1 << 27, 1 << 32, 1 << 59, 1 << 62, (1 << 62) + (1 << 61)):
            assert call(cache(fmt, k_stride=(0, 0, far))) == EUNSUP
            assert call(cache(fmt, v_stride=(0, 0, far))) == EUNSUP
