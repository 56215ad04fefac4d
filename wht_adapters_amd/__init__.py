"""MI355X (gfx950) batched Walsh-Hadamard transforms: orthonormal FWHT,
RHT + per-group RTN quantisation and its inverse, the QWHA adapter forward
and a HARP-style structured rotation; a paged key/value cache in 16 bits or
in the same rotated INT4 codes, and the attention that reads it (windows with
sinks); norms of queries and keys with their rotation, and log probabilities of
tokens, each with its gradient.

The compute lives in the HIP shared library ``libwhtq.so`` (C ABI declared in
``include/whtq.h``); ``wht_adapters_amd.whtq`` is the thin ctypes binding over
it.  Attribute access on this package loads the binding lazily so that the
input generators in ``wht_adapters_amd.synth`` import without the library.
"""

_API = ("wht_batched", "rht_quantize_rtn", "rht_dequantize_inverse",
        "qwha_adapter_forward", "harp_rotate", "KVCache", "kv_cache_alloc",
        "kv_append", "kv_gather", "kv_attention", "qk_norm_rope",
        "qk_norm_rope_backward", "token_logprobs", "token_logprobs_backward", "WhtqError", "lib_path",
        "abi_version")


def __getattr__(name):
    if name in _API:
        from . import whtq
        return getattr(whtq, name)
    raise AttributeError(name)
