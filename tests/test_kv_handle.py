"""KVCache as a handle (no GPU): the addresses that the library gets are its tensors', so tensors cannot be exchanged."""
import dataclasses

import pytest

from wht_adapters_amd import whtq as W


def test_tensors_cannot_be_exchanged():
    cache = object.__new__(W.KVCache)
    for name in ("k", "v", "k_scales", "v_scales", "signs", "dim"):
        with pytest.raises(dataclasses.FrozenInstanceError):
            setattr(cache, name, None)
        with pytest.raises(dataclasses.FrozenInstanceError):
            delattr(cache, name)


def test_handles_compare_and_hash_as_themselves():
    a, b = object.__new__(W.KVCache), object.__new__(W.KVCache)
    assert a == a and a != b and len({a, b}) == 2
