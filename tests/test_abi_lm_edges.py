"""Argument checks of the norms beside those of test_abi_lm.py (no GPU: every check runs before any HIP call)."""
import pytest

from wht_adapters_amd import whtq as W

from tests.test_abi_kv import EALIGN, EINVAL, OK
from tests.test_abi_lm import append, back, dense, norm


@pytest.mark.parametrize("call", [append, dense, back])
@pytest.mark.parametrize("dtype", [W.F32, W.BF16, W.F16])
def test_rows_to_clear(call, dtype):
    """The type of the weights may say which rows a token outside the positions clears, and nothing else."""
    assert call(norm(dtype=dtype | 0x400)) == EINVAL
    assert call(norm(dtype=-1)) == EINVAL
    assert call(norm(dtype=W.I8 | W._CLEAR_Q)) == EINVAL
    for flags in (W._CLEAR_Q, W._CLEAR_K, W._CLEAR_Q | W._CLEAR_K):
        # (strides are still counted in the type's size)
        assert call(norm(dtype=dtype | flags, k_head=66)) == EALIGN
        if call is not back:  # (which has weights' gradients to write without any token)
            assert call(norm(dtype=dtype | flags), n=0) == OK
