"""The size query of the 4-bit attention's workspace at the ends of its arguments' range."""
import ctypes

import pytest


@pytest.mark.parametrize("hq,hkv", [(8, 8), (16, 8), (32, 8), (8, 1)])
def test_more_tokens_than_a_call_takes_have_no_size(hq, hkv):
    """0 for every num_tokens that the calls refuse, also where its product with the group size passes
    32 bits; a size for the others."""
    from sparse_kv_long_sfi_gb300 import _abi, build
    build.build()
    shape, group = _abi.sfi_attn_shape(hq, hkv, 128, 16, 0.0), hq // hkv
    size = lambda batch, T: _abi.lib().sfi_kv4_workspace_size(ctypes.byref(shape), batch, T)  # noqa: E731
    most = 16 // group
    assert all(size(3, T) > 0 for T in range(1, most + 1))
    for T in (0, -1, -2 ** 31, most + 1, 17, 1 << 28, 1 << 29, 1 << 30, (1 << 30) + 1, 2 ** 31 - 1):
        assert size(3, T) == 0, T
    assert size(-1, 1) == 0 and size(0, 1) > 0
