"""Addresses, streams and flags as callers may have them."""
import enum

import pytest


@pytest.fixture(scope="module")
def B():
    from nvfp4_mixture_experts_expert_gb300 import _build
    _build.build()
    from nvfp4_mixture_experts_expert_gb300 import binding
    return binding


def test_addresses_may_be_any_integer(B):
    class Address(int):
        pass

    class Known(enum.IntEnum):
        X = 16

    assert B._p(Address(48)) == 48 and B._p(Known.X) == 16 and B._p(32) == 32 and B._p(None) is None
    # all the way: refused for its size, not for its pointers' type
    with pytest.raises(B.Nvfp4Error) as ei:
        B.nvfp4_fp8_linear(Address(16), 256, Address(20), Known.X, Address(36), 4, 60, 256, Address(48), 64, 0, stream=0)
    assert ei.value.status == B.NVFP4_ERR_INVALID_ARG
