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


class NoTruth:
    def __bool__(self):
        raise ArithmeticError("neither true nor false")


@pytest.mark.parametrize("stream,error", [(-1, OverflowError), (1 << 64, OverflowError)])
def test_a_stream_that_is_no_handle_is_refused(B, stream, error):
    """Before the tensors are looked at, so without a GPU."""
    torch = pytest.importorskip("torch")
    from nvfp4_mixture_experts_expert_gb300 import api
    t = torch.zeros(4, 128)
    for call in (lambda: api.add_rms_norm_fp8(t, t, t, stream=stream), lambda: api.fp8_linear(t, t, t, t, stream=stream),
                 lambda: api.C.moe_few_tokens(t, t, None, None, 0, (1, 2, 3, 4, 5), (t,) * 6, 1.0, 1.0, t, None, stream)):
        with pytest.raises(error):
            call()


def test_flags_that_are_neither_true_nor_false_are_refused(B):
    torch = pytest.importorskip("torch")
    from nvfp4_mixture_experts_expert_gb300 import api
    t = torch.zeros(4, 128)
    for kw in (dict(normed=NoTruth()), dict(quantized=NoTruth())):
        with pytest.raises(ArithmeticError):
            api.add_rms_norm_fp8(t, t, t, **kw)
    with pytest.raises(ValueError):  # with nothing wrong but the tensors' device
        api.add_rms_norm_fp8(t, t, t, stream=0)
