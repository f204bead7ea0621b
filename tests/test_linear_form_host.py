"""nvfp4_debug_linear_form checks its arguments and knows the calls for few rows on the host."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def B():
    from nvfp4_mixture_experts_expert_gb300 import _build
    _build.build()
    from nvfp4_mixture_experts_expert_gb300 import binding
    return binding


def _shape(B, **change):
    return B.linear_shape(**{**dict(M=4, N=64, K=128, type=0), **change})


def test_refusals(B):
    for shape, product in ((_shape(B, M=-1), 0), (_shape(B, M=0), 0), (_shape(B, N=12), 0), (_shape(B, K=0), 1),
                           (_shape(B, type=2), 0), (_shape(B, activation=6), 2), (_shape(B, groups=2), 0),
                           (_shape(B), 3), (_shape(B), -1)):
        with pytest.raises(B.Nvfp4Error) as ei:
            B.nvfp4_debug_linear_form(shape, product)
        assert ei.value.status == 1 and B.nvfp4_last_error()
    form = (ctypes.c_int32 * 4)()
    assert B._linear_form(None, 0, form) == 1 and B._linear_form(ctypes.byref(_shape(B)), 0, None) == 1


def test_few_rows(B):
    few = (0, 0, 0, 1)
    assert B.nvfp4_debug_linear_form(_shape(B)) == few and B.nvfp4_debug_linear_form(_shape(B, M=16)) == few
    assert B.nvfp4_debug_linear_form(_shape(B, M=6, groups=32, offsets=4, counts=4)) == few
    assert B.nvfp4_debug_linear_form(_shape(B, M=32, groups=256, offsets=4, counts=4)) == few


def test_many_rows_of_many_experts_are_not_few(B):
    """All of them may fall to one expert, whose matrix the few-row kernel goes over for every eighth row."""
    for M in (33, 200, 256):
        try:
            assert B.nvfp4_debug_linear_form(_shape(B, M=M, groups=256, offsets=4, counts=4))[0] > 0
        except B.Nvfp4Error as e:  # the tiles' plan asks the device
            assert e.status in (B.NVFP4_ERR_CUDA, B.NVFP4_ERR_DEVICE)
