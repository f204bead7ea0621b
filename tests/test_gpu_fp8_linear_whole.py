"""The FP8 linear writes every element, and each row from its own row alone.

The bounds are those of test_gpu_fp8_linear.py; here an output that is NaN, as
the buffers are before the call, is a fault."""
import pytest

import ops_reference as R
from test_gpu_fp8_linear import _inputs


def check_whole(a, sa, w, sw, out):
    ref, mag = R.linear(a, sa, w, sw)
    tol = mag * ((a.shape[1] / 128 + 40) * R.U32)
    tol = tol + (ref.abs() + tol) * (R.BF16 if out.dtype.itemsize == 2 else R.U32)
    bad = ~((out.double() - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


def test_the_check_sees_one_unwritten_element():
    import torch
    g = torch.Generator().manual_seed(0)
    a, w = (torch.randn(n, 256, generator=g).to(torch.float8_e4m3fn) for n in (5, 24))
    sa, sw = torch.rand(5, 2, generator=g), torch.rand(1, 2, generator=g)
    out = R.linear(a, sa, w, sw)[0].float()
    check_whole(a, sa, w, sw, out)
    out[4, 23] = float("nan")
    with pytest.raises(AssertionError):
        check_whole(a, sa, w, sw, out)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 64, 65, 127, 128, 129, 300])
@pytest.mark.parametrize("N,K", [(8, 16), (48, 4096), (264, 400), (1000, 1296)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_every_element_is_written(M, N, K, dtype):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    a, sa, w, sw = _inputs(M, N, K, seed=M + N + K)
    out = torch.full((M, N), float("nan"), dtype=getattr(torch, dtype), device="cuda")
    api.fp8_linear(a, sa, w, sw, out=out)
    check_whole(a, sa, w, sw, out)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(5, 128, 8192), (20, 4104, 128), (40, 512, 6160), (520, 640, 2048), (1500, 1160, 1040),
                                   (257, 2304, 3584), (20, 136, 66000), (9, 72, 132224), (12, 19464, 400), (32, 6144, 3600)])
def test_every_element_is_written_of_larger_ones(M, N, K):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    a, sa, w, sw = _inputs(M, N, K, seed=M)
    for dtype in (torch.bfloat16, torch.float32):
        buf = torch.full((M + 2, N + 16), float("nan"), dtype=dtype, device="cuda")
        out = buf[1:M + 1, 8:N + 8]
        api.fp8_linear(a, sa, w, sw, out=out)
        check_whole(a, sa, w, sw, out)
        out.fill_(float("nan"))
        assert torch.isnan(buf).all()  # nothing else was written


# every kernel: up to 8 rows, 9 to 32, tiles with K over a cluster, persistent tiles of 64 to 256 columns
@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(3, 256, 1024), (8, 48, 4096), (12, 520, 2048), (32, 6144, 1040), (100, 512, 4096),
                                   (300, 1000, 3600), (400, 4096, 512), (2000, 6144, 384)])
def test_rows_do_not_depend_on_each_other(M, N, K):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    a, sa, w, sw = _inputs(M, N, K, seed=M)
    a = a.contiguous()
    first = api.fp8_linear(a, sa, w, sw, out_dtype=torch.float32)
    changed = [0, M // 2, M - 1]
    other, other_scale, _, _ = _inputs(M, N, K, seed=M + 1)
    a[changed], sa[changed] = other[changed], other_scale[changed]
    a.view(torch.uint8)[M - 1, 5] = 0x7F  # NaN
    again = api.fp8_linear(a, sa, w, sw, out_dtype=torch.float32)
    rest = [m for m in range(M) if m not in changed]
    assert torch.equal(first[rest], again[rest])
    assert torch.isnan(again[M - 1]).all() and not torch.equal(first[0], again[0])
