"""FP8 block-scaled linear against FP64.

Bound of the FP32 sum: products of two E4M3 values are exact; a block of 128
takes at most 8 product steps (2 u32 each), its scale 2 u32, and the blocks are
added one after the other with up to 16 partial sums joined, so the error is
within (K / 128 + 40) u32 of the sum of magnitudes."""
import pytest

import ops_reference as R

pytestmark = pytest.mark.gpu


def _inputs(M, N, K, seed=0, pad=0, w_gain=0.02):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    kb = -(-K // 128)
    buf = (torch.randn(M, K + pad, generator=g, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    w = (torch.randn(N, K, generator=g, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    sa = torch.exp(torch.randn(M, kb, generator=g, device="cuda")) / 100
    sw = torch.exp(torch.randn(-(-N // 128), kb, generator=g, device="cuda")) * w_gain / 100
    return buf[:, :K], sa, w, sw


def _check(a, sa, w, sw, out):
    ref, mag = R.linear(a, sa, w, sw)
    tol = mag * ((a.shape[1] / 128 + 40) * R.U32)
    if out.dtype.itemsize == 2:
        tol = tol + (ref.abs() + tol) * R.BF16
    else:
        tol = tol + ref.abs() * R.U32
    bad = (out.double() - ref).abs() > tol
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 64, 65, 127, 128, 129, 300])
@pytest.mark.parametrize("N,K", [(8, 16), (48, 4096), (264, 400), (1000, 1296)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_linear_matches_fp64(M, N, K, dtype):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    a, sa, w, sw = _inputs(M, N, K, seed=M + N + K)
    out = torch.full((M, N), float("nan"), dtype=getattr(torch, dtype), device="cuda")
    assert api.fp8_linear(a, sa, w, sw, out=out) is out
    _check(a, sa, w, sw, out)


@pytest.mark.parametrize("M,N,K", [(5, 128, 8192), (20, 4104, 128), (40, 512, 6160), (520, 640, 2048),
                                   (1500, 1160, 1040), (257, 2304, 3584)])
def test_linear_larger(M, N, K):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    a, sa, w, sw = _inputs(M, N, K, seed=M)
    _check(a, sa, w, sw, api.fp8_linear(a, sa, w, sw))
    _check(a, sa, w, sw, api.fp8_linear(a, sa, w, sw, out_dtype=torch.float32))


# K in ranges longer than the scales held at a time (9 to 32 rows), more tiles of w than SMs, uneven K ranges
@pytest.mark.parametrize("M,N,K", [(20, 136, 66000), (9, 72, 132224), (12, 19464, 400), (32, 6144, 3600),
                                   (10, 2560, 1168)])
def test_linear_few_rows_over_a_split_k(M, N, K):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    a, sa, w, sw = _inputs(M, N, K, seed=M)
    out = api.fp8_linear(a, sa, w, sw, out_dtype=torch.float32)
    _check(a, sa, w, sw, out)
    assert torch.equal(out, api.fp8_linear(a, sa, w, sw, out_dtype=torch.float32))


@pytest.mark.parametrize("M", [20, 32])
def test_linear_split_k_strided_and_non_finite(M):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    a, sa, w, sw = _inputs(M, 520, 1040, seed=3, pad=48)
    buf = torch.full((M + 2, 544), float("nan"), dtype=torch.bfloat16, device="cuda")
    out = buf[1:M + 1, 8:528]
    api.fp8_linear(a, sa, w, sw, out=out)
    _check(a, sa, w, sw, out)
    want = out.clone()
    buf[1:M + 1, 8:528] = float("nan")
    assert torch.isnan(buf).all()  # nothing else was written
    a.view(torch.uint8)[1, 77] = 0x7F  # NaN
    sa[2, 3] = float("inf")
    w.view(torch.uint8)[130, 5] = 0xFF
    got = api.fp8_linear(a, sa, w, sw)
    assert torch.isnan(got[1]).all() and not torch.isfinite(got[2]).any() and torch.isnan(got[:, 130]).all()
    rows = [m for m in range(M) if m not in (1, 2)]
    cols = [n for n in range(520) if n != 130]
    assert torch.equal(got[rows][:, cols], want[rows][:, cols])


@pytest.mark.parametrize("M", [4, 16, 64])
def test_calls_that_follow_each_other(M):
    """Launches may overlap; each call reads what the one before wrote."""
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    a, sa, w, sw = _inputs(M, 1024, 1024, seed=9)
    x = api.fp8_linear(a, sa, w, sw)
    norm = torch.ones(1024, device="cuda")
    for _ in range(10):
        q, s, _, _ = api.add_rms_norm_fp8(x, None, norm, normed=False)
        x = api.fp8_linear(q, s, w, sw)
        torch.cuda.synchronize()
    y = api.fp8_linear(a, sa, w, sw)
    for _ in range(10):
        q, s, _, _ = api.add_rms_norm_fp8(y, None, norm, normed=False)
        y = api.fp8_linear(q, s, w, sw)
    assert torch.equal(x, y)


@pytest.mark.parametrize("M", [6, 200, 700])
def test_linear_strided_rows_and_a_slice_of_a_wider_output(M):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    a, sa, w, sw = _inputs(M, 520, 1040, seed=3, pad=48)
    buf = torch.full((M + 2, 544), float("nan"), dtype=torch.bfloat16, device="cuda")
    out = buf[1:M + 1, 8:528]
    api.fp8_linear(a, sa, w, sw, out=out)
    _check(a, sa, w, sw, out)
    buf[1:M + 1, 8:528] = float("nan")
    assert torch.isnan(buf).all()  # nothing else was written


@pytest.mark.parametrize("M", [4, 160])
def test_linear_non_finite_rows_and_blocks_stay_in_place(M):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    a, sa, w, sw = _inputs(M, 264, 512, seed=5)
    want = api.fp8_linear(a, sa, w, sw)
    a.view(torch.uint8)[1, 77] = 0x7F  # NaN
    sa[2, 3] = float("inf")
    w.view(torch.uint8)[130, 5] = 0xFF
    got = api.fp8_linear(a, sa, w, sw)
    assert torch.isnan(got[1]).all() and not torch.isfinite(got[2]).any() and torch.isnan(got[:, 130]).all()
    rows = [m for m in range(M) if m not in (1, 2)]
    cols = [n for n in range(264) if n != 130]
    assert torch.equal(got[rows][:, cols], want[rows][:, cols])


def test_linear_zero_scales_and_scale_magnitudes():
    """A row whose scales are 0 gives 0; scales at both ends of FP32's range."""
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    for M in (3, 140):
        a, sa, w, sw = _inputs(M, 136, 384, seed=9)
        sa[0] = 0
        sa[1] *= 1e30
        sw *= 1e-25
        out = api.fp8_linear(a, sa, w, sw, out_dtype=torch.float32)
        assert (out[0] == 0).all()
        _check(a, sa, w, sw, out)


def test_linear_repeats_bit_for_bit_and_rows_do_not_depend_on_each_other():
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    for M in (24, 400):
        a, sa, w, sw = _inputs(M, 1024, 2048, seed=M)
        first = api.fp8_linear(a, sa, w, sw, out_dtype=torch.float32)
        for _ in range(3):
            assert torch.equal(first, api.fp8_linear(a, sa, w, sw, out_dtype=torch.float32))


def test_linear_no_rows_own_stream_and_graph():
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    for M in (0, 12, 260):
        a, sa, w, sw = _inputs(M, 256, 640, seed=M)
        want = api.fp8_linear(a, sa, w, sw)
        assert want.shape == (M, 256)
        if M == 0:
            continue
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = api.fp8_linear(a, sa, w, sw, stream=side)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kept = api.fp8_linear(a, sa, w, sw)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(want, got) and torch.equal(want, kept)


def test_linear_takes_what_the_norm_gives():
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    x = torch.randn(50, 1792, device="cuda").bfloat16()
    q, sa, _, _ = api.add_rms_norm_fp8(x, x, torch.ones(1792, device="cuda"), normed=False)
    _, _, w, sw = _inputs(1, 328, 1792)
    _check(q, sa, w, sw, api.fp8_linear(q, sa, w, sw))


def test_linear_refuses_wrong_tensors():
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api, binding
    a, sa, w, sw = _inputs(4, 64, 256)
    for bad in (lambda: api.fp8_linear(a.float(), sa, w, sw), lambda: api.fp8_linear(a, sa[:, :1], w, sw),
                lambda: api.fp8_linear(a, sa[:3], w, sw), lambda: api.fp8_linear(a[:, :128], sa, w, sw),
                lambda: api.fp8_linear(a, sa, w, sw.half()), lambda: api.fp8_linear(a, sa.T.contiguous().T, w, sw),
                lambda: api.fp8_linear(a, sa, w, sw, out_dtype=torch.float16),
                lambda: api.fp8_linear(a, sa, w, sw, out=torch.empty(4, 63, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(binding.Nvfp4Error):
        api.fp8_linear(a, sa, w[:60], sw)  # N = 60
    torch.cuda.synchronize()
