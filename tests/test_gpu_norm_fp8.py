"""Residual addition + RMSNorm + FP8 blocks against FP64 (bounds: ops_reference).

FP32 chain of y: the row sum adds at most 16 squares per thread and 10 levels
of a tree, all positive (26 u32, halved by the root), rsqrt 4 u32, three
products: under 32 u32 together."""
import pytest

import ops_reference as R

pytestmark = pytest.mark.gpu
REL = 32 * R.U32


def _inputs(T, H, ld=None, weight="bf16", seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rows():
        buf = torch.randn(T, ld or H, generator=g, device="cuda") * torch.exp(
            torch.randn(T, 1, generator=g, device="cuda"))
        return buf.bfloat16()[:, :H]
    w = 1 + 0.2 * torch.randn(H, generator=g, device="cuda")
    return rows(), rows(), w.bfloat16() if weight == "bf16" else w


def _check(x, res, w, eps, q, scale, y, s):
    import torch
    _, y64, scale64, v = R.norm(x, res, w, eps)
    if s is not None:
        assert torch.equal(s, (x.float() + res.float()).bfloat16())
    if y is not None:
        assert ((y.double() - y64).abs() <= (R.BF16 + REL) * y64.abs() + 1e-300).all()
    if q is not None:
        assert ((scale.double() - scale64).abs() <= (REL + 4 * R.U32) * scale64).all()
        err = (q.float().double() - v).abs()
        assert (err <= torch.maximum(v.abs() * 2.0 ** -4, torch.full_like(v, 2.0 ** -10)) * (1 + 1e-4)
                + 2 * REL * v.abs()).all()


@pytest.mark.parametrize("T,H,ld,weight", [
    (1, 16, None, "bf16"), (1, 4096, None, "f32"), (3, 128, None, "bf16"), (7, 144, 160, "f32"),
    (2, 2032, 2048, "bf16"), (65, 3584, 3840, "bf16"), (5, 4112, None, "f32"), (2, 8192, None, "bf16"),
    (3, 32768, None, "f32"), (3, 32752, 32768, "bf16"), (301, 256, None, "bf16"),
])
def test_norm_matches_fp64(T, H, ld, weight):
    from nvfp4_mixture_experts_expert_gb300 import api
    x, res, w = _inputs(T, H, ld, weight, seed=T + H)
    _check(x, res, w, 1e-6, *api.add_rms_norm_fp8(x, res, w, 1e-6))


def test_norm_without_residual_and_single_outputs():
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    x, res, w = _inputs(33, 1792)
    q, scale, y, s = api.add_rms_norm_fp8(x, None, w, 1e-5)
    assert s is None
    _check(x, None, w, 1e-5, q, scale, y, s)
    full = api.add_rms_norm_fp8(x, res, w)
    q, scale, y, s = api.add_rms_norm_fp8(x, res, w, normed=False)
    assert y is None and torch.equal(q.view(torch.uint8), full[0].view(torch.uint8)) and torch.equal(scale, full[1])
    q, scale, y, s = api.add_rms_norm_fp8(x, res, w, quantized=False)
    assert q is None and scale is None and torch.equal(y, full[2]) and torch.equal(s, full[3])


@pytest.mark.parametrize("where", ["x", "residual"])
def test_norm_in_place(where):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    x, res, w = _inputs(19, 4096, 4224)
    want = api.add_rms_norm_fp8(x, res, w)
    into = x if where == "x" else res
    q, scale, y, s = api.add_rms_norm_fp8(x, res, w, residual_out=into)
    assert s is into and torch.equal(s, want[3]) and torch.equal(y, want[2])
    assert torch.equal(q.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(scale, want[1])


def test_norm_zero_rows_zero_blocks_and_tiny_values():
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    x, res, w = _inputs(6, 1024)
    res.zero_()
    x[0] = 0                      # a zero row
    x[1, 128:256] = 0             # a zero block
    x[2] *= 1e-30                 # mean square below eps: y underflows the block floor
    w[512:640] = 0                # a block the weight clears
    q, scale, y, s = api.add_rms_norm_fp8(x, res, w, 1e-6)
    _check(x, res, w, 1e-6, q, scale, y, s)
    assert torch.isfinite(scale).all() and (q.float()[0] == 0).all() and (scale[0] == R.MIN_AMAX / 448).all()
    assert (q.float()[1, 128:256] == 0).all() and (q.float()[:, 512:640] == 0).all()


def test_norm_eps_zero_on_a_zero_row_and_non_finite_rows_stay_in_their_rows():
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    x, res, w = _inputs(8, 768)
    clean = api.add_rms_norm_fp8(x, res, w)
    x[2, 100] = float("nan")
    x[5, 700] = float("inf")
    q, scale, y, s = api.add_rms_norm_fp8(x, res, w)
    assert torch.isnan(y[2]).all() and torch.isnan(scale[2]).all() and torch.isnan(q.float()[2]).all()
    assert torch.isnan(y[5, 700]) and torch.isnan(scale[5, 5]) and (y[5, :700] == 0).all()
    for t in (0, 1, 3, 4, 6, 7):
        assert torch.equal(y[t], clean[2][t]) and torch.equal(scale[t], clean[1][t])
        assert torch.equal(q[t].view(torch.uint8), clean[0][t].view(torch.uint8))


def test_norm_no_rows_own_stream_and_graph():
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    x, res, w = _inputs(40, 2048)
    q, scale, y, s = api.add_rms_norm_fp8(x[:0], res[:0], w)
    assert q.shape == (0, 2048) and scale.shape == (0, 16) and y.shape == s.shape == (0, 2048)
    want = api.add_rms_norm_fp8(x, res, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = api.add_rms_norm_fp8(x, res, w, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = api.add_rms_norm_fp8(x, res, w)
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, kept):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and torch.equal(a.view(torch.uint8),
                                                                                    c.view(torch.uint8))


@pytest.mark.parametrize("T,H", [(1, 128), (3, 144), (1001, 512), (9000, 272)])  # one allocation for all outputs, and one each
def test_outputs_do_not_overlap(T, H):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    outs = api.add_rms_norm_fp8(*_inputs(T, H))
    spans = []
    for i, t in enumerate(outs):
        assert t.is_contiguous() and t.data_ptr() % 16 == 0
        t.view(torch.uint8).fill_(i + 1)
        spans.append((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()))
    assert all((t.view(torch.uint8) == i + 1).all() for i, t in enumerate(outs))
    spans.sort()
    assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))


def test_calls_that_follow_each_other_see_the_sums_before():
    """Launches may overlap; each call reads what the one before wrote."""
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    x, res, w = _inputs(2000, 4096)
    s = res.clone()
    for _ in range(20):
        api.add_rms_norm_fp8(x, s, w, normed=False, quantized=False, residual_out=s)
    want = res
    for _ in range(20):
        want = (want.float() + x.float()).bfloat16()
    assert torch.equal(s, want)


def test_norm_refuses_wrong_tensors():
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api, binding
    x, res, w = _inputs(4, 256)
    for bad in (lambda: api.add_rms_norm_fp8(x.float(), res, w), lambda: api.add_rms_norm_fp8(x, res[:3], w),
                lambda: api.add_rms_norm_fp8(x, res, w[:128]), lambda: api.add_rms_norm_fp8(x, res, w.half()),
                lambda: api.add_rms_norm_fp8(x.T, None, w[:4]),
                lambda: api.add_rms_norm_fp8(x, res, w, residual_out=torch.empty_like(x[:2]))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(binding.Nvfp4Error):
        api.add_rms_norm_fp8(x[:, 8:], None, w[8:], normed=True)  # 248 columns: not a multiple of 16
    with pytest.raises(binding.Nvfp4Error):
        api.add_rms_norm_fp8(x, None, w, normed=False, quantized=False)  # no output at all
    torch.cuda.synchronize()
