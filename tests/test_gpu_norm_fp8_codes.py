"""The FP8 codes of the norm beside ties, and its zero rows with and without eps.

With rows of +-1 the mean square is 1 and, at eps = 0, y is the FP32 weight with
the row's signs, exactly: the codes have one right value."""
import pytest


def beside_ties(seed):
    """FP32 weight [blocks * 128]: per block a largest value A and, for every two neighbouring E4M3
    values, the FP32 numbers next to their midpoint times A / 448."""
    import torch
    g = torch.Generator().manual_seed(seed)
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    ties = (codes[1:] + codes[:-1]) / 2
    blocks = []
    for _ in range(40):
        top = torch.exp(4 * torch.randn((), generator=g))
        near = ties * (top / 448)
        for ulps in range(-2, 3):
            moved = (near.view(torch.int32) + ulps).view(torch.float32)
            blocks.append(torch.cat((top[None], moved, top[None])))
    return torch.cat(blocks)


def quotient_codes(y):
    """(codes, scales) of y [T, 128 * blocks] by the definition: FP32 quotients, rounded to nearest even.
    For tensors on the CPU: torch's division by a number on the GPU is a product with its reciprocal."""
    import torch
    blocks = y.view(y.shape[0], -1, 128)
    scale = blocks.abs().amax(2).clamp_min(2.0 ** -40) / 448
    q = (blocks / scale[..., None]).clamp(-448, 448).reshape(y.shape).to(torch.float8_e4m3fn)
    return q, scale


def test_the_weights_tell_the_two_quotients_apart():
    """Times a rounded 448 / A, some of these values take another code than over the rounded A / 448."""
    import torch
    y = beside_ties(0)[None]
    q, _ = quotient_codes(y)
    inv = 448 / y.view(1, -1, 128).abs().amax(2)
    other = (y.view(1, -1, 128) * inv[..., None]).reshape(y.shape).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert 0 < (q.view(torch.uint8) != other.view(torch.uint8)).sum() < y.numel() // 2


@pytest.mark.gpu
@pytest.mark.parametrize("blocks", [4, 30, 60, 200])  # every form of the kernel with FP32 weights
def test_codes_are_the_quotients_by_the_stored_scale(blocks):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    w = beside_ties(1)[:blocks * 128]
    x = torch.where(torch.rand(3, w.numel(), generator=torch.Generator().manual_seed(2)) < 0.5, -1.0, 1.0)
    q, scale, y, _ = api.add_rms_norm_fp8(x.bfloat16().cuda(), None, w.cuda(), 0.0)
    want_q, want_scale = quotient_codes(x * w)
    assert torch.equal(y.cpu(), (x * w).bfloat16()) and torch.equal(scale.cpu(), want_scale)
    assert torch.equal(q.view(torch.uint8).cpu(), want_q.view(torch.uint8))


@pytest.mark.gpu
def test_zero_rows_without_eps_are_nan_and_with_it_zero():
    """As 32-bit arithmetic has it: 0 * rsqrt(0) = 0 * inf."""
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    x = torch.randn(3, 640, device="cuda").bfloat16()
    x[1] = 0
    w = torch.ones(640, device="cuda")
    q, scale, y, _ = api.add_rms_norm_fp8(x, None, w, 0.0)
    assert torch.isnan(y[1]).all() and torch.isnan(scale[1]).all() and torch.isnan(q[1].float()).all()
    for t in (0, 2):
        assert torch.isfinite(y[t]).all() and torch.isfinite(scale[t]).all() and torch.isfinite(q[t].float()).all()
    q, scale, y, _ = api.add_rms_norm_fp8(x, None, w, 1e-20)
    assert (y[1] == 0).all() and (q[1].float() == 0).all() and (scale[1] == 2.0 ** -40 / 448).all()
