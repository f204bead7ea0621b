"""Infinities and NaN in a row that the linear's gradient uses reach what the formula
lets them reach: the same bits as from finite values where the slope is what counts."""
import math

import pytest

pytestmark = pytest.mark.gpu

INF, NAN = math.inf, math.nan
# one slab of rows and several, products on few and on many rows
SIZES = [(9, 40, 24), (130, 72, 136), (700, 264, 72)]


def _randn(seed, *shape):
    import torch
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def _same(got, want):
    import torch
    for a, b in zip(got, want):
        assert a.isfinite().all() and torch.equal(a, b)


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_relu_of_a_dead_unit_stops_any_gradient(M, N, K, dtype):
    """dz = dy where z > 0, else 0, whatever dy is there (0 times infinity would be NaN)."""
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    t = getattr(torch, dtype)
    x, w, dy, z = (_randn(i, *s).to(t) for i, s in enumerate(((M, K), (N, K), (M, N), (M, N))))
    z[1, 2], z[2, 3] = 0.0, -0.0
    dead = z <= 0
    far = dy.clone()
    for i, v in enumerate((INF, -INF, NAN)):
        at = dead & (torch.arange(N, device="cuda") % 3 == i)
        far[at] = v
    none = torch.where(dead, torch.zeros_like(dy), dy)
    _same(api.linear_grad(far, x, w, z, "relu", bias=True), api.linear_grad(none, x, w, z, "relu", bias=True))
    ids = (torch.arange(M, dtype=torch.int32, device="cuda") % 3)[:, None].contiguous()
    _, order = api.sort_tokens(x, ids, 3)
    we = torch.stack((w, 2 * w, -w))
    _same(api.expert_linear_grad(far, x, we, order, z, "relu", bias=True),
          api.expert_linear_grad(none, x, we, order, z, "relu", bias=True))
    z[3, 4] = NAN  # neither above 0 nor not
    assert api.linear_grad(none, x, w, z, "relu", bias=True)[2].isnan().tolist() == [n == 4 for n in range(N)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_swiglu_slope_at_an_infinite_gate(M, N, K, dtype):
    """A gate without a limit that is infinite (as FP16 keeps a z above 65504): silu' is 1
    there as it is at 1e4, and a limited up half has no gradient."""
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    t = getattr(torch, dtype)
    x, w, dy, z = (_randn(i, *s).to(t) for i, s in enumerate(((M, K), (2 * N, K), (M, N), (M, 2 * N))))
    at = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    at[::2, ::3] = True
    z[:, N:][at] = 5.0  # above its limit
    far = z.clone()
    z[:, :N][at] = 1e4
    far[:, :N][at] = INF
    limits = (INF, 0.75)
    _same(api.linear_grad(dy, x, w, far, "swiglu", *limits, bias=True),
          api.linear_grad(dy, x, w, z, "swiglu", *limits, bias=True))
    # without limits the gate's gradient is dy u, the up's infinite as silu is
    dz = api.linear_grad(dy[:1], x[:1], w, far[:1], "swiglu", inputs=False, weights=False, bias=True)[2]
    first = at[0]
    assert torch.equal(dz[:N][first], dy[0].float()[first] * 5.0) and dz[N:][first].isinf().all()
