"""The few-token MoE layer on activations of a wide range: x is used exactly, h to 11 bits or 2^-39 of its largest.

Weights that are exactly 0 on the columns of the large values leave outputs that
consist of the small ones alone (bounds: ops_reference.moe, in which those columns
do not count)."""
import pytest

import ops_reference as R

pytestmark = pytest.mark.gpu
LIMIT = 3e38  # no clamp

SIZES = [  # T, H, I, E, k: one to four slabs a warp, five to eight, and eight m16 tiles a tile
    (1, 512, 128, 4, 2), (9, 2048, 256, 3, 2), (32, 256, 512, 16, 8), (5, 4096, 128, 2, 1), (3, 8192, 128, 2, 2)]


def _check(out, ref, tol):
    tol = tol + (ref.abs() + tol) * R.BF16
    bad = ~((out.double() - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


@pytest.mark.parametrize("T,H,I,E,k", SIZES)
@pytest.mark.parametrize("kind", range(4))
def test_values_far_below_the_largest_count(T, H, I, E, k, kind):
    """Columns of magnitude 2^40, 1, 2^-40 and 2^-80 in turn; the weights take one of the four."""
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    g = torch.Generator(device="cuda").manual_seed(H + I + kind)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    cols = torch.arange(H, device="cuda") % 4
    w13 = torch.where(cols == kind, normal(E, 2 * I, H) * 2 / H ** 0.5, 0.0).bfloat16()
    w = api.quantize_moe_weights(w13, (normal(E, H, I) / I ** 0.5).bfloat16())
    x = normal(T, H) * torch.exp2(40.0 - 40 * cols) * torch.exp2(torch.arange(T, device="cuda")[:, None] % 5 - 2.0)
    x, logits = x.bfloat16(), normal(T, E)
    if kind == 3:
        x[:, cols == 3] *= 2.0 ** 30  # so that h stays above FP32's smallest values
    layer = api.MoEFewTokens(T, H, I, E, k)
    out = layer(x, logits, w, LIMIT, LIMIT)
    assert layer.status() == 0
    ids, p = R.route(logits, k)
    ref, tol = R.moe(x, ids, p, w, E, H, I, LIMIT, LIMIT)
    assert (ref != 0).all()
    _check(out, ref, tol)


def test_a_column_2_to_36_above_the_others():
    """One such column; the gates do not see it, and half of the up rows do not either."""
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    T, H, I, E, k = 6, 1024, 256, 4, 2
    g = torch.Generator(device="cuda").manual_seed(3)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    w13, w2 = normal(E, 2 * I, H) * 2 / H ** 0.5, normal(E, H, I) / I ** 0.5
    w13[:, :I, 77] = 0
    w13[:, I::2, 77] = 0
    w2[:, :, 1::2] = 0  # the other half's features do not reach the output
    w = api.quantize_moe_weights(w13.bfloat16(), w2.bfloat16())
    x, logits = normal(T, H).bfloat16(), normal(T, E)
    x[1:, 77] = 2.0 ** 36
    x[4, 77] = -2.0 ** 120
    x[5, :8] = 2.0 ** -133  # bf16's smallest
    out = api.MoEFewTokens(T, H, I, E, k)(x, logits, w)
    ids, p = R.route(logits, k)
    _check(out, *R.moe(x, ids, p, w, E, H, I))


@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 128, 4, 2), (9, 512, 1024, 3, 2), (4, 256, 8192, 2, 1)])
def test_h_of_a_wide_range_keeps_its_bound(T, H, I, E, k):
    """Every 16th feature about 2^28 strong, the others behind gates of about -20; half of the outputs do not
    take the strong ones."""
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    g = torch.Generator(device="cuda").manual_seed(I)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    w13, w2 = normal(E, 2 * I, H) / H ** 0.5, normal(E, H, I) / I ** 0.5
    w13[:, :I] = -20 / H * (1 + 0.2 * normal(E, I, H))
    w13[:, 0:I:16] = 2.0 ** 13 / H * (1 + 0.2 * normal(E, I // 16, H))
    w13[:, I::16] *= 2.0 ** 13
    w2[:, ::2, ::16] = 0
    w = api.quantize_moe_weights(w13.bfloat16(), w2.bfloat16())
    x, logits = (1 + 0.1 * normal(T, H)).bfloat16(), normal(T, E)
    out = api.MoEFewTokens(T, H, I, E, k)(x, logits, w, LIMIT, LIMIT)
    ids, p = R.route(logits, k)
    ref, tol = R.moe(x, ids, p, w, E, H, I, LIMIT, LIMIT)
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        gate, up = (x[t].double() @ R.decode_nvfp4(w.w13[e], w.w13_sf[e], w.w13_gs[e], 2 * I, H).T).chunk(2, 1)
        most = (gate * torch.sigmoid(gate) * up).abs().amax(1, keepdim=True)
        w2e = R.decode_nvfp4(w.w2[e], w.w2_sf[e], w.w2_gs[e], H, I)
        tol.index_add_(0, t, p[t, j][:, None] * most * 2.0 ** -39 * w2e.abs().sum(1))
    _check(out, ref, tol)
