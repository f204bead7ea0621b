"""Rules of the few-token MoE layer that hold beside its numbers."""
import pytest

import ops_reference as R

pytestmark = pytest.mark.gpu


def _layer(T, H, I, E, k, seed=0):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    w = api.quantize_moe_weights((normal(E, 2 * I, H) * 2 / H ** 0.5).bfloat16(), (normal(E, H, I) / I ** 0.5).bfloat16())
    return api.MoEFewTokens(T, H, I, E, k), w, normal(T, H).bfloat16(), normal(T, E)


def test_infinite_and_nan_logits_route_as_in_the_whole_forward():
    """+inf (one, two, all) and NaN logits make their tokens' rows NaN in both, and no other row."""
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    T, H, I, E, k = 8, 256, 128, 8, 3
    layer, w, x, logits = _layer(T, H, I, E, k)
    fwd = api.MoEForward(T, H, I, E, k)
    a1, a2 = fwd.calibrate(x, logits, w)
    inf = float("inf")
    logits[1, 4] = inf
    logits[2, [0, 7]] = inf
    logits[4] = inf
    logits[5, 2] = float("nan")
    logits[6, 3] = -inf
    bad = torch.tensor([False, True, True, False, True, True, False, False], device="cuda")
    for out in (layer(x, logits, w), fwd(x, logits, w, a1, a2)):
        assert torch.equal(torch.isnan(out).all(1), bad) and torch.equal(torch.isnan(out).any(1), bad)
