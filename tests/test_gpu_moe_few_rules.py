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


def test_gates_far_below_zero_keep_their_silu():
    """Gates of -85 to -88.6, where 1 + exp(-gate) passes 2^126, under up values of 2^100."""
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    T, H, I = 32, 256, 128
    g = torch.Generator(device="cuda").manual_seed(0)
    w13 = torch.zeros(1, 2 * I, H, device="cuda")
    w13[:, :I, :128] = -0.7
    w13[:, I:, 128] = torch.randn(I, generator=g, device="cuda")
    w = api.quantize_moe_weights(w13.bfloat16(), torch.randn(1, H, I, generator=g, device="cuda").bfloat16())
    w13 = R.decode_nvfp4(w.w13[0], w.w13_sf[0], w.w13_gs[0], 2 * I, H)
    x = torch.zeros(T, H, device="cuda")
    x[:, :128] = (torch.linspace(-85, -88.5, T, device="cuda") / w13[0].sum())[:, None]
    x[:, 128] = 2.0 ** 100
    x = x.bfloat16()
    gate, up = (x.double() @ w13.T).chunk(2, 1)
    assert gate.min() > -88.65 and gate.max() < -84 and (gate < -87.4).sum() >= 4 * I
    out = api.MoEFewTokens(T, H, I, 1, 1)(x, torch.zeros(T, 1, device="cuda"), w, 3e38, 3e38)
    w2 = R.decode_nvfp4(w.w2[0], w.w2_sf[0], w.w2_gs[0], H, I)
    h = gate * torch.sigmoid(gate) * up
    ref = h @ w2.T
    # the gate's absolute error is its silu's relative one; then expf, the quotient and the products, h's 11 bits, the sum
    rel = 1.1 * gate.abs() * ((H / 16 * 2 + 40) * R.U32) + 16 * R.U32 + 2.0 ** -11 + (I / 16 * 2 + 40) * R.U32
    tol = (h.abs() * rel) @ w2.abs().T
    assert ((out.double() - ref).abs() <= tol + (ref.abs() + tol) * R.BF16).all()


def test_routing_tables_of_another_call_are_not_taken():
    """A ready word that an earlier call's failed launches left, in the middle of its tables (the layout: status 256
    bytes, ids 1024, then the word): the next call computes with its own routes and takes the word back."""
    import torch
    T, H, I, E, k = 12, 512, 256, 24, 4
    layer, w, x, logits = _layer(T, H, I, E, k)
    others = [torch.roll(logits, i, 1) for i in range(4)]
    want = []
    for lg in others:
        layer.workspace.fill_(0xFF)
        want.append(layer(x, lg, w).clone())
    word = layer.workspace[1280:1288].view(torch.int64)
    for turn in range(8):
        word.fill_(0x6f75746564214d4b + turn)
        assert torch.equal(layer(x, others[turn % 4], w), want[turn % 4])
        assert word.item() == 0
