"""The few-token MoE layer against FP64 on the weights' exact values (bounds:
ops_reference.moe, then one rounding to bf16)."""
import pytest

import ops_reference as R

pytestmark = pytest.mark.gpu
_kept = {}


def _weights(E, H, I):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    if (E, H, I) not in _kept:
        g = torch.Generator(device="cuda").manual_seed(E + H + I)
        w13 = (torch.randn(E, 2 * I, H, generator=g, device="cuda") * 2 / H ** 0.5).bfloat16()
        w2 = (torch.randn(E, H, I, generator=g, device="cuda") / I ** 0.5).bfloat16()
        _kept[E, H, I] = api.quantize_moe_weights(w13, w2)
    return _kept[E, H, I]


def _x(T, H, seed=0, pad=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H + pad, generator=g, device="cuda") * torch.exp(torch.randn(T, 1, generator=g, device="cuda"))
    x[:, ::37] *= 20
    return x.bfloat16()[:, :H]


def _logits(T, E, seed=1):
    import torch
    return torch.randn(T, E, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def _layer(T, H, I, E, k):
    from nvfp4_mixture_experts_expert_gb300 import api
    layer = api.MoEFewTokens(T, H, I, E, k)
    layer.workspace.fill_(0xFF)  # nothing of an earlier call is needed
    return layer


def _check(out, ref, tol):
    tol = tol + (ref.abs() + tol) * R.BF16
    bad = ~((out.double() - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


SIZES = [  # T, H, I, E, k
    (1, 256, 128, 8, 2), (1, 256, 128, 1, 1), (2, 512, 384, 3, 3), (3, 1792, 640, 12, 4), (5, 768, 1152, 16, 8),
    (8, 1024, 256, 64, 6), (9, 256, 512, 256, 8), (16, 512, 128, 5, 2), (17, 1280, 896, 31, 5), (31, 256, 128, 40, 8),
    (32, 1024, 512, 48, 6), (32, 256, 256, 4, 4), (1, 4096, 2048, 8, 6), (4, 8192, 128, 4, 2), (4, 256, 8192, 4, 2),
    (2, 7168, 2176, 3, 2), (32, 256, 2048, 64, 8), (32, 2048, 128, 200, 8), (20, 512, 256, 38, 1),
]


@pytest.mark.parametrize("T,H,I,E,k", SIZES)
def test_layer_matches_fp64(T, H, I, E, k):
    w, x, logits = _weights(E, H, I), _x(T, H, T), _logits(T, E)
    layer = _layer(T, H, I, E, k)
    out = layer(x, logits, w)
    assert layer.status() == 0
    ids, p = R.route(logits, k)
    _check(out, *R.moe(x, ids, p, w, E, H, I))


@pytest.mark.parametrize("T", [1, 7, 8, 9, 25, 32])
def test_every_token_to_the_same_experts(T):
    """Experts with more tokens than one product takes at a time."""
    import torch
    H, I, E, k = 512, 384, 6, 2
    w, x = _weights(E, H, I), _x(T, H, 4)
    logits = torch.tensor([0.5, 3.0, 0.25, -1.0, 4.0, 0.0], device="cuda").repeat(T, 1)
    out = _layer(T, H, I, E, k)(x, logits, w)
    ids, p = R.route(logits, k)
    _check(out, *R.moe(x, ids, p, w, E, H, I))


def test_ties_go_to_the_lower_expert():
    import torch
    H, I, E, k, T = 256, 128, 40, 4, 6
    w, x = _weights(E, H, I), _x(T, H, 5)
    logits = torch.zeros(T, E, device="cuda")
    logits[1, 10:] = 1
    logits[2, ::2] = -0.0
    out = _layer(T, H, I, E, k)(x, logits, w)
    ids, p = R.route(logits, k)
    assert ids[0].tolist() == [0, 1, 2, 3] and ids[1].tolist() == [10, 11, 12, 13]
    _check(out, *R.moe(x, ids, p, w, E, H, I))


def test_masked_logits():
    """-inf logits: fewer experts than top_k, one, and none (a zero row)."""
    import torch
    H, I, E, k, T = 512, 256, 16, 4, 5
    w, x, logits = _weights(E, H, I), _x(T, H, 6), _logits(5, 16)
    inf = float("inf")
    logits[1, 2:] = -inf
    logits[2, :15] = -inf
    logits[3] = -inf
    logits[4] = torch.finfo(torch.float32).min  # the type's lowest value everywhere: a tie, not a mask
    layer = _layer(T, H, I, E, k)
    out = layer(x, logits, w)
    ids, p = R.route(logits, k)
    assert p[1].count_nonzero() == 2 and p[2].tolist() == [1, 0, 0, 0] and p[3].sum() == 0 and p[4].tolist() == [.25] * 4
    _check(out, *R.moe(x, ids, p, w, E, H, I))
    assert (out[3] == 0).all()
    logits.fill_(-inf)
    assert (layer(x, logits, w) == 0).all()
    assert layer.status() == 0


def test_masked_experts_are_not_read_and_bad_tokens_stay_alone():
    """NaN weights behind a -inf logit, a NaN token and an infinite one leave the others' rows alone."""
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    H, I, E, k, T = 256, 256, 8, 3, 9
    w, x, logits = _weights(E, H, I), _x(T, H, 7), _logits(9, 8)
    logits[:, 5] = -float("inf")
    layer = _layer(T, H, I, E, k)
    want = layer(x, logits, w).clone()
    gs = w.w13_gs.clone()
    gs[5] = float("nan")
    x2 = x.clone()
    x2[1, 3] = float("nan")
    x2[4, 200] = float("inf")
    got = layer(x2, logits, api.MoEWeights(w.w13, w.w13_sf, gs, w.w2, w.w2_sf, w.w2_gs))
    rows = [0, 2, 3, 5, 6, 7, 8]
    assert torch.equal(got[rows], want[rows]) and torch.isnan(got[1]).all() and not torch.isfinite(got[4]).all()


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e6, 1e18])
def test_activations_of_any_magnitude(scale):
    import torch
    H, I, E, k, T = 512, 256, 4, 2, 3
    w, x, logits = _weights(E, H, I), (_x(T, H, 8).float() * scale).bfloat16(), _logits(3, 4)
    lim = 3e38  # no clamp
    out = _layer(T, H, I, E, k)(x, logits, w, gate_limit=lim, up_limit=lim)
    ids, p = R.route(logits, k)
    ref, tol = R.moe(x, ids, p, w, E, H, I, lim, lim)
    # at 1e18 one token's h and output pass FP32's range in the definition itself: that row is inf or NaN
    fine = ref.abs().amax(1) < torch.finfo(torch.float32).max
    assert fine.sum() >= T - 1 and not torch.isfinite(out[~fine]).all(1).any()
    # below FP32's normal range nothing is promised but smallness
    out, ref, tol = out.double()[fine], ref[fine], tol[fine]
    assert ((out - ref).abs() <= tol + (ref.abs() + tol) * R.BF16 + 2e-38).all()


@pytest.mark.parametrize("T,H,I,E,k,total,start", [(5, 1792, 640, 12, 4, 24, 6), (1, 256, 128, 4, 8, 64, 60),
                                                    (32, 512, 256, 6, 6, 48, 40), (3, 256, 128, 2, 2, 64, 62)])
def test_routed_layer(T, H, I, E, k, total, start):
    """Global ids, of which some, all or none are held here; top_k above E."""
    import torch
    w, x = _weights(E, H, I), _x(T, H, 9)
    ids, p = R.route(_logits(T, total, T), k)
    p32 = p.float()
    layer = _layer(T, H, I, E, k)
    out = layer.routed(x, ids.int(), p32, start, w)
    assert layer.status() == 0
    _check(out, *R.moe(x, ids - start, p32, w, E, H, I))
    none = torch.full_like(ids, start + E).int()
    assert (layer.routed(x, none, p32, start, w) == 0).all()
    none[:, 0] = -2 ** 31  # far outside
    assert (layer.routed(x, none, p32, start, w) == 0).all()


def test_routed_layer_repeated_ids_zero_and_negative_weights():
    import torch
    H, I, E, k, T = 256, 384, 5, 4, 4
    w, x = _weights(E, H, I), _x(T, H, 10)
    ids = torch.tensor([[1, 1, 2, 1], [0, 3, 3, 0], [4, 4, 4, 4], [2, 0, 1, 9]], dtype=torch.int32, device="cuda")
    p = torch.tensor([[.25, .5, 1., -.125], [0., .5, .25, 0.], [1, 2, 3, 4], [-1., 0., 2., 5.]], device="cuda")
    out = _layer(T, H, I, E, k).routed(x, ids, p, 0, w)
    _check(out, *R.moe(x, ids.long(), p.double(), w, E, H, I))


def test_fewer_tokens_than_the_layer_was_made_for_strided_rows_and_repeats():
    import torch
    H, I, E, k = 1024, 384, 10, 3
    w, x, logits = _weights(E, H, I), _x(20, H, 11, pad=72), _logits(20, 10)
    layer = _layer(32, H, I, E, k)
    full = layer(x, logits, w)
    ids, p = R.route(logits, k)
    _check(full, *R.moe(x, ids, p, w, E, H, I))
    for T in (1, 6, 13, 20):
        buf = torch.full((T + 2, H), float("nan"), dtype=torch.bfloat16, device="cuda")
        layer(x[:T], logits[:T], w, out=buf[1:T + 1])
        assert torch.isnan(buf[0]).all() and torch.isnan(buf[-1]).all()
        _check(buf[1:T + 1], *R.moe(x[:T], ids[:T], p[:T], w, E, H, I))
    for _ in range(4):
        assert torch.equal(full, layer(x, logits, w))
    assert layer(x[:0], logits[:0], w).shape == (0, H)


def test_limits():
    H, I, E, k, T = 512, 256, 4, 2, 4
    w, x, logits = _weights(E, H, I), _x(T, H, 12), _logits(4, 4)
    for gl, ul in ((0.5, 10.0), (10.0, 0.25), (1e-3, 1e-3)):
        out = _layer(T, H, I, E, k)(x, logits, w, gl, ul)
        ids, p = R.route(logits, k)
        _check(out, *R.moe(x, ids, p, w, E, H, I, gl, ul))


def test_own_stream_and_graph():
    import torch
    H, I, E, k, T = 1024, 512, 48, 6, 8
    w, x, logits = _weights(E, H, I), _x(T, H, 13), _logits(8, 48)
    layer = _layer(T, H, I, E, k)
    want = layer(x, logits, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = layer(x, logits, w, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = layer(x, logits, w)
    for _ in range(3):
        kept.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(want, kept)
    assert torch.equal(want, got) and layer.status() == 0


def test_routes_of_earlier_calls_are_not_used():
    """The second launch takes the first's routing tables; those of a call before
    are still in the workspace."""
    import torch
    H, I, E, k, T = 512, 256, 24, 4, 12
    w, x, layer = _weights(E, H, I), _x(T, H, 14), _layer(T, H, I, E, k)
    every = [_logits(T, E, seed) for seed in range(6)]
    want = []
    for logits in every:
        ids, p = R.route(logits, k)
        want.append(R.moe(x, ids, p, w, E, H, I))
        _check(layer(x, logits, w), *want[-1])
    ids, p = R.route(every[0], k)
    ids, p = ids.int().contiguous(), p.float().contiguous()
    _check(layer.routed(x, ids, p, 0, w), *want[0])
    static = every[5].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x, static, w)
    outs = []
    for logits in every:  # replays back to back
        static.copy_(logits)
        graph.replay()
        outs.append(out.clone())
    for got, ref in zip(outs, want):
        _check(got, *ref)


def test_nearer_to_the_weights_layer_than_the_quantized_forward():
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    H, I, E, k, T = 1024, 512, 8, 2, 16
    w, x, logits = _weights(E, H, I), _x(T, H, 14), _logits(16, 8)
    fwd = api.MoEForward(T, H, I, E, k)
    a1, a2 = fwd.calibrate(x, logits, w)
    q = fwd(x, logits, w, a1, a2).double()
    out = _layer(T, H, I, E, k)(x, logits, w).double()
    ref, _ = R.moe(x, *R.route(logits, k), w, E, H, I)
    assert torch.linalg.norm(out - ref) <= torch.linalg.norm(q - ref)


def test_refuses_wrong_tensors():
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api, binding
    H, I, E, k, T = 256, 128, 4, 2, 3
    w, x, logits = _weights(E, H, I), _x(T, H), _logits(T, E)
    layer = _layer(T, H, I, E, k)
    ids, p = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.ones(T, k, device="cuda")
    for bad in (lambda: layer(x.float(), logits, w), lambda: layer(_x(4, H), _logits(4, E), w),
                lambda: layer(x, logits[:, :3], w), lambda: layer(x, logits.double(), w),
                lambda: layer(x, logits, _weights(5, H, I)), lambda: layer(x, logits, w, out=x[:2]),
                lambda: layer.routed(x, ids.long(), p, 0, w), lambda: layer.routed(x, ids, p[:, :1], 0, w),
                lambda: api.MoEFewTokens(33, H, I, E, k), lambda: api.MoEFewTokens(4, 300, I, E, k),
                lambda: api.MoEFewTokens(4, 16384, I, E, k)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(binding.Nvfp4Error):
        layer(x, logits, w, gate_limit=0.0)
    torch.cuda.synchronize()
