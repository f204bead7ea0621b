"""The FFN-block operators check their arguments on the host before anything is
launched (no device call is made here)."""
import pytest


@pytest.fixture(scope="module")
def B():
    from nvfp4_mixture_experts_expert_gb300 import _build
    _build.build()
    from nvfp4_mixture_experts_expert_gb300 import binding
    return binding


def _refused(B, call, kw, change, code):
    with pytest.raises(B.Nvfp4Error) as ei:
        call(**{**kw, **change}, stream=0)
    assert ei.value.status == code and B.nvfp4_last_error()


NORM = dict(x=16, ld_x=256, residual=32, ld_residual=256, weight=48, weight_is_f32=0, T=4, H=256, eps=1e-6,
            residual_out=64, ld_residual_out=256, normed=80, q=96, scales=112)
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID), (dict(H=0), UNSUPPORTED), (dict(H=248), UNSUPPORTED),
    (dict(H=32784, ld_x=32784), UNSUPPORTED), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(residual_out=None, normed=None, q=None, scales=None), INVALID), (dict(scales=None), INVALID),
    (dict(q=None), INVALID), (dict(x=None), INVALID), (dict(weight=None), INVALID), (dict(ld_x=248), INVALID),
    (dict(ld_x=260), INVALID), (dict(ld_residual=0), INVALID), (dict(ld_residual_out=8), INVALID),
    (dict(x=24), INVALID), (dict(q=100), INVALID), (dict(scales=114), INVALID),
    (dict(residual_out=32, ld_residual_out=264), INVALID), (dict(residual_out=16, ld_residual_out=264), INVALID),
])
def test_norm_refusals(B, change, code):
    _refused(B, B.nvfp4_add_rmsnorm_fp8, NORM, change, code)


LINEAR = dict(a=16, ld_a=256, a_scale=20, w=32, w_scale=36, M=4, N=64, K=256, out=48, ld_out=64, out_is_f32=0)


@pytest.mark.parametrize("change", [
    dict(M=-1), dict(M=(1 << 20) + 1), dict(N=0), dict(N=60), dict(N=1 << 21), dict(K=0), dict(K=250), dict(K=1 << 21),
    dict(ld_a=240), dict(ld_a=264), dict(ld_out=56), dict(ld_out=68), dict(a=None), dict(w=None), dict(a_scale=None),
    dict(w_scale=None), dict(out=None), dict(a=20), dict(w=40), dict(out=52), dict(a_scale=18), dict(w_scale=33),
])
def test_linear_refusals(B, change):
    _refused(B, B.nvfp4_fp8_linear, LINEAR, change, INVALID)


WS = dict(w13=16, w13_sf=32, w13_gs=48, w2=64, w2_sf=80, w2_gs=96, gate_limit=10.0, up_limit=10.0, workspace=256,
          workspace_bytes=1 << 30, out=112)
FEW = dict(hidden=16, ld_hidden=256, router_logits=32, T=4, H=256, I=128, E=8, top_k=2, **WS)
COMMON = [
    (dict(T=33), UNSUPPORTED), (dict(T=-1), INVALID), (dict(top_k=0), INVALID), (dict(top_k=9), INVALID),
    (dict(H=128, ld_hidden=256), UNSUPPORTED), (dict(H=8448, ld_hidden=8448), UNSUPPORTED), (dict(I=64), UNSUPPORTED),
    (dict(I=8320), UNSUPPORTED), (dict(E=0), UNSUPPORTED), (dict(E=257), UNSUPPORTED), (dict(gate_limit=0.0), INVALID),
    (dict(up_limit=-1.0), INVALID), (dict(up_limit=float("nan")), INVALID), (dict(hidden=None), INVALID),
    (dict(w2_gs=None), INVALID), (dict(out=None), INVALID), (dict(ld_hidden=252), INVALID),
    (dict(ld_hidden=260), INVALID), (dict(w13=20), INVALID), (dict(out=120), INVALID),
    (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=100), WORKSPACE), (dict(workspace=128), INVALID),
]


@pytest.mark.parametrize("change,code", COMMON + [
    (dict(router_logits=None), INVALID), (dict(router_logits=34), INVALID), (dict(E=2, top_k=3), INVALID)])
def test_few_tokens_refusals(B, change, code):
    _refused(B, B.nvfp4_moe_few_tokens, FEW, change, code)


@pytest.mark.parametrize("change,code", COMMON + [
    (dict(topk_ids=None), INVALID), (dict(topk_weights=None), INVALID), (dict(topk_ids=33), INVALID)])
def test_few_tokens_routed_refusals(B, change, code):
    kw = {k: v for k, v in FEW.items() if k != "router_logits"}
    _refused(B, B.nvfp4_moe_few_tokens_routed, dict(kw, topk_ids=32, topk_weights=36, experts_start=0), change, code)


def test_few_tokens_workspace_size(B):
    size = B.nvfp4_moe_few_tokens_workspace_size
    assert size(32, 4096, 2048, 48, 6) >= 32 * 6 * (4096 + 2048) * 4
    assert size(1, 256, 128, 1, 1) < size(2, 256, 128, 1, 1)
    for bad in ((33, 256, 128, 8, 2), (1, 300, 128, 8, 2), (1, 256, 100, 8, 2), (1, 256, 128, 0, 2),
                (1, 256, 128, 8, 9), (-1, 256, 128, 8, 2), (1, 8448, 128, 8, 2)):
        assert size(*bad) == 0


def test_no_work_is_not_an_error(B):
    B.nvfp4_add_rmsnorm_fp8(**{**NORM, "T": 0, "x": None}, stream=0)
    B.nvfp4_fp8_linear(**{**LINEAR, "M": 0, "a": None}, stream=0)
    B.nvfp4_moe_few_tokens(**{**FEW, "T": 0, "hidden": None}, stream=0)


def test_quantize_fp8_weight():
    torch = pytest.importorskip("torch")
    from nvfp4_mixture_experts_expert_gb300 import api
    w = torch.randn(200, 272, generator=torch.Generator().manual_seed(0))
    w[:128, :128] = 0
    codes, scale = api.quantize_fp8_weight(w)
    assert codes.shape == w.shape and codes.dtype is torch.float8_e4m3fn and scale.shape == (2, 3)
    for i in range(2):
        for j in range(3):
            part = w[128 * i:128 * i + 128, 128 * j:128 * j + 128]
            top = max(float(part.abs().max()), 2.0 ** -40)
            assert abs(float(scale[i, j]) * 448 / top - 1) < 1e-6
            err = (codes[128 * i:128 * i + 128, 128 * j:128 * j + 128].float() * scale[i, j] - part).abs()
            # half a unit of three mantissa bits, or of the subnormals 2^-9 apart
            assert (err <= torch.maximum(part.abs() / 16, scale[i, j] * 2.0 ** -10) * (1 + 1e-5)).all()
