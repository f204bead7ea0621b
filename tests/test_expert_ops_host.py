"""The token sort, combine and linear calls check their arguments on the host before
anything is launched (no device call is made here)."""
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


INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
NAN, INF = float("nan"), float("inf")

SORT = dict(x=16, ld_x=64, type=0, topk_ids=4, experts_start=0, T=8, H=64, E=4, top_k=2, align=1, capacity=16, rows=32,
            ld_rows=64, offsets=8, counts=12, source=16, inverse=20)


@pytest.mark.parametrize("change,code", [
    (dict(type=3), INVALID), (dict(type=-1), INVALID), (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID),
    (dict(H=0), UNSUPPORTED), (dict(H=60), UNSUPPORTED), (dict(H=1 << 25), UNSUPPORTED), (dict(E=0), UNSUPPORTED),
    (dict(E=257), UNSUPPORTED), (dict(top_k=0), UNSUPPORTED), (dict(top_k=33), UNSUPPORTED), (dict(align=0), INVALID),
    (dict(align=24), INVALID), (dict(align=256), INVALID), (dict(capacity=15), INVALID),
    (dict(align=16, capacity=75), INVALID), (dict(capacity=1 << 31), INVALID), (dict(T=1 << 30, top_k=32), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(topk_ids=None), INVALID), (dict(offsets=None), INVALID), (dict(counts=None), INVALID),
    (dict(source=None), INVALID), (dict(inverse=None), INVALID), (dict(ld_x=56), INVALID), (dict(ld_x=68), INVALID),
    (dict(ld_rows=0), INVALID), (dict(x=8), INVALID), (dict(rows=40), INVALID), (dict(topk_ids=2), INVALID),
    (dict(source=18), INVALID),
])
def test_sort_refusals(B, change, code):
    _refused(B, B.nvfp4_sort_tokens, SORT, change, code)


def test_sort_capacity(B):
    size = B.nvfp4_sort_tokens_capacity
    assert size(8, 4, 2) == 16 and size(8, 4, 2, 128) == 16 + 4 * 127 and size(1, 48, 6, 128) == 6 * 128
    assert size(0, 4, 2) == 0
    for bad in ((-1, 4, 2, 1), (8, 0, 2, 1), (8, 257, 2, 1), (8, 4, 0, 1), (8, 4, 33, 1), (8, 4, 2, 3), (8, 4, 2, 256),
                (1 << 31, 4, 1, 1), (1 << 27, 4, 16, 1)):
        assert size(*bad) == 0


COMBINE = dict(rows=16, ld_rows=64, type=1, weights=4, inverse=8, residual=32, ld_residual=64, T=8, H=64, top_k=2,
               out=48, ld_out=64)


@pytest.mark.parametrize("change,code", [
    (dict(type=7), INVALID), (dict(T=-1), INVALID), (dict(H=4), UNSUPPORTED), (dict(top_k=33), UNSUPPORTED),
    (dict(rows=None), INVALID), (dict(weights=None), INVALID), (dict(inverse=None), INVALID), (dict(out=None), INVALID),
    (dict(ld_rows=60), INVALID), (dict(ld_residual=66), INVALID), (dict(ld_out=8), INVALID),
    (dict(residual=48, ld_residual=72), INVALID), (dict(rows=20), INVALID), (dict(residual=36), INVALID),
    (dict(weights=6), INVALID),
])
def test_combine_refusals(B, change, code):
    _refused(B, B.nvfp4_combine_tokens, COMBINE, change, code)


GRAD = dict(dout=16, ld_dout=64, rows=32, ld_rows=64, type=0, weights=4, offsets=8, counts=12, inverse=16, T=8, H=64,
            E=4, top_k=2, align=1, drows=48, ld_drows=64, dweights=20)


@pytest.mark.parametrize("change,code", [
    (dict(E=0), UNSUPPORTED), (dict(E=300), UNSUPPORTED), (dict(top_k=0), UNSUPPORTED), (dict(align=6), INVALID),
    (dict(H=12), UNSUPPORTED), (dict(dout=None), INVALID), (dict(counts=None), INVALID), (dict(dweights=None), INVALID),
    (dict(ld_dout=56), INVALID), (dict(ld_drows=65), INVALID), (dict(drows=50), INVALID), (dict(dweights=22), INVALID),
])
def test_combine_grad_refusals(B, change, code):
    _refused(B, B.nvfp4_combine_tokens_grad, GRAD, change, code)


SHAPE = dict(M=4, N=64, K=128, type=0)
LINEAR = dict(x=16, ld_x=128, w=32, bias=48, bias_type=0, residual=64, ld_residual=64, preact=80, out=96, ld_out=64,
              out_type=0)
LGRAD = dict(dy=16, ld_dy=64, x=32, ld_x=128, w=48, preact=64, dx=80, ld_dx=128, dw=96, dbias=100, workspace=256,
             workspace_bytes=1 << 30)
SHAPES = [
    (dict(M=-1), INVALID), (dict(M=(1 << 22) + 1), INVALID), (dict(N=0), INVALID), (dict(N=60), INVALID),
    (dict(N=131080), INVALID), (dict(K=0), INVALID), (dict(K=12), INVALID), (dict(K=131080), INVALID),
    (dict(type=2), INVALID), (dict(activation=6), INVALID), (dict(activation=-1), INVALID),
    (dict(activation=5, gate_limit=0.0), INVALID), (dict(activation=5, up_limit=NAN), INVALID),
    (dict(groups=-1), UNSUPPORTED), (dict(groups=257, offsets=4, counts=4), UNSUPPORTED), (dict(groups=2), INVALID),
    (dict(groups=2, offsets=4), INVALID), (dict(groups=2, offsets=4, counts=6), INVALID),
]


@pytest.mark.parametrize("change,code", SHAPES)
def test_linear_shape_refusals(B, change, code):
    shape = B.linear_shape(**{**SHAPE, **change})
    _refused(B, B.nvfp4_linear, dict(LINEAR, shape=shape), {}, code)
    _refused(B, B.nvfp4_linear_grad, dict(LGRAD, shape=shape), {}, code)
    assert B.nvfp4_linear_grad_workspace_size(shape) == 0


@pytest.mark.parametrize("change", [
    dict(x=None), dict(w=None), dict(out=None), dict(ld_x=120), dict(ld_x=132), dict(ld_out=56), dict(ld_out=68),
    dict(ld_residual=0), dict(bias_type=1), dict(out_type=1), dict(out_type=5), dict(x=24), dict(w=40), dict(bias=52),
    dict(residual=72), dict(preact=88), dict(out=100), dict(residual=96, ld_residual=72),
    dict(residual=96, out_type=2), dict(shape=None),
])
def test_linear_refusals(B, change):
    if "shape" in change:
        import ctypes
        assert B._linear(ctypes.POINTER(B.LinearShape)(), 16, 128, 32, None, 0, None, 0, None, 96, 64, 0, None) == INVALID
        return
    _refused(B, B.nvfp4_linear, dict(LINEAR, shape=B.linear_shape(**SHAPE)), change, INVALID)


@pytest.mark.parametrize("change,code", [
    (dict(dy=None), INVALID), (dict(preact=None), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID),
    (dict(ld_dy=60), INVALID), (dict(ld_x=0), INVALID), (dict(ld_dx=132), INVALID), (dict(dy=24), INVALID),
    (dict(dw=100), INVALID), (dict(dbias=102), INVALID), (dict(workspace=None), WORKSPACE),
    (dict(workspace_bytes=255), WORKSPACE), (dict(workspace=128), INVALID),
])
def test_linear_grad_refusals(B, change, code):
    _refused(B, B.nvfp4_linear_grad, dict(LGRAD, shape=B.linear_shape(**SHAPE, activation=2)), change, code)


def test_linear_grad_workspace_size(B):
    size = B.nvfp4_linear_grad_workspace_size
    plain, silu, pairs = (B.linear_shape(**{**SHAPE, "M": 1000}, activation=a) for a in (0, 2, 5))
    assert size(plain) == 0 and size(plain, dbias=True) >= 16 * 64 * 4
    assert size(silu) >= 1000 * 64 * 2 and size(pairs) >= 1000 * 128 * 2 and size(silu, products=False) == 0
    assert size(B.linear_shape(**{**SHAPE, "M": 0}, activation=2), dbias=True) == 0


def test_no_work_is_not_an_error(B):
    B.nvfp4_combine_tokens(**{**COMBINE, "T": 0, "rows": None}, stream=0)
    B.nvfp4_combine_tokens_grad(**{**GRAD, "T": 0, "dout": None}, stream=0)
    B.nvfp4_sort_tokens_grad(None, 64, 0, None, 0, 64, 2, None, 64, stream=0)
    B.nvfp4_linear(B.linear_shape(**{**SHAPE, "M": 0}), **{**LINEAR, "x": None}, stream=0)


def test_activation_names():
    torch = pytest.importorskip("torch")
    from nvfp4_mixture_experts_expert_gb300 import api
    x = torch.zeros(2, 8, dtype=torch.bfloat16)
    for bad in ("tanh", 3, ["relu"]):
        with pytest.raises(ValueError):
            api.linear(x, x, activation=bad)
    with pytest.raises(ValueError):
        api.linear(x, x, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        api.linear(x, x)  # not on a GPU
