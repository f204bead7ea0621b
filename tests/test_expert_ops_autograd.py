"""The operators with gradient calls of their own refuse tensors that autograd follows
instead of dropping their gradients (on the host, before anything else is checked)."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def api():
    from nvfp4_mixture_experts_expert_gb300 import _build
    _build.build()
    from nvfp4_mixture_experts_expert_gb300 import api
    return api


def _calls(api):
    """Each call as (function of its tensors, the tensors): on the CPU, where no call gets any further."""
    bf16 = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    order = api.TokenOrder(i32(3), i32(2), i32(8), i32(4, 2))
    x, w, b, we, p = bf16(8, 16), bf16(16, 16), bf16(16), bf16(2, 16, 16), torch.zeros(4, 2)
    return {
        "sort": (lambda x: api.sort_tokens(x, i32(8, 1), 2), [x]),
        "sort_grad": (lambda d: api.sort_tokens_grad(d, order), [x]),
        "combine": (lambda r, p, res: api.combine_tokens(r, p, order, res), [x, p, bf16(4, 16)]),
        "combine_grad": (lambda d, r, p: api.combine_tokens_grad(d, r, p, order), [bf16(4, 16), x, p]),
        "linear": (lambda x, w, b, res: api.linear(x, w, b, residual=res), [x, w, b, x.clone()]),
        "linear_grad": (lambda d, x, w, z: api.linear_grad(d, x, w, z, "silu"), [x.clone(), x, w, x.clone()]),
        "expert_linear": (lambda x, w: api.expert_linear(x, w, order), [x, we]),
        "expert_linear_grad": (lambda d, x, w: api.expert_linear_grad(d, x, w, order), [x.clone(), x, we]),
        "layer": (lambda x, p: api.ExpertFFN(bf16(2, 32, 16), we)(x, i32(8, 1), p), [x, p]),
    }


@pytest.mark.parametrize("name", ["sort", "sort_grad", "combine", "combine_grad", "linear", "linear_grad",
                                  "expert_linear", "expert_linear_grad", "layer"])
def test_a_tensor_that_requires_grad_is_refused(api, name):
    call, tensors = _calls(api)[name]
    with pytest.raises(ValueError, match="CUDA"):  # the next check: no tensor is on a GPU here
        call(*tensors)
    for i in range(len(tensors) if name != "layer" else 1):
        for leaf in (True, False):
            t = tensors[i].clone().requires_grad_()
            args = [*tensors[:i], t if leaf else 2 * t, *tensors[i + 1:]]
            with pytest.raises(ValueError, match="no_grad"):
                call(*args)
            for mode in (torch.no_grad, torch.inference_mode):
                with mode(), pytest.raises(ValueError, match="CUDA"):
                    call(*args)


def test_an_autograd_function_of_the_calls_is_not_refused(api):
    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            with pytest.raises(ValueError, match="CUDA"):
                api.linear(x, w)
            ctx.save_for_backward(x, w)
            return x @ w.t()

        @staticmethod
        def backward(ctx, grad):
            x, w = ctx.saved_tensors
            with pytest.raises(ValueError, match="CUDA"):
                api.linear_grad(grad, x, w)
            return grad @ w, grad.t() @ x

    x, w = (torch.ones(8, 16, dtype=torch.bfloat16, requires_grad=True) for _ in range(2))
    Linear.apply(x, w).sum().backward()
    assert x.grad is not None and w.grad is not None
