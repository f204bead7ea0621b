"""The token sort in one launch up to its limit of 1024 assignments, and just above it in
two: order, rows and gradients as everywhere else, and as the other path gives them."""
import pytest

import test_gpu_token_sort as S

pytestmark = pytest.mark.gpu

# (T, H, E, k, experts of the model, align): 500 to 1024 assignments in one launch (a whole table of ids, as many
# blocks as assignments, 32 experts a token, blocks of pad rows for 256 experts), 1025 to 1040 in two
CASES = [(100, 264, 9, 5, 18, 1), (33, 40, 48, 30, 48, 16), (1024, 16, 3, 1, 3, 1), (1024, 24, 256, 1, 300, 16),
         (32, 72, 256, 32, 256, 128), (128, 72, 7, 8, 7, 8), (64, 1032, 12, 16, 24, 128),
         (1025, 16, 3, 1, 3, 1), (129, 72, 7, 8, 7, 8), (41, 72, 256, 25, 256, 128)]


@pytest.mark.parametrize("T,H,E,k,model,align", CASES)
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_sort_and_combine_with_gradients(T, H, E, k, model, align, dtype):
    S.test_sort_and_its_gradient(T, H, E, k, model, align, dtype)
    S.test_combine_and_its_gradient(T, H, E, k, model, align, dtype, True)


@pytest.mark.parametrize("align", [1, 128])
def test_both_paths_give_one_order(align):
    """The first 1024 of 1025 assignments, of which the last belongs to no expert here."""
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    ids = S._ids(1025, 1, 40, seed=3)
    ids[-1] = 99
    x = S._rows(1025, 64, "bfloat16")
    few_rows, few = api.sort_tokens(x[:1024], ids[:1024].cuda(), 33, 4, align)
    rows, order = api.sort_tokens(x, ids.cuda(), 33, 4, align)
    n = int(order.offsets[-1])
    for name in ("offsets", "counts"):
        assert torch.equal(getattr(few, name), getattr(order, name))
    assert torch.equal(few.inverse, order.inverse[:1024]) and int(order.inverse[-1]) == -1
    assert torch.equal(few.source[:n], order.source[:n]) and torch.equal(few_rows[:n], rows[:n])
