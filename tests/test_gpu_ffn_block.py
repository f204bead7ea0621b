"""The FFN block: its three operators one after the other, as a decoder layer runs them."""
import pytest

import ops_reference as R

pytestmark = pytest.mark.gpu


def _block(T, H, I, E, k, seed=0):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    weights = api.quantize_moe_weights((normal(E, 2 * I, H) * 2 / H ** 0.5).bfloat16(),
                                       (normal(E, H, I) / I ** 0.5).bfloat16())
    router = api.quantize_fp8_weight(normal(E, H) * 2 / H ** 0.5)
    norm = (1 + 0.1 * normal(H)).bfloat16()
    return api.FFNBlock(T, H, I, E, k, norm, router, weights), normal(T, H).bfloat16(), normal(T, H).bfloat16() * 3


@pytest.mark.parametrize("T,H,I,E,k", [(1, 1024, 512, 16, 4), (8, 512, 256, 48, 6), (32, 1792, 640, 24, 2)])
def test_block_is_its_operators(T, H, I, E, k):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    block, x, res = _block(T, H, I, E, k)
    block.layer.workspace.fill_(0xFF)
    out, s = block(x, res)
    q, scales, y, s1 = api.add_rms_norm_fp8(x, res, block.norm_weight)
    logits = api.fp8_linear(q, scales, *block.router, out_dtype=torch.float32)
    assert torch.equal(s, s1) and torch.equal(s, (x.float() + res.float()).bfloat16())
    ref, mag = R.linear(q, scales, *block.router)
    assert ((logits.double() - ref).abs() <= mag * ((H / 128 + 40) * R.U32) + ref.abs() * R.U32).all()
    ids, p = R.route(logits, k)
    ref, tol = R.moe(y, ids, p, block.weights, E, H, I)
    tol = tol + (ref.abs() + tol) * R.BF16
    assert ((out.double() - ref).abs() <= tol).all()
    assert block.layer.status() == 0


def test_two_blocks_in_a_graph_on_another_stream():
    import torch
    first, x, res = _block(8, 512, 256, 16, 4)
    second, _, _ = _block(8, 512, 256, 16, 4, seed=1)

    def run(**kw):
        y, s = first(x, res, **kw)
        return second(y, s, **kw)
    want = [t.clone() for t in run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = run()
        for _ in range(3):
            graph.replay()
        side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    torch.cuda.current_stream().wait_stream(side)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = run(stream=other)
    other.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
