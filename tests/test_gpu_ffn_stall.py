"""Failure detection of the FFN-block pipelines, without a fault: with the loads
stopped after the first block, the bounded waits run out, the call reports a
device timeout and returns with nothing in flight, and the same context then
computes right answers with a clean status."""
import pytest

import ops_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture
def stall():
    from nvfp4_mixture_experts_expert_gb300 import binding as B
    B.nvfp4_device_status(reset=True)
    yield B.nvfp4_moe_set_debug_stall
    B.nvfp4_moe_set_debug_stall(0)
    B.nvfp4_device_status(reset=True)


# 9 to 32 rows over a cluster and in one CTA, tiles with K over a cluster, persistent tiles of 64 to 256 columns
@pytest.mark.parametrize("M,N,K", [(16, 512, 4096), (20, 19464, 512), (100, 512, 4096), (300, 4096, 1024), (2000, 6144, 512)])
def test_stalled_linear(stall, M, N, K):
    import time
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api, binding as B
    g = torch.Generator(device="cuda").manual_seed(M)
    a = torch.randn(M, K, generator=g, device="cuda").to(torch.float8_e4m3fn)
    w = torch.randn(N, K, generator=g, device="cuda").to(torch.float8_e4m3fn)
    sa = torch.rand(M, K // 128, generator=g, device="cuda")
    sw = torch.rand(-(-N // 128), K // 128, generator=g, device="cuda")
    want = api.fp8_linear(a, sa, w, sw, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert B.nvfp4_device_status() == B.NVFP4_OK
    start = time.time()
    stall(1000)
    api.fp8_linear(a, sa, w, sw)
    stall(0)
    torch.cuda.synchronize()
    assert time.time() - start < 30
    assert B.nvfp4_device_status(reset=True) == B.NVFP4_ERR_DEVICE_TIMEOUT
    assert torch.equal(want, api.fp8_linear(a, sa, w, sw, out_dtype=torch.float32))
    ref, mag = R.linear(a, sa, w, sw)
    assert ((want.double() - ref).abs() <= mag * ((K / 128 + 40) * R.U32) + ref.abs() * R.U32).all()
    assert B.nvfp4_device_status() == B.NVFP4_OK


@pytest.mark.parametrize("T,H,I,E,k", [(1, 4096, 2048, 8, 6), (16, 1024, 512, 16, 4), (2, 8192, 256, 4, 2)])
def test_stalled_few_token_layer(stall, T, H, I, E, k):
    import time
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api, binding as B
    g = torch.Generator(device="cuda").manual_seed(T)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    w = api.quantize_moe_weights((normal(E, 2 * I, H) * 2 / H ** 0.5).bfloat16(), (normal(E, H, I) / I ** 0.5).bfloat16())
    x, logits = normal(T, H).bfloat16(), normal(T, E)
    layer = api.MoEFewTokens(T, H, I, E, k)
    want = layer(x, logits, w)
    assert layer.status() == B.NVFP4_OK
    start = time.time()
    stall(1000)
    layer(x, logits, w)
    stall(0)
    torch.cuda.synchronize()
    assert time.time() - start < 30
    assert layer.status() == B.NVFP4_ERR_DEVICE_TIMEOUT
    assert B.nvfp4_device_status() == B.NVFP4_OK  # the word of the call's workspace alone
    assert torch.equal(want, layer(x, logits, w)) and layer.status() == B.NVFP4_OK
