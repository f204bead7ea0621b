"""Tokens sorted into slots of 128 rows through quantize, grouped_gemm and combine_tokens
without the host looking at the order, as the README has it."""
import dataclasses

import numpy as np
import pytest

import expert_ops_reference as R
import ops_reference

pytestmark = pytest.mark.gpu


def _through(api, x, ids, p, start, w, w_sf, w_gs, N, given=None):
    """(rows, order, codes, scales, global scale, D [E, S, N], combined)."""
    import torch
    T, K = x.shape
    E = w.shape[0]
    n = api.B.nvfp4_sort_tokens_capacity(T, E, ids.shape[1], 128)
    # quantize takes its scale from all rows: those behind the last expert's, which are not written, are zeros
    rows, order = api.sort_tokens(x, ids, E, start, align=128, out=torch.zeros(n, K, dtype=x.dtype, device=x.device))
    a, a_sf, a_gs = api.quantize(rows, gs=given)
    S = max(T, -(-n // E))  # rows of an expert in D, at most T of them used; the order's n rows in all
    D = torch.full((E, S, N), float("nan"), dtype=torch.bfloat16, device=x.device)
    api.grouped_gemm(a, a_sf, a_gs.expand(E).contiguous(), w, w_sf, w_gs, order.offsets, order.counts, N, K, D, N, S * N)
    # row i of expert e is row e * S + i of D
    shift = torch.arange(E, dtype=torch.int32, device=x.device) * S - order.offsets[:-1]
    inverse = torch.where(order.inverse < 0, order.inverse, order.inverse + shift[(ids - start).clamp(0, E - 1)])
    out = api.combine_tokens(D.view(-1, N), p, dataclasses.replace(order, inverse=inverse))
    return rows, order, a, a_sf, a_gs, D, out


@pytest.mark.parametrize("T,K,N,E,model,k", [(150, 256, 384, 5, 9, 2), (1, 128, 128, 8, 8, 8), (128, 64, 256, 8, 8, 7),
                                             (700, 512, 640, 3, 12, 4)])
def test_slots_through_the_grouped_product_and_back(T, K, N, E, model, k):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    start = (model - E) // 2
    top = torch.rand(T, model, generator=g, device="cuda").topk(k, dim=1)
    ids, p = top.indices.to(torch.int32), torch.softmax(top.values, 1)
    w, w_sf, w_gs = api.quantize_expert_weights(torch.randn(E, N, K, generator=g, device="cuda").bfloat16())
    for given in (None, torch.full((1,), 500.0, device="cuda")):
        rows, order, a, a_sf, a_gs, D, out = _through(api, x, ids, p, start, w, w_sf, w_gs, N, given)
        if given is None:  # of the tokens that have an expert here, and of nothing else
            here = ((ids >= start) & (ids < start + E)).any(1)
            amax = float(x[here].abs().max()) if here.any() else 0.0
            # one IEEE division, as on the host (torch's 2688 / tensor on the GPU rounds a reciprocal before the product)
            assert float(a_gs) == (float(np.float32(2688) / np.float32(amax)) if amax > 0 else 1.0)
        A = ops_reference.decode_nvfp4(a, a_sf, a_gs, a.shape[0], K)
        counts, first = order.counts.tolist(), order.offsets.tolist()
        ref = torch.zeros(T, N, dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(ref)
        for e in range(E):
            B = ops_reference.decode_nvfp4(w[e], w_sf[e], w_gs[e], N, K)
            at = slice(first[e], first[e] + counts[e])
            want, size = A[at] @ B.T, A[at].abs() @ B.abs().T
            R.check(D[e, :counts[e]], want, R.rounded(want, size * ((K / 16 * 2 + 40) * R.U32), D.dtype))
            assert D[e, counts[e]:].isnan().all()
            f = order.source[at].long()
            v = p.view(-1)[f, None].double() * D[e, :counts[e]].double()
            ref.index_add_(0, f // k, v)
            mag.index_add_(0, f // k, v.abs())
        R.check(out, ref, R.rounded(ref, mag * ((k + 1) * R.U32), out.dtype))


def test_slots_in_a_graph():
    """No step of it synchronises: the whole is captured, and replayed with other routing."""
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    T, K, N, E, k = 200, 128, 256, 6, 2
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    route = lambda: torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)
    ids, p = route(), torch.rand(T, k, generator=g, device="cuda")
    w = api.quantize_expert_weights(torch.randn(E, N, K, generator=g, device="cuda").bfloat16())
    _through(api, x, ids, p, 0, *w, N)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _through(api, x, ids, p, 0, *w, N)[-1]
    for _ in range(2):
        ids.copy_(route())
        x.mul_(1.5)
        graph.replay()
        assert torch.equal(out, _through(api, x, ids, p, 0, *w, N)[-1])
