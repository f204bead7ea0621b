"""Sort, expert products and combine together, as a layer runs them, with its
gradients; and sorted rows through the NVFP4 grouped product."""
import math

import pytest

import expert_ops_reference as R
import ops_reference

pytestmark = pytest.mark.gpu


def _layer(T, H, I, E, k, model, dtype, seed=0):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    t = getattr(torch, dtype)
    x = randn(T, H).to(t)
    w13, w2 = (randn(E, 2 * I, H) / math.sqrt(H)).to(t), (randn(E, H, I) / math.sqrt(I)).to(t)
    logits = randn(T, model)
    top = logits.topk(k, dim=1)
    p = torch.softmax(top.values, 1)
    start = (model - E) // 2
    return api.ExpertFFN(w13, w2, start, 2.0, 1.5), x, top.indices.to(torch.int32), p, randn(T, H).to(t)


def _limited(z, kept, limits):
    """SwiGLU in FP64 with the limits in force where they are for the kept z: the gradient is
    defined from z as it was rounded, and a z within its rounding of a limit (the share of
    about 2^-11 of them, 2 % of the norm) may lie on either side of it."""
    import torch
    (g, u), (kg, ku) = z.chunk(2, 1), kept.double().chunk(2, 1)
    g = torch.where(kg > limits[0], limits[0], g)
    u = torch.where(ku.abs() > limits[1], limits[1] * ku.sign(), u)
    return g * torch.sigmoid(g) * u


def _reference(layer, x, ids, p, residual, order, z):
    """The layer in FP64 on leaves that take gradients, and a bound on the output's error:
    the products' (see expert_ops_reference) carried on through the layer."""
    import torch
    leaves = [v.double().requires_grad_() for v in (x, p, layer.w13, layer.w2)]
    X, P, W13, W2 = leaves
    lim = (layer.limits["gate_limit"], layer.limits["up_limit"])
    out = residual.double()
    tol = torch.zeros_like(out)
    mag = out.abs()
    for e in range(W13.shape[0]):
        t, j = (ids - layer.experts_start == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        first = int(order.offsets[e])
        h = _limited(X[t] @ W13[e].T, z[first:first + t.numel()], lim)
        y = h @ W2[e].T
        out = out.index_add(0, t, P[t, j, None] * y)
        with torch.no_grad():
            _, _, _, dh = R.linear(x[t], layer.w13[e], None, "swiglu", None, lim, x.dtype)
            top = h.abs() + dh
            dy = dh @ W2[e].abs().T + (top @ W2[e].abs().T) * ((h.shape[1] / 16 * 2 + 40) * R.U32)
            dy = R.rounded(y, dy, x.dtype)
            pt = P[t, j, None].abs()
            tol.index_add_(0, t, pt * dy)
            mag.index_add_(0, t, pt * (y.abs() + dy))
    k = ids.shape[1]
    return leaves, out, R.rounded(out.detach(), tol + mag * ((k + 1) * R.U32), x.dtype)


@pytest.mark.parametrize("T,H,I,E,k,model,dtype", [
    (1, 264, 136, 8, 2, 8, "bfloat16"), (5, 128, 72, 3, 4, 12, "float16"), (64, 520, 200, 16, 4, 32, "bfloat16"),
    (700, 256, 128, 6, 2, 6, "bfloat16"), (1500, 136, 264, 40, 3, 40, "float16")])
def test_layer_and_its_gradients(T, H, I, E, k, model, dtype):
    import torch
    layer, x, ids, p, res = _layer(T, H, I, E, k, model, dtype, seed=T)
    out, kept = layer(x, ids, p, res, keep=True)
    leaves, ref, tol = _reference(layer, x, ids, p, res, *kept[1:3])
    R.check(out, ref.detach(), tol)
    assert torch.equal(out, layer(x, ids, p, res))
    dout = torch.randn(T, H, generator=torch.Generator(device="cuda").manual_seed(9), device="cuda").to(x.dtype)
    ref.backward(dout.double())
    # Roundings on the way, half a step of the type each, as parts of the norm: y, z, h; p dout, dh, dz, the
    # rows' gradients and the result: 8; a product's norm passes each on about as large as it found it, at most
    # twice through the activation's slope (1.1) and its curvature (z's error): below 16 half steps.
    for got, leaf in zip(layer.grad(dout, kept), leaves):
        err = (got.double() - leaf.grad).norm() / leaf.grad.norm().clamp_min(1e-30)
        assert err <= 16 * R.half_step(x.dtype), float(err)


def test_layer_without_tokens_or_experts():
    import torch
    layer, x, ids, p, res = _layer(20, 128, 72, 3, 2, 3, "bfloat16")
    out, kept = layer(x[:0], ids[:0], p[:0], keep=True)
    dx, dp, d13, d2 = layer.grad(out, kept)
    assert out.shape == dx.shape == (0, 128) and dp.shape == (0, 2) and not d13.any() and not d2.any()
    ids.fill_(77)  # all held elsewhere
    out, kept = layer(x, ids, p, res, keep=True)
    assert torch.equal(out, res)
    assert all(not g.any() for g in layer.grad(res, kept))


def test_layer_in_a_graph_and_two_layers_at_once():
    import torch
    a, x, ids, p, res = _layer(300, 264, 136, 8, 2, 8, "bfloat16")
    b, xb, idb, pb, resb = _layer(40, 264, 136, 8, 2, 16, "bfloat16", seed=4)
    want, kept = a(x, ids, p, res, keep=True)
    grads = a.grad(res, kept)
    other = b(xb, idb, pb, resb)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (sa, sb):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(8):  # the calls share no scratch memory
        got, kept = a(x, ids, p, res, keep=True, stream=sa)
        more = a.grad(res, kept, stream=sa)
        gotb = b(xb, idb, pb, resb, stream=sb)
    sa.synchronize(), sb.synchronize()
    assert torch.equal(got, want) and torch.equal(gotb, other) and all(map(torch.equal, more, grads))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got, kept = a(x, ids, p, res, keep=True)
        more = a.grad(res, kept)
    ids.copy_(ids.flip(0))
    x.copy_(x.flip(0))
    g.replay()
    g.replay()
    want, kept = a(x, ids, p, res, keep=True)
    assert torch.equal(got, want) and all(map(torch.equal, more, a.grad(res, kept)))


def test_sorted_rows_through_the_nvfp4_grouped_product():
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    T, K, N, E, k = 150, 256, 384, 5, 2
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    w, w_sf, w_gs = api.quantize_expert_weights(torch.randn(E, N, K, generator=g, device="cuda").bfloat16())
    n = api.B.nvfp4_sort_tokens_capacity(T, E, k, 128)
    rows, order = api.sort_tokens(x, ids, E, align=128, out=torch.zeros(n, K, dtype=x.dtype, device="cuda"))
    a, a_sf, a_gs = api.quantize(rows)
    R128 = a.shape[0]
    d = torch.full((R128, N), 7.0, dtype=x.dtype, device="cuda")
    for e in range(E):  # a group's rows start at its own place in one buffer
        at = int(order.offsets[e])
        one = torch.tensor([at, int(order.offsets[e + 1])], dtype=torch.int32, device="cuda")
        api.grouped_gemm(a, a_sf, a_gs, w[e:e + 1], w_sf[e:e + 1], w_gs[e:e + 1], one, order.counts[e:e + 1].contiguous(),
                         N, K, d[at:], N, 0)
    A = ops_reference.decode_nvfp4(a, a_sf, a_gs, R128, K)
    for e in range(E):
        at = slice(int(order.offsets[e]), int(order.offsets[e]) + int(order.counts[e]))
        B = ops_reference.decode_nvfp4(w[e], w_sf[e], w_gs[e], N, K)
        ref, mag = A[at] @ B.T, A[at].abs() @ B.abs().T
        R.check(d[at], ref, R.rounded(ref, mag * ((K / 16 * 2 + 40) * R.U32), d.dtype))
        assert (d[at.stop:int(order.offsets[e + 1])] == 7).all()


def test_layer_next_to_the_quantized_one():
    """The layer on the weights that the quantized layer decodes to, given the same routing,
    lies within that layer's own roundings of it (activations to E2M1 twice)."""
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    T, H, I, E, k = 130, 256, 128, 6, 2
    layer, x, ids, p, _ = _layer(T, H, I, E, k, E, "bfloat16", seed=2)
    w = api.quantize_moe_weights(layer.w13, layer.w2)
    dec = lambda q, sf, gs, r, c: torch.stack([ops_reference.decode_nvfp4(q[e], sf[e], gs[e], r, c).bfloat16()
                                               for e in range(E)])
    plain = api.ExpertFFN(dec(w.w13, w.w13_sf, w.w13_gs, 2 * I, H), dec(w.w2, w.w2_sf, w.w2_gs, H, I))
    few = api.MoEFewTokens(32, H, I, E, k)
    got = torch.cat([few.routed(x[t:t + 32], ids[t:t + 32].contiguous(), p[t:t + 32].contiguous(), 0, w)
                     for t in range(0, T, 32)])
    ref = plain(x, ids, p)
    # both: bf16 outputs (half a step each); here also y (half a step), h (half a step) and the decoded weights' bf16
    # (half a step, both matrices): 6 half steps as parts of the norm, and h there to 11 bits
    err = (got.double() - ref.double()).norm() / ref.double().norm()
    assert err <= 7 * R.half_step(x.dtype), float(err)
