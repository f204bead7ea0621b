"""Tokens sorted by expert and back against the definitions in 64 bits."""
import pytest

import expert_ops_reference as R

pytestmark = pytest.mark.gpu

TYPES = ["bfloat16", "float16", "float32"]


def _ids(T, k, n, seed=0, low=0):
    import torch
    g = torch.Generator().manual_seed(seed)
    return torch.randint(low, n, (T, k), generator=g, dtype=torch.int32)  # an expert may come twice


def _rows(n, H, dtype, seed=0, pad=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, H + pad, generator=g, device="cuda").to(getattr(torch, dtype))[:, :H]


def _same_order(order, ids, E, start, align):
    import torch
    for got, want in zip((order.offsets, order.counts, order.source, order.inverse), R.order(ids, E, start, align)):
        assert torch.equal(got.cpu(), want)


# (T, H, E, k, experts of the model, align): one launch up to 2048 assignments, two above
CASES = [(1, 8, 1, 1, 1, 1), (1, 4096, 32, 6, 32, 1), (3, 264, 5, 2, 9, 16), (37, 1000, 48, 8, 48, 128),
         (256, 72, 7, 8, 7, 8), (257, 72, 7, 8, 7, 8), (300, 640, 256, 32, 300, 1), (2048, 16, 3, 1, 3, 128),
         (2049, 16, 3, 1, 3, 128), (4099, 136, 48, 6, 96, 64), (9000, 32, 256, 3, 256, 2), (1001, 3584, 12, 4, 24, 1)]


@pytest.mark.parametrize("T,H,E,k,model,align", CASES)
@pytest.mark.parametrize("dtype", TYPES)
def test_sort_and_its_gradient(T, H, E, k, model, align, dtype):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    start = (model - E) // 2
    ids = _ids(T, k, model, seed=T)
    x = _rows(T, H, dtype, seed=T, pad=8)
    size = T * k + min(T * k, E) * (align - 1)
    out = torch.full((size, H), 7.0, dtype=x.dtype, device="cuda")
    rows, order = api.sort_tokens(x, ids.cuda(), E, start, align, out=out)
    assert rows is out or rows.data_ptr() == out.data_ptr()
    _same_order(order, ids, E, start, align)
    src = order.source.long()
    inside = torch.arange(size, device="cuda") < order.offsets[-1]
    want = torch.where((src >= 0)[:, None], x[(src.clamp(min=0) // k)], torch.zeros_like(out))
    assert torch.equal(rows, torch.where(inside[:, None], want, torch.full_like(out, 7.0)))
    assert api.sort_tokens(x, ids.cuda(), E, start, align)[0].shape == rows.shape
    d = _rows(size, H, dtype, seed=T + 1, pad=16)
    dx = api.sort_tokens_grad(d, order)
    ref, mag = R.combine(d, None, order.inverse)
    R.check(dx, ref, R.rounded(ref, mag * (k * R.U32), dx.dtype))


@pytest.mark.parametrize("T,H,E,k,model,align", CASES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("residual", [False, True])
def test_combine_and_its_gradient(T, H, E, k, model, align, dtype, residual):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    start = (model - E) // 2
    ids = _ids(T, k, model, seed=T + 1)
    x = _rows(T, H, dtype)
    rows, order = api.sort_tokens(x, ids.cuda(), E, start, align)
    rows = _rows(rows.shape[0], H, dtype, seed=3, pad=8)
    src = order.source >= 0
    rows[~src] = float("nan")  # no row that no assignment has is read
    p = torch.randn(T, k, device="cuda")
    res = _rows(T, H, dtype, seed=4, pad=8) if residual else None
    out = api.combine_tokens(rows, p, order, residual=res)
    clean = torch.where(src[:, None], rows, torch.zeros_like(rows))
    ref, mag = R.combine(clean, p, order.inverse, res)
    R.check(out, ref, R.rounded(ref, mag * ((k + 1) * R.U32), out.dtype))
    dout = _rows(T, H, dtype, seed=5, pad=8)
    buf = torch.full(rows.shape, 7.0, dtype=rows.dtype, device="cuda")
    drows, dp = api.combine_tokens_grad(dout, rows, p, order, out=buf)
    f = order.source.clamp(min=0).long()
    want = torch.where(src[:, None], p.view(-1)[f, None].double() * dout[f // k].double(), 0.0)
    inside = torch.arange(rows.shape[0], device="cuda") < order.offsets[-1]
    want = torch.where(inside[:, None], want, 7.0)
    R.check(drows, want, torch.where(src[:, None], R.rounded(want, want.abs() * R.U32, drows.dtype), 0.0))
    v = clean.double()[order.inverse.clamp(min=0).long()] * dout.double()[:, None, :]
    v = torch.where((order.inverse >= 0)[..., None], v, 0.0)
    R.check(dp, v.sum(2), v.abs().sum(2) * ((H / 64 + 24) * R.U32))


def test_no_local_expert_and_no_tokens():
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    for T in (5, 3000):
        x = _rows(T, 64, "bfloat16")
        ids = torch.full((T, 2), -5, dtype=torch.int32, device="cuda")
        ids[:, 1] = 2 ** 31 - 1
        out = torch.full((2 * T, 64), 3.0, dtype=x.dtype, device="cuda")
        rows, order = api.sort_tokens(x, ids, 4, 7, out=out)
        assert (rows == 3).all() and not order.offsets.any() and not order.counts.any()
        assert (order.source == -1).all() and (order.inverse == -1).all()
        p = torch.ones(T, 2, device="cuda")
        assert not api.combine_tokens(rows, p, order).any() and not api.sort_tokens_grad(rows, order).any()
        assert torch.equal(api.combine_tokens(rows, p, order, residual=x), x)
        drows, dp = api.combine_tokens_grad(x, rows, p, order, out=out)
        assert (drows == 3).all() and not dp.any()
    x = _rows(0, 64, "bfloat16")
    rows, order = api.sort_tokens(x, torch.empty(0, 2, dtype=torch.int32, device="cuda"), 4)
    assert rows.shape == (0, 64) and not order.offsets.any() and not order.counts.any()
    p = torch.empty(0, 2, device="cuda")
    assert api.combine_tokens(rows, p, order).shape == (0, 64)
    assert api.combine_tokens_grad(x, rows, p, order)[1].shape == (0, 2)


def test_offsets_beyond_32_bits():
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    T, H, E = 300000, 4096, 7
    x = torch.randn(T, H, dtype=torch.bfloat16, device="cuda")
    ids = _ids(T, 2, E).cuda()
    rows, order = api.sort_tokens(x, ids, E)  # 2.5e9 elements
    src = order.source.long() // 2
    assert torch.equal(order.source.sort().values, torch.arange(2 * T, dtype=torch.int32, device="cuda"))
    for s in (0, 524200, 2 * T - 1000):
        assert torch.equal(rows[s:s + 1000], x[src[s:s + 1000]])
    p = torch.rand(T, 2, device="cuda")
    out = api.combine_tokens(rows, p, order)
    dx = api.sort_tokens_grad(rows, order)
    drows, dp = api.combine_tokens_grad(x, rows, p, order)
    for at in (slice(0, 500), slice(T - 500, T)):
        v = rows[order.inverse[at].long()].double()
        w = p[at, :, None].double()
        R.check(out[at], (w * v).sum(1), R.rounded((w * v).sum(1), (w * v).abs().sum(1) * (3 * R.U32), out.dtype))
        R.check(dx[at], v.sum(1), R.rounded(v.sum(1), v.abs().sum(1) * (2 * R.U32), out.dtype))
        want = w * x[at, None, :].double()
        R.check(drows[order.inverse[at].long()], want, R.rounded(want, want.abs() * R.U32, out.dtype))
        dot = v * x[at, None, :].double()
        R.check(dp[at], dot.sum(2), dot.abs().sum(2) * ((H / 64 + 24) * R.U32))


def test_non_finite_rows_stay_their_own():
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    x = _rows(40, 128, "bfloat16")
    ids = _ids(40, 3, 6).cuda()
    rows, order = api.sort_tokens(x, ids, 6)
    p = torch.rand(40, 3, device="cuda")
    want = api.combine_tokens(rows, p, order)
    x[7] = float("nan")
    x[9, 5] = float("inf")
    rows, order = api.sort_tokens(x, ids, 6)
    got = api.combine_tokens(rows, p, order)
    other = torch.ones(40, dtype=torch.bool, device="cuda")
    other[7] = other[9] = False
    assert torch.equal(got[other], want[other]) and got[7].isnan().all() and got[9, 5].isinf()


def test_residual_in_place_other_stream_and_graph():
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    x, res = _rows(600, 256, "bfloat16"), _rows(600, 256, "bfloat16", seed=2)
    ids, p = _ids(600, 4, 9).cuda(), torch.rand(600, 4, device="cuda")
    rows, order = api.sort_tokens(x, ids, 9, align=16)
    want = api.combine_tokens(rows, p, order, residual=res)
    mine = res.clone()
    assert api.combine_tokens(rows, p, order, residual=mine, out=mine).data_ptr() == mine.data_ptr()
    assert torch.equal(mine, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r2, o2 = api.sort_tokens(x, ids, 9, align=16, stream=s)
    got = api.combine_tokens(r2, p, o2, residual=res, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r3, o3 = api.sort_tokens(x, ids, 9, align=16)
        out = api.combine_tokens(r3, p, o3, residual=res)
    x.copy_(_rows(600, 256, "bfloat16", seed=8))
    ids.copy_(_ids(600, 4, 9, seed=8))
    for _ in range(2):
        g.replay()
    rows, order = api.sort_tokens(x, ids, 9, align=16)
    assert torch.equal(out, api.combine_tokens(rows, p, order, residual=res))
    assert torch.equal(o3.source, order.source)


def test_refusals_of_the_python_calls():
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api, binding
    x, ids = _rows(8, 64, "bfloat16"), _ids(8, 2, 4).cuda()
    rows, order = api.sort_tokens(x, ids, 4)
    p = torch.ones(8, 2, device="cuda")
    for call in (lambda: api.sort_tokens(x.cpu(), ids, 4), lambda: api.sort_tokens(x.double(), ids, 4),
                 lambda: api.sort_tokens(x, ids.long(), 4), lambda: api.sort_tokens(x, ids[:7], 4),
                 lambda: api.sort_tokens(x, ids, 4, out=rows[:3]), lambda: api.sort_tokens(x.t(), ids, 4),
                 lambda: api.sort_tokens(x, ids, 4, 1 << 40), lambda: api.combine_tokens(rows, p.double(), order),
                 lambda: api.combine_tokens(rows, p[:4], order), lambda: api.combine_tokens(rows, p, order, residual=x[:3]),
                 lambda: api.combine_tokens(rows, p, order, out=x.float()),
                 lambda: api.combine_tokens_grad(x.half(), rows, p, order),
                 lambda: api.sort_tokens_grad(rows[0], order)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: api.sort_tokens(x, ids, 0), lambda: api.sort_tokens(x, ids, 257),
                 lambda: api.sort_tokens(x, ids, 4, align=3), lambda: api.sort_tokens(x[:, :12], ids, 4),
                 lambda: api.sort_tokens(x, ids[:, :0], 4)):
        with pytest.raises(binding.Nvfp4Error):
            call()
