"""The linear with bias, activation and residual, its expert form and their
gradients against 64 bits."""
import math

import pytest

import expert_ops_reference as R

pytestmark = pytest.mark.gpu

INF = math.inf
ACTS = [None, "relu", "silu", "gelu", "gelu_tanh", "swiglu"]


def _randn(g, *shape):
    import torch
    return torch.randn(*shape, generator=g, device="cuda")


def _inputs(M, N, K, dtype, act, bias, residual, seed=0, pad=8, experts=None):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = getattr(torch, dtype)
    wide = 2 * N if act == "swiglu" else N
    lead = () if experts is None else (experts,)
    x = _randn(g, M, K + pad).to(t)[:, :K]
    w = (_randn(g, *lead, wide, K) / math.sqrt(K)).to(t)
    b = None if bias is None else _randn(g, *lead, wide).to(t if bias == "same" else torch.float32)
    res = _randn(g, M, N + pad).to(t)[:, :N] if residual else None
    return x, w, b, res


def _check(x, w, b, res, act, limits, out_dtype, out, z=None):
    zr, zt, yr, yt = R.linear(x, w, b, act, res, limits, out_dtype)
    R.check(out, yr, yt)
    if z is not None:
        R.check(z, zr, R.rounded(zr, zt, z.dtype))


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 31, 64, 127, 128, 129, 300])
@pytest.mark.parametrize("N,K", [(8, 8), (48, 4096), (264, 400), (1000, 1288)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_linear_plain(M, N, K, dtype):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    x, w, _, _ = _inputs(M, N, K, dtype, None, None, False, seed=M)
    for out_dtype in (x.dtype, torch.float32):
        out = torch.full((M, N), float("nan"), dtype=out_dtype, device="cuda")
        assert api.linear(x, w, out=out).data_ptr() == out.data_ptr()
        _check(x, w, None, None, None, (INF, INF), out_dtype, out)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 40, 264), (6, 136, 1032), (70, 72, 2056), (333, 264, 520), (1500, 1160, 328)])
@pytest.mark.parametrize("dtype,bias,residual,f32", [("bfloat16", "same", True, False), ("float16", "f32", False, True),
                                                      ("float16", None, True, False), ("bfloat16", "f32", True, True)])
def test_linear_epilogue(M, N, K, act, dtype, bias, residual, f32):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    x, w, b, res = _inputs(M, N, K, dtype, act, bias, residual, seed=N)
    limits = (1.5, 0.75) if act == "swiglu" and bias else (INF, INF)
    out_dtype = torch.float32 if f32 else x.dtype
    out, z = api.linear(x, w, b, act, res, *limits, out_dtype=out_dtype, preact=True)
    _check(x, w, b, res, act, limits, out_dtype, out, z)
    assert torch.equal(out, api.linear(x, w, b, act, res, *limits, out_dtype=out_dtype))


@pytest.mark.parametrize("M,N,K", [(20, 136, 66000), (3, 8, 131072), (128, 8200, 200), (2048, 2304, 1032),
                                   (4100, 520, 136)])
def test_linear_larger(M, N, K):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    x, w, b, res = _inputs(M, N, K, "bfloat16", None, "same", True, seed=1)
    out = api.linear(x, w, b, residual=res, out_dtype=torch.float32)
    _check(x, w, b, res, None, (INF, INF), torch.float32, out)
    assert torch.equal(out, api.linear(x, w, b, residual=res, out_dtype=torch.float32))


# Sizes at which the plan takes each tile form (64, 128 and 256 columns, CTA pairs, K over a cluster) with 152 SMs,
# for each of the three epilogues
FORMS = [(777, 4240, 72), (135, 1560, 2824), (2600, 4640, 72), (390, 4944, 584), (1300, 4448, 72), (260, 4872, 40),
         (135, 776, 2856), (135, 4872, 584)]


@pytest.mark.parametrize("M,N,K", FORMS)
@pytest.mark.parametrize("act,dtype", [(None, "bfloat16"), ("gelu", "float16"), ("swiglu", "bfloat16")])
def test_linear_tile_forms(M, N, K, act, dtype):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    x, w, b, res = _inputs(M, N, K, dtype, act, "same", True, seed=M)
    limits = (1.5, 0.75) if act == "swiglu" else (INF, INF)
    buf = torch.full((M + 1, N + 16), float("nan"), dtype=x.dtype, device="cuda")
    out, z = api.linear(x, w, b, act, res, *limits, preact=True, out=buf[1:, 8:N + 8])
    _check(x, w, b, res, act, limits, x.dtype, out, z)
    assert buf[0].isnan().all() and buf[:, :8].isnan().all() and buf[:, N + 8:].isnan().all()
    _check(x, w, None, None, act, limits, torch.float32, api.linear(x, w, None, act, None, *limits, out_dtype=torch.float32))


@pytest.mark.parametrize("M,N,K", [(70, 1168, 2944), (3300, 3128, 72), (70, 3984, 2960), (777, 776, 2784), (2100, 16, 16),
                                   (1300, 72, 2688), (135, 2856, 1544), (4100, 72, 2968), (777, 584, 2768)])
@pytest.mark.parametrize("act,dtype", [(None, "float16"), ("swiglu", "bfloat16")])
def test_linear_grad_tile_forms(M, N, K, act, dtype):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    g = torch.Generator(device="cuda").manual_seed(M)
    x, w, _, _ = _inputs(M, N, K, dtype, act, None, False, seed=N)
    dy = _randn(g, M, N + 8).to(x.dtype)[:, :N]
    z = None if act is None else (2 * _randn(g, M, 2 * N)).to(x.dtype)
    buf = torch.full((M + 1, K + 16), float("nan"), dtype=x.dtype, device="cuda")
    dx, dw, db = api.linear_grad(dy, x, w, z, act, 1.5, 0.75, bias=True, out=buf[1:, 8:K + 8])
    for got, (ref, tol) in zip((dx, dw, db), R.linear_grad(dy, x, w, z, act, (1.5, 0.75), x.dtype)):
        R.check(got, ref, tol)
    assert buf[0].isnan().all() and buf[:, :8].isnan().all() and buf[:, K + 8:].isnan().all()


def test_offsets_beyond_32_bits():
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    M, N, K = 600000, 4096, 64
    x, w, b, _ = _inputs(M, N, K, "bfloat16", None, "same", False, pad=0)
    out = api.linear(x, w, b)  # 2.5e9 elements
    for at in (slice(0, 300), slice(524200, 524400), slice(M - 300, M)):
        _check(x[at], w, b, None, None, (INF, INF), out.dtype, out[at])
    # dy's rows lie that far apart too; dx by its rows, dw over all of them
    dx, dw, _ = api.linear_grad(out, x, w)
    (rx, tx), _, _ = R.linear_grad(out[-300:], x[-300:], w, None, None, (INF, INF), x.dtype)
    R.check(dx[-300:], rx, tx)
    dw64 = torch.zeros(N, K, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(dw64)
    for s in range(0, M, 20000):
        d, v = out[s:s + 20000].double(), x[s:s + 20000].double()
        dw64 += d.T @ v
        mag += d.abs().T @ v.abs()
    R.check(dw, dw64, R.rounded(dw64, mag * ((M / 16 * 2 + 40) * R.U32), dw.dtype))


def test_rows_depend_on_themselves_alone_and_extremes():
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    for M in (8, 200):
        x, w, b, _ = _inputs(M, 72, 264, "bfloat16", "silu", "same", False)
        want = api.linear(x, w, b, "silu")
        x[3] = float("nan")
        x[5, 0] = float("inf")
        got = api.linear(x, w, b, "silu")
        keep = torch.ones(M, dtype=torch.bool, device="cuda")
        keep[3] = keep[5] = False
        assert torch.equal(got[keep], want[keep]) and got[3].isnan().all() and not got[5].isfinite().all()
    # far arguments of the activations, through an identity product
    v = torch.tensor([-3e38, -1e4, -200, -89, -20, 0, 20, 89, 200, 1e4, 3e38, float("inf"), -float("inf"),
                      float("nan"), -0.0, 1e-30], device="cuda")
    x = torch.zeros(16, 16, device="cuda")
    x[:, 0] = v
    w = torch.zeros(16, 16, device="cuda")
    w[:8, 0] = 1
    for rows in (16, 8):
        for act in ACTS[1:5]:
            got = api.linear(x[:rows].bfloat16(), w.bfloat16()[:8], activation=act, out_dtype=torch.float32)[:, 0]
            z = x[:rows, 0].bfloat16().double()
            ref = torch.where(z.isinf() & (z < 0), 0.0 * z if act != "relu" else 0.0, R.act(z, act))
            fin = z.isfinite()
            R.check(got[fin], ref[fin], 16 * R.U32 * (1 + z[fin].abs()))
            assert got[z.isnan()].isnan().all() and (got[z == INF] == INF).all()


def test_residual_in_place_and_strided_output():
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    for M in (5, 150):
        x, w, b, res = _inputs(M, 136, 264, "float16", "gelu", "same", True)
        want = api.linear(x, w, b, "gelu", res)
        buf = torch.full((M + 2, 160), float("nan"), dtype=x.dtype, device="cuda")
        out = buf[1:M + 1, 8:144]
        out.copy_(res)
        api.linear(x, w, b, "gelu", out, out=out)
        assert torch.equal(out, want)
        buf[1:M + 1, 8:144] = float("nan")
        assert buf.isnan().all()


# ------------------------------------------------------------------ gradient


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 40, 264), (9, 264, 72), (130, 136, 1032), (700, 72, 136), (1500, 1160, 328)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_linear_grad(M, N, K, act, dtype):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    g = torch.Generator(device="cuda").manual_seed(M)
    x, w, _, _ = _inputs(M, N, K, dtype, act, None, False, seed=N)
    dy = _randn(g, M, N + 8).to(x.dtype)[:, :N]
    z = None if act is None else (2 * _randn(g, M, w.shape[0])).to(x.dtype)
    limits = (1.5, 0.75) if act == "swiglu" else (INF, INF)
    dx, dw, db = api.linear_grad(dy, x, w, z, act, *limits, bias=True)
    (rx, tx), (rw, tw), (rb, tb) = R.linear_grad(dy, x, w, z, act, limits, x.dtype)
    R.check(db, rb, tb)
    R.check(dx, rx, tx)
    R.check(dw, rw, tw)
    only = api.linear_grad(dy, x, w, z, act, *limits, weights=False)
    assert torch.equal(only[0], dx) and only[1] is None and only[2] is None
    only = api.linear_grad(dy, x, w, z, act, *limits, inputs=False)
    assert only[0] is None and torch.equal(only[1], dw)
    only = api.linear_grad(dy, x, w, z, act, *limits, inputs=False, weights=False, bias=True)
    assert torch.equal(only[2], db)


@pytest.mark.parametrize("act", ACTS)
def test_linear_grad_against_differences(act):
    """Central differences of the FP64 definition: off by h^2 of the third derivative."""
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    g = torch.Generator(device="cuda").manual_seed(5)
    x, w, b, _ = _inputs(24, 16, 40, "bfloat16", act, "same", False, seed=5)
    dy = _randn(g, 24, 16).to(x.dtype)
    limits = (1.0, 1.0)
    _, z = api.linear(x, w, b, act, None, *limits, preact=True)
    dx, dw, db = api.linear_grad(dy, x, w, z, act, *limits, bias=True)
    # the gradient is taken at the rounded z: the constant that makes it the definition's z
    shift = z.double() - x.double() @ w.double().T

    def loss(x, w, extra):
        return (dy.double() * R.act(x @ w.T + shift + extra, act, limits)).sum()

    h = 1e-6
    X, W, Z = x.double(), w.double(), torch.zeros(w.shape[0], dtype=torch.float64, device="cuda")
    (_, tx), (_, tw), (_, tb) = R.linear_grad(dy, x, w, z, act, limits, x.dtype)
    near = {"relu": (0.0,), "swiglu": (1.0, -1.0)}.get(act, ())  # no difference across a kink
    assert all(((z.double() - v).abs() > 1e-4).all() for v in near) or act in ("relu", "swiglu")
    for k in range(12):
        for at, (which, got, tol) in ((divmod(7 * k, 40), (0, dx, tx)), ((k % w.shape[0], 3 * k % 40), (1, dw, tw)),
                                      ((k % w.shape[0],), (2, db, tb))):
            args = [X.clone(), W.clone(), Z.clone()]
            args[which][at] += h
            up = loss(*args)
            args[which][at] -= 2 * h
            diff = (up - loss(*args)) / (2 * h)
            assert abs(float(got[at]) - float(diff)) <= float(tol[at]) + 1e-4, (act, which, at)


def test_linear_no_rows():
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    x, w, b, _ = _inputs(0, 16, 24, "bfloat16", "silu", "same", False)
    out, z = api.linear(x, w, b, "silu", preact=True)
    assert out.shape == (0, 16) and z.shape == (0, 16)
    dx, dw, db = api.linear_grad(out, x, w, z, "silu", bias=True)
    assert dx.shape == (0, 24) and not dw.any() and not db.any()


# ------------------------------------------------------------------ experts


def _experts(T, k, E, model, K, N, dtype, act, bias, seed=0, align=1, skew=False):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, model, generator=g) + (4.0 * torch.randn(1, model, generator=g) if skew else 0)
    ids = logits.topk(k, dim=1).indices.to(torch.int32)
    t = getattr(torch, dtype)
    x = torch.zeros(T, 8, dtype=t, device="cuda")
    _, order = api.sort_tokens(x, ids.cuda(), E, (model - E) // 2, align)
    n = order.source.numel()
    rows, w, b, res = _inputs(n, N, K, dtype, act, bias, True, seed=seed, experts=E)
    rows = torch.where((order.source >= 0)[:, None], rows, torch.full_like(rows, float("nan")))
    return rows, w, b, res, order


# the last nine: the tile forms, as above
EXPERTS = [(1, 6, 32, 32, 264, 136), (1, 32, 256, 256, 72, 40), (60, 4, 256, 256, 264, 72), (90, 8, 256, 300, 72, 136), (9, 2, 5, 10, 72, 264), (40, 4, 12, 24, 520, 72), (300, 3, 7, 7, 264, 200),
           (1500, 2, 5, 5, 136, 1032), (700, 8, 100, 130, 72, 40),
           (379, 2, 5, 5, 72, 3496), (1573, 2, 5, 5, 72, 3472), (68, 2, 5, 5, 680, 3856), (927, 2, 3, 3, 72, 2840),
           (70, 2, 3, 3, 584, 2632), (1381, 2, 5, 5, 1968, 40), (64, 2, 5, 5, 1064, 2288), (2836, 2, 5, 5, 1992, 64),
           (392, 2, 5, 5, 1984, 616)]


def _slices(order):
    ends, counts = order.offsets.tolist(), order.counts.tolist()
    return [slice(ends[e], ends[e] + counts[e]) for e in range(len(counts))]


@pytest.mark.parametrize("T,k,E,model,K,N", EXPERTS)
@pytest.mark.parametrize("act,dtype,bias,align,skew", [(None, "bfloat16", None, 1, False),
                                                       ("swiglu", "bfloat16", "f32", 1, True),
                                                       ("gelu", "float16", "same", 16, True),
                                                       ("swiglu", "float16", "same", 128, False)])
def test_expert_linear(T, k, E, model, K, N, act, dtype, bias, align, skew):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    rows, w, b, res, order = _experts(T, k, E, model, K, N, dtype, act, bias, seed=T, align=align, skew=skew)
    limits = (1.5, 0.75) if act == "swiglu" else (INF, INF)
    for residual in (None, res):
        out = torch.full((rows.shape[0], N), 7.0, dtype=rows.dtype, device="cuda")
        got, z = api.expert_linear(rows, w, order, b, act, residual, *limits, preact=True, out=out)
        assert got.data_ptr() == out.data_ptr()
        used = torch.zeros(rows.shape[0], dtype=torch.bool, device="cuda")
        for e, at in enumerate(_slices(order)):
            used[at] = True
            _check(rows[at], w[e], None if b is None else b[e], None if residual is None else residual[at], act, limits,
                   out.dtype, out[at], z[at])
        assert (out[~used] == 7).all()


@pytest.mark.parametrize("T,k,E,model,K,N", EXPERTS)
@pytest.mark.parametrize("act,dtype,align,skew", [(None, "bfloat16", 1, True), ("swiglu", "bfloat16", 1, False),
                                                  ("silu", "float16", 16, True)])
def test_expert_linear_grad(T, k, E, model, K, N, act, dtype, align, skew):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    rows, w, _, _, order = _experts(T, k, E, model, K, N, dtype, act, None, seed=T, align=align, skew=skew)
    n = rows.shape[0]
    g = torch.Generator(device="cuda").manual_seed(T)
    nan = lambda t: torch.where((order.source >= 0)[:, None], t, torch.full_like(t, float("nan")))
    dy = nan(_randn(g, n, N).to(rows.dtype))
    z = None if act is None else nan((2 * _randn(g, n, w.shape[1])).to(rows.dtype))
    limits = (1.5, 0.75) if act == "swiglu" else (INF, INF)
    out = torch.full((n, K), 7.0, dtype=rows.dtype, device="cuda")
    dx, dw, db = api.expert_linear_grad(dy, rows, w, order, z, act, *limits, bias=True, out=out)
    used = torch.zeros(n, dtype=torch.bool, device="cuda")
    for e, at in enumerate(_slices(order)):
        used[at] = True
        (rx, tx), (rw, tw), (rb, tb) = R.linear_grad(dy[at], rows[at], w[e], None if z is None else z[at], act, limits,
                                                     rows.dtype)
        R.check(dx[at], rx, tx)
        R.check(dw[e], rw, tw)
        R.check(db[e], rb, tb)
        if at.start == at.stop:
            assert not dw[e].any() and not db[e].any()
    assert (dx[~used] == 7).all()


# Rows of experts at the edges of tiles: none, one, around 32 and 256, several tiles, many.
COUNTS = (0, 1, 31, 33, 256, 257, 300, 513, 1793)


def _experts_of(counts, K, N, dtype, act, bias, align, seed):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    ids = torch.repeat_interleave(torch.arange(len(counts), dtype=torch.int32), torch.tensor(counts))
    ids = ids[torch.randperm(ids.numel(), generator=torch.Generator().manual_seed(seed))][:, None]
    t = getattr(torch, dtype)
    _, order = api.sort_tokens(torch.zeros(ids.shape[0], 8, dtype=t, device="cuda"), ids.cuda(), len(counts), 0, align)
    assert order.counts.tolist() == list(counts)
    rows, w, b, res = _inputs(order.source.numel(), N, K, dtype, act, bias, True, seed=seed, experts=len(counts))
    nan = torch.full_like(rows, float("nan"))
    return torch.where((order.source >= 0)[:, None], rows, nan), w, b, res, order


@pytest.mark.parametrize("act,dtype,bias,f32", [(None, "bfloat16", None, False), (None, "float16", "same", True),
                                                ("swiglu", "bfloat16", "f32", False), ("swiglu", "float16", "same", True),
                                                ("silu", "bfloat16", "same", True), ("gelu", "float16", "f32", False)])
@pytest.mark.parametrize("K,N,align", [(1032, 1000, 1), (1032, 1000, 16), (1992, 1176, 1), (2048, 1304, 128)])
def test_expert_linear_counts(K, N, align, act, dtype, bias, f32):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    rows, w, b, res, order = _experts_of(COUNTS, K, N, dtype, act, bias, align, seed=K + align)
    limits = (1.5, 0.75) if act == "swiglu" else (INF, INF)
    n, out_dtype = rows.shape[0], torch.float32 if f32 else rows.dtype
    pad = torch.full((n + 1, N + 24), 7.0, dtype=out_dtype, device="cuda")
    for residual in (None, res):
        out = pad[1:, 8:N + 8]
        got, z = api.expert_linear(rows, w, order, b, act, residual, *limits, preact=True, out=out)
        used = torch.zeros_like(pad, dtype=torch.bool)
        for e, at in enumerate(_slices(order)):
            used[1:, 8:N + 8][at] = True
            _check(rows[at], w[e], None if b is None else b[e], None if residual is None else residual[at], act, limits,
                   out_dtype, out[at], z[at])
        assert (pad[~used] == 7).all()
    if not f32:  # in place of the residual, and without the sums
        want, place = out.clone(), res.clone()
        api.expert_linear(rows, w, order, b, act, place, *limits, out=place)
        for at in _slices(order):
            assert torch.equal(place[at], want[at])
    again = api.expert_linear(rows, w, order, b, act, res, *limits, out_dtype=out_dtype)
    for at in _slices(order):
        assert torch.equal(again[at], out[at])


@pytest.mark.parametrize("act,dtype", [(None, "bfloat16"), ("swiglu", "float16"), ("silu", "bfloat16")])
@pytest.mark.parametrize("K,N,align", [(1000, 1032, 1), (1304, 2048, 16), (2600, 1096, 1)])
def test_expert_linear_grad_counts(K, N, align, act, dtype):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    rows, w, _, res, order = _experts_of(COUNTS, K, N, dtype, act, None, align, seed=N)
    used = (order.source >= 0)[:, None]
    nan = lambda t: torch.where(used, t, torch.full_like(t, float("nan")))
    dy = nan(res)
    g = torch.Generator(device="cuda").manual_seed(K)
    z = None if act is None else nan((2 * _randn(g, rows.shape[0], w.shape[1])).to(rows.dtype))
    limits = (1.5, 0.75) if act == "swiglu" else (INF, INF)
    out = torch.full((rows.shape[0], K + 8), 7.0, dtype=rows.dtype, device="cuda")
    dx, dw, db = api.expert_linear_grad(dy, rows, w, order, z, act, *limits, bias=True, out=out[:, :K])
    for e, at in enumerate(_slices(order)):
        want = R.linear_grad(dy[at], rows[at], w[e], None if z is None else z[at], act, limits, rows.dtype)
        for got, (ref, tol) in zip((dx[at], dw[e], db[e]), want):
            R.check(got, ref, tol)
    assert (out[:, K:] == 7).all() and (dx[~used[:, 0]] == 7).all()


def test_expert_linear_without_rows():
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    for T in (4, 700):
        ids = torch.full((T, 2), 99, dtype=torch.int32, device="cuda")
        rows, order = api.sort_tokens(torch.ones(T, 16, dtype=torch.bfloat16, device="cuda"), ids, 3)
        w = torch.ones(3, 8, 16, dtype=torch.bfloat16, device="cuda")
        out = torch.full((2 * T, 8), 7.0, dtype=torch.bfloat16, device="cuda")
        api.expert_linear(rows, w, order, out=out)
        assert (out == 7).all()
        dx = torch.full((2 * T, 16), 7.0, dtype=torch.bfloat16, device="cuda")
        _, dw, db = api.expert_linear_grad(out, rows, w, order, bias=True, out=dx)
        assert (dx == 7).all() and not dw.any() and not db.any()


def test_refusals_of_the_python_calls():
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api, binding
    x, w, b, res = _inputs(12, 16, 24, "bfloat16", None, "same", True)
    rows, order = api.sort_tokens(x, torch.zeros(12, 1, dtype=torch.int32, device="cuda"), 2)
    we = torch.stack((w, w))
    for call in (lambda: api.linear(x, w.half()), lambda: api.linear(x.float(), w.float()), lambda: api.linear(x, w.cpu()),
                 lambda: api.linear(x, w[:, :16]), lambda: api.linear(x, we), lambda: api.linear(x, w, b[:8]),
                 lambda: api.linear(x, w, b.half()), lambda: api.linear(x, w, residual=res[:4]),
                 lambda: api.linear(x, w, residual=res.float()), lambda: api.linear(x, w, out=res[:4]),
                 lambda: api.linear(x[0], w), lambda: api.linear(x.t(), w), lambda: api.linear(x, w[:15], activation="swiglu"),
                 lambda: api.linear(x, w, out_dtype=torch.float16),
                 lambda: api.linear_grad(res, x, w, activation="silu"), lambda: api.linear_grad(res[:4], x, w),
                 lambda: api.linear_grad(res[:, :8], x, w), lambda: api.linear_grad(res, x, w, inputs=False, out=x),
                 lambda: api.expert_linear(rows, w, order), lambda: api.expert_linear(rows, we[:1], order),
                 lambda: api.expert_linear(rows, we, order, bias=b)):
        with pytest.raises(ValueError):
            call()
    few = rows[:11]  # fewer than the order's tables name
    for call in (lambda: api.expert_linear(few, we, order), lambda: api.expert_linear_grad(res[:11], few, we, order),
                 lambda: api.combine_tokens(few, torch.ones(12, 1, device="cuda"), order),
                 lambda: api.combine_tokens_grad(x, few, torch.ones(12, 1, device="cuda"), order),
                 lambda: api.sort_tokens_grad(few, order)):
        with pytest.raises(ValueError, match="rows of the order"):
            call()
    for call in (lambda: api.linear(x[:, :20], w[:, :20].contiguous()), lambda: api.linear(x, w[:12].contiguous()),
                 lambda: api.linear(x, w, activation="swiglu", gate_limit=-1.0)):
        with pytest.raises(binding.Nvfp4Error):
            call()


def test_other_stream_and_graph():
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    x, w, b, res = _inputs(200, 264, 520, "bfloat16", "silu", "same", True)
    want, z = api.linear(x, w, b, "silu", res, preact=True)
    grads = api.linear_grad(res, x, w, z, "silu", bias=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, zs = api.linear(x, w, b, "silu", res, preact=True, stream=s)
    more = api.linear_grad(res, x, w, zs, "silu", bias=True, stream=s)
    s.synchronize()
    assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(grads, more))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, z = api.linear(x, w, b, "silu", res, preact=True)
        more = api.linear_grad(res, x, w, z, "silu", bias=True)
    x.mul_(0.5)
    for _ in range(2):
        g.replay()
    want, z = api.linear(x, w, b, "silu", res, preact=True)
    assert torch.equal(out, want)
    assert all(torch.equal(a, b) for a, b in zip(more, api.linear_grad(res, x, w, z, "silu", bias=True)))


def test_a_stalled_product_is_reported():
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api, binding
    x, w, _, _ = _inputs(300, 136, 520, "bfloat16", None, None, False)
    want = api.linear(x, w)
    torch.cuda.synchronize()
    assert binding.nvfp4_device_status(reset=True) == 0
    binding.nvfp4_moe_set_debug_stall(50)
    try:
        api.linear(x, w)
        torch.cuda.synchronize()
    finally:
        binding.nvfp4_moe_set_debug_stall(0)
    assert binding.nvfp4_device_status(reset=True) == binding.NVFP4_ERR_DEVICE_TIMEOUT
    assert torch.equal(api.linear(x, w), want) and binding.nvfp4_device_status() == 0


@pytest.mark.parametrize("act", [None, "swiglu"])
def test_a_stalled_expert_product_is_reported(act):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api, binding
    rows, w, _, _, order = _experts_of(COUNTS, 1032, 1000, "bfloat16", act, None, 1, seed=3)
    want = api.expert_linear(rows, w, order, activation=act)
    torch.cuda.synchronize()
    assert binding.nvfp4_device_status(reset=True) == 0
    binding.nvfp4_moe_set_debug_stall(50)
    try:
        api.expert_linear(rows, w, order, activation=act)
        torch.cuda.synchronize()
    finally:
        binding.nvfp4_moe_set_debug_stall(0)
    assert binding.nvfp4_device_status(reset=True) == binding.NVFP4_ERR_DEVICE_TIMEOUT
    assert torch.equal(api.expert_linear(rows, w, order, activation=act), want) and binding.nvfp4_device_status() == 0


def test_expert_products_in_a_graph_and_on_two_streams():
    import dataclasses
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    calls = []
    for seed, counts in ((1, COUNTS), (2, COUNTS[::-1])):
        rows, w, b, res, order = _experts_of(counts, 1032, 1000, "bfloat16", "swiglu", "same", 1, seed=seed)
        calls.append((rows, w, b, res, order))

    def run(rows, w, b, res, order, stream=None):
        y, z = api.expert_linear(rows, w, order, b, "swiglu", res, preact=True, stream=stream)
        return (y, *api.expert_linear_grad(res, rows, w, order, z, "swiglu", bias=True, stream=stream))

    want = [run(*c) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(3):
        got = [run(*c, stream=s) for c, s in zip(calls, streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, w))
    # a captured call takes the tables that it finds at its replay
    inputs = [t.clone() if torch.is_tensor(t) else
              dataclasses.replace(t, **{f: getattr(t, f).clone() for f in ("offsets", "counts", "source", "inverse")})
              for t in calls[0]]
    run(*inputs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(*inputs)
    for c, w in zip(calls[::-1], want[::-1]):
        for to, of in zip(inputs[:4], c[:4]):
            to.copy_(of)
        for f in ("offsets", "counts", "source", "inverse"):
            getattr(inputs[4], f).copy_(getattr(c[4], f))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, w))
