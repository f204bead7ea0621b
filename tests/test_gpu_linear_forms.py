"""Every form of the linear's kernels by name: the sizes here are asked which form they
run in, and give results within the bounds and follow the activations at their far
arguments there."""
import math

import pytest

import expert_ops_reference as R

pytestmark = pytest.mark.gpu

INF, NAN = math.inf, math.nan
FEW, C64, C64_SPLIT, C128, C128_SPLIT, C256, PAIR, TURNED = (
    "few rows", "64 columns", "64 columns, split K", "128 columns", "128 columns, split K", "256 columns", "pairs",
    "turned pairs")
_NAMES = {(0, 0, 0, False): FEW, (64, 0, 0, False): C64, (64, 0, 0, True): C64_SPLIT, (128, 0, 0, False): C128,
          (128, 0, 0, True): C128_SPLIT, (256, 0, 0, False): C256, (256, 1, 0, False): PAIR, (256, 1, 1, False): TURNED}
ACT = {None: 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4, "swiglu": 5}
E = 5  # experts

# form -> (M, N, K), (M, N, K) with SwiGLU; experts: M rows over E of them.  The plan knows how many clusters of a size
# a device holds: sizes are such that the form is the same with some fewer of them.
LINEAR = {FEW: [(16, 72, 264)] * 2, C64: [(41, 136, 72)] * 2, C64_SPLIT: [(35, 136, 2056)] * 2,
          C128: [(777, 4240, 72)] * 2, C128_SPLIT: [(300, 2504, 7688), (300, 1256, 7688)], C256: [(2600, 4640, 72)] * 2,
          PAIR: [(803, 3032, 720)] * 2}
EXPERTS = {FEW: [(5, 72, 136)] * 2, C64: [(41, 72, 136)] * 2, C128: [(60, 3096, 360)] * 2,
           C256: [(2470, 4552, 72)] * 2, TURNED: [(900, 2056, 1032)] * 2}
SPLIT = (C64_SPLIT, C128_SPLIT)  # one or the other, by the device's clusters
# M, N, K, activation, form of dx, form of dw
GRADS = [(41, 72, 136, None, C64, C64), (2100, 16, 16, None, C64, C64_SPLIT),
         (70, 1168, 2944, "swiglu", C64_SPLIT, C128), (1300, 72, 2688, None, C128, C64),
         (300, 7688, 2504, None, C128_SPLIT, C128), (7688, 304, 2504, "relu", C128, C128_SPLIT),
         (3300, 3128, 72, None, SPLIT, SPLIT), (4100, 72, 2968, "gelu", C256, SPLIT),
         (777, 776, 2784, None, PAIR, PAIR), (777, 776, 2784, "swiglu", PAIR, C256)]
EXPERT_GRADS = [(41, 72, 136, None, C64, C64), (60, 328, 2456, "swiglu", C128, C128),
                (64, 744, 3888, None, C256, C128), (900, 1032, 2056, "silu", TURNED, C256)]


def _form(M, N, K, act=None, groups=0, product=0):
    from nvfp4_mixture_experts_expert_gb300 import binding as B
    table = 16 if groups else None  # looked at for NULL alone
    shape = B.linear_shape(M, N, K, B.NVFP4_BF16, ACT[act], groups=groups, offsets=table, counts=table)
    columns, pair, turned, split = B.nvfp4_debug_linear_form(shape, product)
    return _NAMES[columns, pair, turned, split > 1]


def _randn(g, *shape):
    import torch
    return torch.randn(*shape, generator=g, device="cuda")


def _order(M, seed):
    """M rows over E experts, unevenly, one of them without any where M allows it."""
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    share = torch.tensor([0.3, 0.0, 0.05, 0.5, 0.15])
    ids = torch.multinomial(share, M, True, generator=torch.Generator().manual_seed(seed)).to(torch.int32)[:, None]
    return api.sort_tokens(torch.zeros(M, 8, dtype=torch.bfloat16, device="cuda"), ids.cuda(), E)[1]


def _slices(order):
    at, counts = order.offsets.tolist(), order.counts.tolist()
    return [slice(a, a + c) for a, c in zip(at, counts)]


def _run(x, w, b, act, res, limits, out_dtype, order):
    from nvfp4_mixture_experts_expert_gb300 import api
    kw = dict(out_dtype=out_dtype, preact=True)
    if order is None:
        return api.linear(x, w, b, act, res, *limits, **kw)
    return api.expert_linear(x, w, order, b, act, res, *limits, **kw)


def _all(sizes):
    return [(form, act, *at[act == "swiglu"]) for form, at in sizes.items()
            for act in (None, "relu", "silu", "gelu", "gelu_tanh", "swiglu")]


@pytest.mark.parametrize("experts", [False, True])
def test_the_lists_name_every_form(experts):
    forms = set(_NAMES.values()) - ({PAIR, C64_SPLIT, C128_SPLIT} if experts else {TURNED})
    assert set(EXPERTS if experts else LINEAR) == forms
    grads = EXPERT_GRADS if experts else GRADS
    assert {g[4] for g in grads} - {SPLIT} == forms - {FEW}
    assert {g[5] for g in grads} - {SPLIT} == forms - {FEW, TURNED}  # groups' rows as the contraction: single CTAs


@pytest.mark.parametrize("form,act,M,N,K,experts", [(*c, False) for c in _all(LINEAR)] + [(*c, True) for c in _all(EXPERTS)])
def test_forward(form, act, M, N, K, experts):
    import torch
    assert _form(M, N, K, act, E if experts else 0) == form
    g = torch.Generator(device="cuda").manual_seed(M)
    wide, lead = (2 * N if act == "swiglu" else N), (E,) if experts else ()
    order = _order(M, M) if experts else None
    x, res = _randn(g, M, K + 8).bfloat16()[:, :K], _randn(g, M, N).bfloat16()
    w, b = (_randn(g, *lead, wide, K) / math.sqrt(K)).bfloat16(), _randn(g, *lead, wide)
    limits = (1.5, 0.75) if act == "swiglu" else (INF, INF)
    for out_dtype in (torch.bfloat16, torch.float32):
        out, z = _run(x, w, b, act, res, limits, out_dtype, order)
        for e, at in enumerate(_slices(order) if experts else [slice(0, M)]):
            zr, zt, yr, yt = R.linear(x[at], w[e] if experts else w, b[e] if experts else b, act, res[at], limits, out_dtype)
            R.check(out[at], yr, yt)
            R.check(z[at], zr, R.rounded(zr, zt, z.dtype))


# far arguments: FP32's exponential is subnormal below -87, infinite above 88
FAR = [0.0, -0.0, 1e-30, -1e-30, 0.5, -3.0, 17.0, -20.0, 89.0, -89.0, -103.0, 200.0, -200.0, 1e4, -1e4, 1e30, -1e30, INF,
       -INF, NAN]
UP = [1.0, INF, NAN, -2.0, 0.0, 1e4, -INF]


def _same_far(got, ref, tol):
    """got against a reference that has infinities and NaN."""
    import torch
    assert torch.equal(got.isnan(), ref.isnan())
    inf = ref.isinf()
    assert torch.equal(got[inf].double(), ref[inf])
    R.check(got[ref.isfinite()], ref[ref.isfinite()], tol[ref.isfinite()])


@pytest.mark.parametrize("form,act,M,N,K,experts", [(*c, False) for c in _all(LINEAR) if c[1]] +
                                                   [(*c, True) for c in _all(EXPERTS) if c[1]])
def test_far_arguments_of_the_activations(form, act, M, N, K, experts):
    """z is the bias alone (x is zeros): columns take the arguments in turn.  As the formulas
    have it -inf times a sigmoid of 0 is NaN; relu gives 0.  Bounds: the functions within 16
    units of FP32 of 1 + |z| (see expert_ops_reference), SwiGLU's times the up half, whose
    product is rounded once."""
    import torch
    assert _form(M, N, K, act, E if experts else 0) == form
    order = _order(M, M + 1) if experts else None
    lead = (E,) if experts else ()
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    at = torch.arange(N, device="cuda")
    z = torch.tensor(FAR, device="cuda")[at % len(FAR)]
    if act == "swiglu":
        z = torch.cat((z, torch.tensor(UP, device="cuda")[at // len(FAR) % len(UP)]))
    w = torch.randn(*lead, z.numel(), K, device="cuda").bfloat16()
    b = z.expand(*lead, -1).contiguous()
    for limits in ((INF, INF), (7.0, 3.0)) if act == "swiglu" else ((INF, INF),):
        Z = z.double()
        defined = torch.ones(N, dtype=torch.bool, device="cuda")
        if act == "swiglu":
            gate, up = Z[:N].clamp(max=limits[0]), Z[N:].clamp(-limits[1], limits[1])
            y = gate * torch.sigmoid(gate) * up
            tol = 16 * R.U32 * (1 + gate.abs()) * up.abs() + R.U32 * y.abs()
            # an infinite up half of a gate whose silu FP32 has as a subnormal number or 0: either
            defined = ~(up.isinf() & (gate < 0) & ((gate * torch.sigmoid(gate)).abs() < 2.0 ** -126))
        elif act == "relu":
            y, tol = torch.where(Z < 0, 0.0, Z), torch.zeros_like(Z)
        else:
            y = {"silu": lambda: Z * torch.sigmoid(Z), "gelu": lambda: Z * torch.special.ndtr(Z),
                 "gelu_tanh": lambda: Z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (Z + 0.044715 * Z ** 3))}[act]()
            tol = 16 * R.U32 * (1 + Z.abs())
        for out_dtype in (torch.float32, torch.bfloat16):
            out, kept = _run(x, w, b, act, None, limits, out_dtype, order)
            for s in _slices(order) if experts else [slice(0, M)]:
                if s.start == s.stop:
                    continue
                rows = out[s]
                assert torch.equal(rows.nan_to_num(nan=12.0), rows[:1].expand_as(rows).nan_to_num(nan=12.0))
                _same_far(rows[0][defined], y[defined], R.rounded(y, tol, out_dtype)[defined])
                _same_far(kept[s][-1], Z, R.rounded(Z, torch.zeros_like(Z), kept.dtype))


@pytest.mark.parametrize("M,N,K,act,dx_form,dw_form,experts", [(*c, False) for c in GRADS] + [(*c, True) for c in EXPERT_GRADS])
def test_gradients(M, N, K, act, dx_form, dw_form, experts):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    groups = E if experts else 0
    for product, form in ((1, dx_form), (2, dw_form)):
        assert _form(M, N, K, act, groups, product) in (form if form is SPLIT else (form,))
    g = torch.Generator(device="cuda").manual_seed(N)
    wide, lead = (2 * N if act == "swiglu" else N), (E,) if experts else ()
    x, dy = _randn(g, M, K).bfloat16(), _randn(g, M, N + 8).bfloat16()[:, :N]
    w = (_randn(g, *lead, wide, K) / math.sqrt(K)).bfloat16()
    z = None if act is None else (2 * _randn(g, M, wide)).bfloat16()
    if experts:
        order = _order(M, M + 2)
        dx, dw, db = api.expert_linear_grad(dy, x, w, order, z, act, 1.5, 0.75, bias=True)
    else:
        dx, dw, db = api.linear_grad(dy, x, w, z, act, 1.5, 0.75, bias=True)
    if act == "relu":  # relu'(0) = 0, where the reference's derivative of clamp is 1; z decides on the slope alone
        z = torch.where(z == 0, torch.full_like(z, -1), z)
    for e, at in enumerate(_slices(order) if experts else [slice(0, M)]):
        want = R.linear_grad(dy[at], x[at], w[e] if experts else w, None if z is None else z[at], act, (1.5, 0.75), x.dtype)
        for got, (ref, tol) in zip((dx[at], dw[e], db[e]) if experts else (dx, dw, db), want):
            R.check(got, ref, tol)


@pytest.mark.parametrize("M", [16, 17])
@pytest.mark.parametrize("N,K", [(8, 8), (48, 4096), (1000, 1288)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_around_the_few_rows_limit(M, N, K, dtype):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    assert (_form(M, N, K) == FEW) == (M == 16)
    g = torch.Generator(device="cuda").manual_seed(M)
    t = getattr(torch, dtype)
    x, w = _randn(g, M, K).to(t), (_randn(g, N, K) / math.sqrt(K)).to(t)
    for out_dtype in (t, torch.float32):
        _, _, ref, tol = R.linear(x, w, None, None, None, (INF, INF), out_dtype)
        R.check(api.linear(x, w, out_dtype=out_dtype), ref, tol)


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh", "swiglu"])
def test_gradient_against_differences_away_from_kinks(act):
    """Central differences of the FP64 definition, off by h^2 of its third derivative (below 10
    h^2 a term); z is moved away from where the definition has a kink."""
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    g = torch.Generator(device="cuda").manual_seed(5)
    M, N, K = 24, 16, 40
    wide, limits = (2 * N if act == "swiglu" else N), (1.0, 1.0)
    x, dy = _randn(g, M, K).bfloat16(), _randn(g, M, N).bfloat16()
    w, z = (_randn(g, wide, K) / math.sqrt(K)).bfloat16(), (1.5 * _randn(g, M, wide)).bfloat16()
    kinks = {"relu": (0.0,), "swiglu": (1.0, -1.0)}.get(act, ())
    for v in kinks:
        z[(z - v).abs() < 0.05] = v + 0.0625
    assert all(((z.double() - v).abs() > 0.01).all() for v in kinks)
    dx, dw, db = api.linear_grad(dy, x, w, z, act, *limits, bias=True)
    (_, tx), (_, tw), (_, tb) = R.linear_grad(dy, x, w, z, act, limits, x.dtype)
    shift = z.double() - x.double() @ w.double().T  # the gradient is taken at z as given

    def loss(x, w, extra):
        return (dy.double() * R.act(x @ w.T + shift + extra, act, limits)).sum()

    h = 1e-5
    X, W, Z = x.double(), w.double(), torch.zeros(wide, dtype=torch.float64, device="cuda")
    for k in range(40):
        for at, (which, got, tol) in ((divmod(23 * k, K), (0, dx, tx)), ((k % wide, 3 * k % K), (1, dw, tw)),
                                      ((k % wide,), (2, db, tb))):
            args = [X.clone(), W.clone(), Z.clone()]
            args[which][at] += h
            up = loss(*args)
            args[which][at] -= 2 * h
            diff = (up - loss(*args)) / (2 * h)
            assert abs(float(got[at]) - float(diff)) <= float(tol[at]) + 1e-6, (act, which, at)


@pytest.mark.parametrize("M,groups", [(32, 32), (32, 256), (33, 256), (24, 24), (25, 24), (250, 256)])
@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("share", [1, 0.5, 0])
def test_rows_as_many_as_experts(M, groups, act, share):
    """All rows of one expert, half of them, each of an expert of its own (as far as there are any)."""
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    N, K = 72, 264
    assert (_form(M, N, K, act, groups) == FEW) == (M <= min(groups, 32))
    g = torch.Generator(device="cuda").manual_seed(M)
    ids = (torch.arange(M, dtype=torch.int32) * 7 + 3) % groups
    ids[:int(share * M)] = groups - 2
    _, order = api.sort_tokens(torch.zeros(M, 8, dtype=torch.bfloat16, device="cuda"), ids[:, None].cuda(), groups)
    wide = 2 * N if act else N
    x, res = _randn(g, M, K).bfloat16(), _randn(g, M, N).bfloat16()
    w, b = (_randn(g, groups, wide, K) / math.sqrt(K)).bfloat16(), _randn(g, groups, wide).bfloat16()
    out, z = api.expert_linear(x, w, order, b, act, res, 1.5, 0.75, out_dtype=torch.float32, preact=True)
    for e, at in enumerate(_slices(order)):
        if at.start < at.stop:
            zr, zt, yr, yt = R.linear(x[at], w[e], b[e], act, res[at], (1.5, 0.75), out.dtype)
            R.check(out[at], yr, yt)
            R.check(z[at], zr, R.rounded(zr, zt, z.dtype))
