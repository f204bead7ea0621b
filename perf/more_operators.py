"""Measured cases of the operators around unquantized experts: tokens sorted by expert and back, the linear with bias,
activation and residual in its epilogue, and the same product per expert over sorted rows, each with its gradient.

Each operator has a plain form here (elementary torch operations in 32 bits, rounded once at the end), the call a user
makes of the package (`own`), and its definition in 64 bits (`exact`), written apart from the plain form.

  sort     assignment f = t * k + j of token t belongs to expert ids[t][j] - start, where that lies in [0, E), else to
           none.  Rows ordered by expert, then by f; an expert's first row is a multiple of `align`, rows between are 0.
           rows[inverse[t][j]] = x[t].  Gradient: dx[t] = sum over j of drows[inverse[t][j]].
  combine  out[t] = residual[t] + sum over j of weight[t][j] * rows[inverse[t][j]].  Gradient:
           drows[inverse[t][j]] = weight[t][j] * dout[t],  dweight[t][j] = dout[t] . rows[inverse[t][j]].
  linear   z = x w^T + bias,  y = act(z) + residual.  Gradient from z:  dz = dy * act'(z),  dx = dz w,  dw = dz^T x,
           dbias = the columns' sums of dz.  act: none, relu, silu, gelu (by erf), gelu_tanh, or swiglu, where z is a
           gate half g and an up half u and act = silu(min(g, gate_limit)) * clamp(u, +-up_limit).
  expert   the linear with each expert's own weights and bias over the expert's rows.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh", "swiglu")
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
LIMIT = 10.0


def listed():
    return [
        # one new token's copies for the experts of a decode layer: latency alone
        dict(name="sort 1x4096", op="sort", T=1, H=4096, ld=4096, E=32, k=6, all=32, align=1, type="bf16", grad=False),
        # an odd batch, rows inside a wider buffer, half of the model's experts here, and its gradient
        dict(name="sort 1001x3584 shard f16 + grad", op="sort", T=1001, H=3584, ld=3840, E=12, k=4, all=24, align=1,
             type="f16", grad=True),
        # the prefill layer's batch into slots of 128 rows, as the NVFP4 grouped product takes them
        dict(name="sort 8192x4096 slots", op="sort", T=8192, H=4096, ld=4096, E=48, k=6, all=48, align=128,
             type="bf16", grad=False),
        # a few tokens of a small layer, FP32 rows, added to the shared expert's output
        dict(name="combine 5x1792 f32", op="combine", T=5, H=1792, E=12, k=4, all=12, align=1, type="f32",
             residual=True, grad=False),
        # the prefill layer's batch as a training step has it: output, then the gradients of rows and weights
        dict(name="combine 8192x4096 + grad", op="combine", T=8192, H=4096, E=48, k=6, all=48, align=1, type="bf16",
             residual=False, grad=True),
        # a projection for one new token
        dict(name="linear 1x4096x4096 silu", op="linear", M=1, N=4096, K=4096, ld=4096, type="bf16", out="bf16",
             act="silu", bias=True, residual=True),
        # a short prompt with a ragged row count and ragged sizes, rows inside a wider buffer, FP32 output
        dict(name="linear 300x1000x3600 f16 gelu", op="linear", M=300, N=1000, K=3600, ld=3840, type="f16", out="f32",
             act="gelu", bias=True, residual=False),
        # a projection of a prefill batch, added to the hidden states
        dict(name="linear 8192x4096x4096", op="linear", M=8192, N=4096, K=4096, ld=4096, type="bf16", out="bf16",
             act="none", bias=True, residual=True),
        # the gradients of the dense linear of the package's own benchmark
        dict(name="linear grad 2048x6144x3584 gelu_tanh", op="linear_grad", M=2048, N=6144, K=3584, ld=3584,
             type="bf16", act="gelu_tanh", bias=True),
        # gate and up products of the decode layer for a handful of users
        dict(name="experts 8 tokens", op="expert", T=8, E=32, k=6, all=32, K=4096, N=2048, type="bf16", act="swiglu",
             bias=False),
        # gate and up products of the prefill layer
        dict(name="experts 8192 tokens", op="expert", T=8192, E=48, k=6, all=48, K=4096, N=2048, type="bf16",
             act="swiglu", bias=False),
        # their gradients in a training step of a smaller batch
        dict(name="experts grad 2049 tokens", op="expert_grad", T=2049, E=32, k=6, all=32, K=4096, N=2048, type="bf16",
             act="swiglu", bias=True),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step - 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(("sort", "combine", "linear", "linear_grad", "expert", "expert_grad"))
    if op in ("sort", "combine"):
        H = _log(rng, 64, 8192, 8)
        E = _log(rng, 2, 48)
        k = rng.randint(1, min(8, E))
        T = _log(rng, 1, min(16384, 8192 * 4096 * 6 // (H * k)))
        case = dict(op=op, T=T, H=H, E=E, k=k, all=E * rng.choice((1, 1, 2)), align=rng.choice((1, 1, 16, 128)),
                    type=rng.choice(("bf16", "f16", "bf16" if T * H * k > 1 << 26 else "f32")),
                    grad=rng.random() < 0.5)
        case.update(dict(ld=H + rng.choice((0, 0, 8, 256))) if op == "sort" else dict(residual=rng.random() < 0.5))
        return case
    if op in ("linear", "linear_grad"):
        N, K = _log(rng, 32, 6144, 8), _log(rng, 64, 6144, 8)
        most = (8192 if op == "linear" else 2730) * 4096 * 4096 // (N * K)
        case = dict(op=op, M=_log(rng, 1, min(8192, most)), N=N, K=K, ld=K + rng.choice((0, 0, 8, 256)),
                    type=rng.choice(("bf16", "f16")), act=rng.choice(ACTS[:5]), bias=rng.random() < 0.5)
        if op == "linear":
            case.update(out=rng.choice((case["type"], "f32")), residual=rng.random() < 0.5)
        return case
    E = _log(rng, 2, 48)
    k = rng.randint(1, min(8, E))
    N, K = _log(rng, 64, 2048, 8), _log(rng, 64, 4096, 8)
    return dict(op=op, T=_log(rng, 1, (8192 if op == "expert" else 2049) * 6 // k), E=E, k=k,
                all=E * rng.choice((1, 1, 2)), K=K, N=N, type=rng.choice(("bf16", "f16")), act=rng.choice(ACTS),
                bias=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs


def _activations(g, rows, cols, dtype):
    """Hidden states: N(0, 1) with rows of different magnitude and a few strong channels."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    strong = torch.rand(cols, generator=g, device="cuda") < 0.02
    x *= torch.where(strong, 5.0, 1.0)
    return x.to(dtype)


def _strided(x, ld):
    """x as the leading columns of a buffer with `ld` columns."""
    if ld == x.shape[1]:
        return x
    buf = torch.zeros(x.shape[0], ld, dtype=x.dtype, device=x.device)
    buf[:, :x.shape[1]] = x
    return buf[:, :x.shape[1]]


def _ids(g, case):
    """The model router's choice among all its experts, some of them more popular than others."""
    T, k, n = case["T"], case["k"], case["all"]
    logits = torch.randn(T, n, generator=g, device="cuda") + 0.5 * torch.randn(1, n, generator=g, device="cuda")
    return logits.sort(dim=1, descending=True).indices[:, :k].to(torch.int32).contiguous()


def _capacity(case):
    n = case["T"] * case["k"]
    return n + min(n, case["E"]) * (case.get("align", 1) - 1)


def _plan(case, ids):
    """Where the rows lie: offsets, counts, source (assignment of a row, -1: none), inverse (row of an assignment)."""
    E, align, n = case["E"], case.get("align", 1), ids.numel()
    e = ids.view(-1).long() - _start(case)
    e = torch.where((e >= 0) & (e < E), e, E)
    order = e.sort(stable=True)
    counts = (e[:, None] == torch.arange(E, device=e.device)).sum(0)
    padded = (counts + align - 1) // align * align
    ends, dense = padded.cumsum(0), torch.nn.functional.pad(counts.cumsum(0), (1, 0))
    offsets = torch.nn.functional.pad(ends, (1, 0))
    at = torch.arange(n, device=e.device)
    row = torch.where(order.values < E, at - dense[order.values.clamp(max=E)] + offsets[order.values.clamp(max=E)], -1)
    inverse = torch.empty_like(row)
    inverse[order.indices] = row
    size = _capacity(case)
    source = torch.full((size + 1,), -1, dtype=torch.int64, device=e.device)
    source[torch.where(row >= 0, row, size)] = order.indices
    return (offsets.to(torch.int32), counts.to(torch.int32), source[:size].to(torch.int32),
            inverse.view(ids.shape).to(torch.int32))


def _start(case):
    return (case["all"] - case["E"]) // 2


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = dict(case)
    dtype = TYPES[case["type"]]
    if "E" in case:
        st["ids"] = _ids(g, case)
        st["start"] = _start(case)
        size = _capacity(case)
    if case["op"] == "sort":
        st["x"] = _strided(_activations(g, case["T"], case["H"], dtype), case["ld"])
        if case["grad"]:
            st["drows"] = _activations(g, size, case["H"], dtype)
        st["rows"] = torch.zeros(size, case["H"], dtype=dtype, device="cuda")  # a buffer that the program keeps
        return st
    if case["op"] in ("linear", "linear_grad"):
        M, N, K = case["M"], case["N"], case["K"]
        st["x"] = _strided(_activations(g, M, K, dtype), case["ld"])
        st["w"] = (torch.randn(N, K, generator=g, device="cuda") / math.sqrt(K)).to(dtype)
        st["b"] = torch.randn(N, generator=g, device="cuda").to(dtype) if case["bias"] else None
        if case["op"] == "linear":
            st["res"] = _activations(g, M, N, dtype) if case["residual"] else None
        else:
            st["z"] = None if case["act"] == "none" else torch.randn(M, N, generator=g, device="cuda").to(dtype)
            st["dy"] = _activations(g, M, N, dtype)
        return st
    if case["op"] == "combine":
        p = torch.rand(case["T"], case["k"], generator=g, device="cuda") + 0.1
        st["p"] = p / p.sum(1, keepdim=True)
        st["rows"] = _activations(g, size, case["H"], dtype)
        st["res"] = _activations(g, case["T"], case["H"], dtype) if case["residual"] else None
        if case["grad"]:
            st["dout"] = _activations(g, case["T"], case["H"], dtype)
            st["drows"] = torch.zeros(size, case["H"], dtype=dtype, device="cuda")
    else:
        E, K, N = case["E"], case["K"], case["N"]
        wide = 2 * N if case["act"] == "swiglu" else N
        st["rows"] = _activations(g, size, K, dtype)
        st["w"] = torch.stack([(torch.randn(wide, K, generator=g, device="cuda") / math.sqrt(K)).to(dtype)
                               for _ in range(E)])
        st["b"] = torch.randn(E, wide, generator=g, device="cuda").to(dtype) if case["bias"] else None
        if case["op"] == "expert":
            st["out"] = torch.zeros(size, N, dtype=dtype, device="cuda")
        else:
            st["z"] = None if case["act"] == "none" else (2 * torch.randn(size, wide, generator=g,
                                                                          device="cuda")).to(dtype)
            st["dy"] = _activations(g, size, N, dtype)
            st["dx"] = torch.zeros(size, K, dtype=dtype, device="cuda")
    # the rows' places, which the sort before has left to the program
    if own:
        from nvfp4_mixture_experts_expert_gb300 import api
        x = torch.zeros(case["T"], 16, dtype=torch.bfloat16, device="cuda")
        st["order"] = api.sort_tokens(x, st["ids"], case["E"], st["start"], case.get("align", 1))[1]
    else:
        st["plan"] = _plan(case, st["ids"])
    return st


# ------------------------------------------------------------------ one pass


def run(st):
    return (_own if own else _plain)[st["op"]](st)


def _act_args(st):
    act = st["act"]
    args = dict(activation=None if act == "none" else act)
    if act == "swiglu":
        args.update(gate_limit=LIMIT, up_limit=LIMIT)
    return args


def _own_sort(st):
    from nvfp4_mixture_experts_expert_gb300 import api
    rows, order = api.sort_tokens(st["x"], st["ids"], st["E"], st["start"], st["align"], out=st["rows"])
    out = dict(rows=rows, offsets=order.offsets, counts=order.counts, source=order.source, inverse=order.inverse)
    if st["grad"]:
        out["dx"] = api.sort_tokens_grad(st["drows"], order)
    return out


def _own_combine(st):
    from nvfp4_mixture_experts_expert_gb300 import api
    out = dict(out=api.combine_tokens(st["rows"], st["p"], st["order"], residual=st["res"]))
    if st["grad"]:
        out["drows"], out["dp"] = api.combine_tokens_grad(st["dout"], st["rows"], st["p"], st["order"],
                                                          out=st["drows"])
    return out


def _own_linear(st):
    from nvfp4_mixture_experts_expert_gb300 import api
    return api.linear(st["x"], st["w"], st["b"], residual=st["res"], out_dtype=TYPES[st["out"]], **_act_args(st))


def _own_linear_grad(st):
    from nvfp4_mixture_experts_expert_gb300 import api
    dx, dw, db = api.linear_grad(st["dy"], st["x"], st["w"], st["z"], bias=st["b"] is not None, **_act_args(st))
    return dict(dx=dx, dw=dw, db=db)


def _own_expert(st):
    from nvfp4_mixture_experts_expert_gb300 import api
    return api.expert_linear(st["rows"], st["w"], st["order"], st["b"], out=st["out"], **_act_args(st))


def _own_expert_grad(st):
    from nvfp4_mixture_experts_expert_gb300 import api
    dx, dw, db = api.expert_linear_grad(st["dy"], st["rows"], st["w"], st["order"], st["z"], bias=st["b"] is not None,
                                        out=st["dx"], **_act_args(st))
    return dict(dx=dx, dw=dw, db=db)


def _plain_sort(st):
    offsets, counts, source, inverse = _plan(st, st["ids"])
    inside = torch.arange(source.numel(), device=source.device) < offsets[-1]
    token = source.clamp(min=0).long() // st["k"]
    rows = torch.where((source >= 0)[:, None], st["x"].float()[token], 0.0)
    torch.where(inside[:, None], rows.to(st["x"].dtype), st["rows"], out=st["rows"])
    out = dict(rows=st["rows"], offsets=offsets, counts=counts, source=source, inverse=inverse)
    if st["grad"]:
        dx = torch.zeros(st["T"], st["H"], device=source.device)
        for j in range(st["k"]):
            at = inverse[:, j].long()
            dx += torch.where((at >= 0)[:, None], st["drows"][at.clamp(min=0)].float(), 0.0)
        out["dx"] = dx.to(st["x"].dtype)
    return out


def _plain_combine(st):
    offsets, _, source, inverse = st["plan"]
    rows, p = st["rows"], st["p"]
    acc = st["res"].float() if st["res"] is not None else torch.zeros(st["T"], st["H"], device=rows.device)
    for j in range(st["k"]):
        at = inverse[:, j].long()
        acc = acc + torch.where((at >= 0)[:, None], p[:, j, None] * rows[at.clamp(min=0)].float(), 0.0)
    out = dict(out=acc.to(rows.dtype))
    if st["grad"]:
        dout = st["dout"].float()
        dp = torch.zeros_like(p)
        for j in range(st["k"]):
            at = inverse[:, j].long()
            dp[:, j] = torch.where(at >= 0, (dout * rows[at.clamp(min=0)].float()).sum(1), 0.0)
        f = source.clamp(min=0).long()
        drows = torch.where((source >= 0)[:, None], p.view(-1)[f, None] * dout[f // st["k"]], 0.0)
        inside = torch.arange(source.numel(), device=source.device) < offsets[-1]
        torch.where(inside[:, None], drows.to(rows.dtype), st["drows"], out=st["drows"])
        out["drows"], out["dp"] = st["drows"], dp
    return out


def _plain_act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "swiglu":
        g, u = z[:, :z.shape[1] // 2].clamp(max=LIMIT), z[:, z.shape[1] // 2:].clamp(-LIMIT, LIMIT)
        return g / (1 + torch.exp(-g)) * u
    return z


def _plain_dz(dy, z, act):
    if act == "none":
        return dy
    if act == "relu":
        return torch.where(z > 0, dy, 0.0)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return dy * s * (1 + z * (1 - s))
    if act == "gelu":
        return dy * (0.5 * (1 + torch.erf(z / math.sqrt(2))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return dy * (0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z))
    n = z.shape[1] // 2
    g, u = z[:, :n].clamp(max=LIMIT), z[:, n:].clamp(-LIMIT, LIMIT)
    s = 1 / (1 + torch.exp(-g))
    dg = torch.where(z[:, :n] <= LIMIT, dy * u * s * (1 + g * (1 - s)), 0.0)
    du = torch.where(z[:, n:].abs() <= LIMIT, dy * g * s, 0.0)
    return torch.cat((dg, du), 1)


def _plain_linear(st):
    z = st["x"].float() @ st["w"].float().T
    if st["b"] is not None:
        z = z + st["b"].float()
    y = _plain_act(z, st["act"])
    if st["res"] is not None:
        y = y + st["res"].float()
    return y.to(TYPES[st["out"]])


def _plain_grad(dy, x, w, z, act):
    dz = _plain_dz(dy.float(), None if z is None else z.float(), act)
    return dz @ w.float(), dz.T @ x.float(), dz.sum(0)


def _plain_linear_grad(st):
    dx, dw, db = _plain_grad(st["dy"], st["x"], st["w"], st["z"], st["act"])
    return dict(dx=dx.to(st["x"].dtype), dw=dw.to(st["w"].dtype), db=db if st["b"] is not None else None)


def _plain_expert(st):
    ends = st["plan"][0].tolist()
    for e in range(st["E"]):
        at = slice(ends[e], ends[e + 1])
        if ends[e] < ends[e + 1]:
            z = st["rows"][at].float() @ st["w"][e].float().T
            if st["b"] is not None:
                z = z + st["b"][e].float()
            st["out"][at] = _plain_act(z, st["act"]).to(st["out"].dtype)
    return st["out"]


def _plain_expert_grad(st):
    ends = st["plan"][0].tolist()
    dw = torch.zeros_like(st["w"])
    db = torch.zeros(st["w"].shape[:2], device=dw.device) if st["b"] is not None else None
    for e in range(st["E"]):
        at = slice(ends[e], ends[e + 1])
        if ends[e] < ends[e + 1]:
            dx, dwe, dbe = _plain_grad(st["dy"][at], st["rows"][at], st["w"][e],
                                       None if st["z"] is None else st["z"][at], st["act"])
            st["dx"][at], dw[e] = dx.to(dw.dtype), dwe.to(dw.dtype)
            if db is not None:
                db[e] = dbe
    return dict(dx=st["dx"], dw=dw, db=db)


_own = {"sort": _own_sort, "combine": _own_combine, "linear": _own_linear, "linear_grad": _own_linear_grad,
        "expert": _own_expert, "expert_grad": _own_expert_grad}
_plain = {"sort": _plain_sort, "combine": _plain_combine, "linear": _plain_linear, "linear_grad": _plain_linear_grad,
          "expert": _plain_expert, "expert_grad": _plain_expert_grad}


# ------------------------------------------------------------------ 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    return {"sort": _exact_sort, "combine": _exact_combine, "linear": _exact_linear, "linear_grad": _exact_linear_grad,
            "expert": _exact_expert, "expert_grad": _exact_expert_grad}[case["op"]](st)


def _exact_places(st):
    """(rows of each expert: a list of their assignments; first rows; row of each assignment), worked out on the host."""
    E, align, members = st["E"], st.get("align", 1), [[] for _ in range(st["E"])]
    flat = st["ids"].cpu().view(-1).tolist()
    for f, e in enumerate(flat):
        if 0 <= e - st["start"] < E:
            members[e - st["start"]].append(f)
    first = [0]
    for m in members:
        first.append(first[-1] + -(-len(m) // align) * align)
    row = [-1] * len(flat)
    for e, m in enumerate(members):
        for i, f in enumerate(m):
            row[f] = first[e] + i
    return members, first, torch.tensor(row, device="cuda").view(st["T"], st["k"])


def _exact_sort(st):
    members, first, row = _exact_places(st)
    source = torch.full((st["rows"].shape[0],), -1, dtype=torch.int32)
    for e, m in enumerate(members):
        source[first[e]:first[e] + len(m)] = torch.tensor(m, dtype=torch.int32)
    rows = torch.zeros(st["rows"].shape, dtype=torch.float64, device="cuda")
    t, j = (row >= 0).nonzero(as_tuple=True)
    rows[row[t, j]] = st["x"].double()[t]
    out = dict(rows=rows, offsets=torch.tensor(first, dtype=torch.int32, device="cuda"),
               counts=torch.tensor([len(m) for m in members], dtype=torch.int32, device="cuda"),
               source=source.cuda(), inverse=row.to(torch.int32))
    if st["grad"]:
        out["dx"] = torch.zeros(st["T"], st["H"], dtype=torch.float64, device="cuda")
        out["dx"].index_add_(0, t, st["drows"][row[t, j]].double())
    return out


def _exact_combine(st):
    _, _, row = _exact_places(st)
    t, j = (row >= 0).nonzero(as_tuple=True)
    out = torch.zeros(st["T"], st["H"], dtype=torch.float64, device="cuda")
    for s in range(0, t.numel(), 8192):
        a, b = t[s:s + 8192], j[s:s + 8192]
        out.index_add_(0, a, st["p"][a, b].double()[:, None] * st["rows"][row[a, b]].double())
    if st["res"] is not None:
        out += st["res"].double()
    result = dict(out=out)
    if st["grad"]:
        drows = torch.zeros(st["rows"].shape, dtype=torch.float64, device="cuda")
        dp = torch.zeros(st["T"], st["k"], dtype=torch.float64, device="cuda")
        for s in range(0, t.numel(), 8192):
            a, b = t[s:s + 8192], j[s:s + 8192]
            d = st["dout"][a].double()
            drows[row[a, b]] = d * st["p"][a, b].double()[:, None]
            dp[a, b] = torch.linalg.vecdot(d, st["rows"][row[a, b]].double())
        result.update(drows=drows, dp=dp)
    return result


def _exact_act(z, act, dy=None):
    """act(z), or with dy its gradient dy * act'(z), in FP64."""
    one = dy is None
    if act == "none":
        return z if one else dy
    if act == "relu":
        return torch.maximum(z, torch.zeros_like(z)) if one else dy * (z > 0)
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s if one else dy * (s + z * s * torch.sigmoid(-z))
    if act == "gelu":
        phi = torch.special.ndtr(z)
        return z * phi if one else dy * (phi + z * torch.exp(-z ** 2 / 2) / (2 * math.pi) ** 0.5)
    if act == "gelu_tanh":  # (1 + tanh(a)) / 2 = sigmoid(2a)
        a2 = 2 * (2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)
        s = torch.sigmoid(a2)
        return z * s if one else dy * (s + z * s * torch.sigmoid(-a2) * 2 * (2 / math.pi) ** 0.5 *
                                       (1 + 0.134145 * z ** 2))
    g, u = z.chunk(2, 1)
    gc, uc = torch.clamp(g, max=LIMIT), torch.clamp(u, -LIMIT, LIMIT)
    s = torch.sigmoid(gc)
    if one:
        return gc * s * uc
    return torch.cat((dy * uc * (s + gc * s * torch.sigmoid(-gc)) * (g <= LIMIT), dy * gc * s * (u.abs() <= LIMIT)), 1)


def _exact_product(x, w, b, act):
    z = torch.mm(x.double(), w.double().t())
    return _exact_act(z if b is None else z + b.double(), act)


def _exact_gradients(dy, x, w, z, act):
    dz = _exact_act(None if z is None else z.double(), act, dy.double())
    return torch.mm(dz, w.double()), torch.mm(dz.t(), x.double()), dz.sum(0)


def _exact_linear(st):
    y = _exact_product(st["x"], st["w"], st["b"], st["act"])
    return y if st["res"] is None else y + st["res"].double()


def _exact_linear_grad(st):
    dx, dw, db = _exact_gradients(st["dy"], st["x"], st["w"], st["z"], st["act"])
    return dict(dx=dx, dw=dw, db=db if st["b"] is not None else None)


def _exact_expert(st):
    members, first, _ = _exact_places(st)
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    for e, m in enumerate(members):
        at = slice(first[e], first[e] + len(m))
        out[at] = _exact_product(st["rows"][at], st["w"][e], None if st["b"] is None else st["b"][e], st["act"])
    return out


def _exact_expert_grad(st):
    members, first, _ = _exact_places(st)
    dx = torch.zeros(st["dx"].shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros(st["w"].shape, dtype=torch.float64, device="cuda")
    db = torch.zeros(st["w"].shape[:2], dtype=torch.float64, device="cuda")
    for e, m in enumerate(members):
        at = slice(first[e], first[e] + len(m))
        dx[at], dw[e], db[e] = _exact_gradients(st["dy"][at], st["rows"][at], st["w"][e],
                                                None if st["z"] is None else st["z"][at], st["act"])
    return dict(dx=dx, dw=dw, db=db if st["b"] is not None else None)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    size = 4 if case["type"] == "f32" else 2
    if case["op"] in ("sort", "combine"):
        T, H, E, k = (case[n] for n in ("T", "H", "E", "k"))
        here = T * k * E // case["all"]
        slots = here + min(here, E) * (case["align"] - 1) // 2
        if case["op"] == "sort":
            moved = T * H + slots * H + ((here + T) * H if case["grad"] else 0)
            return {"bytes": moved * size + 4 * (2 * T * k + slots + 2 * E), "flops": here * H if case["grad"] else 0}
        moved = here * H + T * H * (2 if case["residual"] else 1)
        if case["grad"]:  # the rows are read once more, after dout has come
            moved += T * H + here * H + slots * H
        return {"bytes": moved * size + (24 if case["grad"] else 8) * T * k,
                "flops": here * H * (5 if case["grad"] else 2)}
    K, N = case["K"], case["N"]
    if case["op"] in ("linear", "linear_grad"):
        rows, wide, mats = case["M"], N, 1
    else:
        rows = case["T"] * case["k"] * case["E"] // case["all"]
        wide = 2 * N if case["act"] == "swiglu" else N
        mats = case["E"] * (1 - (1 - case["k"] / case["all"]) ** case["T"])  # experts that have rows
    if case["op"].endswith("grad"):
        z = 0 if case["act"] == "none" else rows * wide
        return {"bytes": int(2 * (rows * N + z + 2 * rows * K + 2 * mats * wide * K)), "flops": 4 * rows * wide * K}
    out = rows * N * (4 if case.get("out") == "f32" else 2) + (2 * rows * N if case.get("residual") else 0)
    return {"bytes": int(2 * (rows * K + mats * wide * K)) + out, "flops": 2 * rows * wide * K}
