"""Measured cases of the operators around the MoE FFN layer: the residual addition with RMSNorm and an FP8 output,
the FP8 block-scaled linear, and the whole MoE layer for a few tokens.

Each operator has a plain form here (elementary torch operations in 32 bits, rounded once at the end), the call a user
makes of the package (`own`), and its definition in 64 bits (`exact`), written apart from the plain form.

  norm    s = x + residual;  y = s * rsqrt(mean(s^2) + eps) * weight;  per 128 columns of a row:
          scale = max(max|y|, 2^-40) / 448,  q = E4M3(y / scale).  Returned: q, scale, bf16(y), bf16(s).
  linear  out[m][n] = sum over blocks c of 128 columns of a_scale[m][c] * w_scale[n / 128][c] * (a . w over the block).
  moe     top_k of the FP32 logits (ties: lower expert), softmax over the chosen;  h = silu(min(g, gate_limit)) *
          clamp(u, +-up_limit) with g, u = W13 x;  out = sum over the chosen of weight * W2 h.  NVFP4 weights
          (E2M1 pairs, one E4M3 scale per 16 columns in the 128 x 4 tile layout, one FP32 scale per expert).
"""
import math

import torch

own = False

EPS = 1e-6
FP8_MAX = 448.0
MIN_AMAX = 2.0 ** -40
GATE_LIMIT = UP_LIMIT = 10.0
BLOCK = 128


def listed():
    return [
        # one new token's hidden state before a layer: latency alone
        dict(name="norm 1x4096", op="norm", T=1, H=4096, ld=4096, residual=True, normed=True, weight="bf16"),
        # an odd batch, rows inside a wider buffer, FP32 norm weights, only the FP8 form wanted
        dict(name="norm 1001x3584 strided", op="norm", T=1001, H=3584, ld=3840, residual=True, normed=False, weight="f32"),
        # the hidden states of a prefill batch
        dict(name="norm 8192x4096", op="norm", T=8192, H=4096, ld=4096, residual=True, normed=True, weight="bf16"),
        # the router of a 48-expert layer for one token, FP32 logits
        dict(name="linear 1x48x4096 f32", op="linear", M=1, N=48, K=4096, ld=4096, out="f32"),
        # a projection of a decode batch
        dict(name="linear 16x4096x4096", op="linear", M=16, N=4096, K=4096, ld=4096, out="bf16"),
        # a short prompt with a ragged row count and ragged output and inner sizes
        dict(name="linear 300x1000x3600", op="linear", M=300, N=1000, K=3600, ld=3840, out="bf16"),
        # the dense linear of the package's own benchmark, FP32 output
        dict(name="linear 2048x6144x3584 f32", op="linear", M=2048, N=6144, K=3584, ld=3584, out="f32"),
        # a projection of a prefill batch
        dict(name="linear 8192x4096x4096", op="linear", M=8192, N=4096, K=4096, ld=4096, out="bf16"),
        # the decode layer of the package's own benchmark for one token
        dict(name="moe 1 token", op="moe", T=1, H=4096, I=2048, E=32, k=6, routed=False),
        # a small odd layer, with the model's router elsewhere and half of its experts here
        dict(name="moe 5 tokens routed", op="moe", T=5, H=1792, I=640, E=12, k=4, routed=True),
        # the same decode layer for a handful of users
        dict(name="moe 8 tokens", op="moe", T=8, H=4096, I=2048, E=32, k=6, routed=False),
        # as many tokens as the operator takes, over the prefill layer's 48 experts
        dict(name="moe 32 tokens", op="moe", T=32, H=4096, I=2048, E=48, k=6, routed=False),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step - 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(("norm", "linear", "moe"))
    if op == "norm":
        H = _log(rng, 128, 8192, 16)
        T = _log(rng, 1, min(8192, 8192 * 4096 // H))
        return dict(op=op, T=T, H=H, ld=H + rng.choice((0, 0, 16, 256)), residual=rng.random() < 0.8,
                    normed=rng.random() < 0.6, weight=rng.choice(("bf16", "f32")))
    if op == "linear":
        N, K = _log(rng, 32, 6144, 8), _log(rng, 128, 6144, 16)
        M = _log(rng, 1, min(8192, 8192 * 4096 * 4096 // (N * K)))
        return dict(op=op, M=M, N=N, K=K, ld=K + rng.choice((0, 0, 16, 256)), out=rng.choice(("bf16", "f32")))
    H, I = _log(rng, 256, 4096, 256), _log(rng, 128, 2048, 128)
    E = _log(rng, 4, 48)
    return dict(op=op, T=_log(rng, 1, 32), H=H, I=I, E=E, k=rng.randint(1, min(8, E)), routed=rng.random() < 0.3)


# ------------------------------------------------------------------ inputs


def _activations(g, rows, cols):
    """Hidden states: N(0, 1) with rows of different magnitude and a few strong channels."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    strong = torch.rand(cols, generator=g, device="cuda") < 0.02
    return torch.where(strong, x * 20, x)


def _strided(x, ld):
    """x as the leading columns of a buffer with `ld` columns."""
    buf = torch.zeros(x.shape[0], ld, dtype=x.dtype, device=x.device)
    buf.view(torch.uint8)[:, :x.shape[1] * x.element_size()] = x.view(torch.uint8)
    return buf[:, :x.shape[1]]


def _fp8_blocks(x, block_rows):
    """E4M3 codes and scales of x in blocks of block_rows x 128."""
    R, C = x.shape
    rb, cb = -(-R // block_rows), -(-C // BLOCK)
    p = torch.zeros(rb * block_rows, cb * BLOCK, device=x.device)
    p[:R, :C] = x
    p = p.view(rb, block_rows, cb, BLOCK)
    scale = p.abs().amax(dim=(1, 3)).clamp_min(MIN_AMAX) / FP8_MAX
    q = (p / scale[:, None, :, None]).clamp(-FP8_MAX, FP8_MAX).view(rb * block_rows, -1)[:R, :C]
    return q.contiguous().to(torch.float8_e4m3fn), scale.contiguous()


def _tile_layout(s):
    """[rows, cols] bytes -> the 128-row x 4-column tile layout, flat."""
    R, C = s.shape
    return s.view(R // 128, 4, 32, C // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _nvfp4(w):
    """NVFP4 of one expert's matrix: packed codes, scales in the tile layout, the global scale."""
    N, K = w.shape
    gs = 2688.0 / w.abs().max()
    b = (w * gs).view(N, K // 16, 16)
    s = (b.abs().amax(-1) / 6).to(torch.float8_e4m3fn)
    d = s.float()
    q = torch.where(d[..., None] > 0, b / d[..., None].clamp_min(1e-3), torch.zeros_like(b)).view(N, K)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    mag = torch.bucketize(q.abs(), edges, out_int32=True).to(torch.uint8)
    code = torch.where((q < 0) & (mag > 0), mag + 8, mag)
    return code[:, 0::2] | (code[:, 1::2] << 4), _tile_layout(s.view(torch.uint8)), gs


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = dict(case)
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        st["x"] = _strided(_activations(g, T, H).bfloat16(), case["ld"])
        st["res"] = _strided(_activations(g, T, H).bfloat16(), case["ld"]) if case["residual"] else None
        w = 1 + 0.1 * torch.randn(H, generator=g, device="cuda")
        st["w"] = w.bfloat16() if case["weight"] == "bf16" else w
    elif case["op"] == "linear":
        a, st["a_scale"] = _fp8_blocks(_activations(g, case["M"], case["K"]), 1)
        st["a"] = _strided(a, case["ld"])
        w = 0.02 * torch.randn(case["N"], case["K"], generator=g, device="cuda")
        st["w"], st["w_scale"] = _fp8_blocks(w, BLOCK)
    else:
        T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
        st["x"] = _activations(g, T, H).bfloat16()
        logits = torch.randn(T, 2 * E if case["routed"] else E, generator=g, device="cuda")
        if case["routed"]:  # the model has 2E experts; [E/2, E/2 + E) of them are here
            top = logits.sort(dim=1, descending=True, stable=True)
            st["start"] = E // 2
            st["ids"] = top.indices[:, :k].to(torch.int32).contiguous()
            st["p"] = torch.softmax(top.values[:, :k], 1)
        else:
            st["logits"] = logits
        up = [_nvfp4((0.02 * torch.randn(2 * I, H, generator=g, device="cuda")).bfloat16().float()) for _ in range(E)]
        down = [_nvfp4((0.02 * torch.randn(H, I, generator=g, device="cuda")).bfloat16().float()) for _ in range(E)]
        st["w13"] = [torch.stack(t) for t in zip(*up)]
        st["w2"] = [torch.stack(t) for t in zip(*down)]
        if own:  # the layer's workspace, kept by the program beside its weights
            from nvfp4_mixture_experts_expert_gb300 import api
            st["layer"] = api.MoEFewTokens(T, H, I, E, k)
            st["weights"] = api.MoEWeights(*st["w13"], *st["w2"])
    return st


# ------------------------------------------------------------------ one pass


def run(st):
    if own:
        return _own(st)
    return {"norm": _plain_norm, "linear": _plain_linear, "moe": _plain_moe}[st["op"]](st)


def _own(st):
    from nvfp4_mixture_experts_expert_gb300 import api
    if st["op"] == "norm":
        q, scale, y, s = api.add_rms_norm_fp8(st["x"], st["res"], st["w"], EPS, normed=st["normed"])
        return dict(q=q, scale=scale, y=y, s=s)
    if st["op"] == "linear":
        dtype = torch.float32 if st["out"] == "f32" else torch.bfloat16
        return api.fp8_linear(st["a"], st["a_scale"], st["w"], st["w_scale"], out_dtype=dtype)
    if st["routed"]:
        return st["layer"].routed(st["x"], st["ids"], st["p"], st["start"], st["weights"], GATE_LIMIT, UP_LIMIT)
    return st["layer"](st["x"], st["logits"], st["weights"], GATE_LIMIT, UP_LIMIT)


def _plain_norm(st):
    T, H = st["T"], st["H"]
    s = st["x"].float()
    if st["res"] is not None:
        s = s + st["res"].float()
    y = s * torch.rsqrt((s * s).mean(1, keepdim=True) + EPS) * st["w"].float()
    cb = -(-H // BLOCK)
    p = torch.nn.functional.pad(y, (0, cb * BLOCK - H)).view(T, cb, BLOCK)
    scale = p.abs().amax(2).clamp_min(MIN_AMAX) / FP8_MAX
    q = (p / scale[:, :, None]).clamp(-FP8_MAX, FP8_MAX).view(T, -1)[:, :H]
    return dict(q=q.to(torch.float8_e4m3fn), scale=scale, y=y.bfloat16() if st["normed"] else None,
                s=s.bfloat16() if st["res"] is not None else None)


def _plain_linear(st):
    M, N, K = st["M"], st["N"], st["K"]
    a = st["a"].float() * st["a_scale"].repeat_interleave(BLOCK, 1)[:, :K]
    w = st["w"].float() * st["w_scale"].repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
    return (a @ w.T).to(torch.float32 if st["out"] == "f32" else torch.bfloat16)


def _decode(packed, sf, gs, which, rows, cols):
    """The FP32 values of the experts `which`: [len(which), rows, cols]."""
    n = which.numel()
    half = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=packed.device)
    pairs = torch.stack((half.repeat(16), half.repeat_interleave(16)), 1)
    v = pairs.index_select(0, packed[which].view(-1).int()).view(n, rows, cols // 16, 16)
    s = sf[which].view(n, rows // 128, cols // 64, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(n, rows, cols // 16)
    s = s.contiguous().view(torch.float8_e4m3fn).float() / gs[which].view(n, 1, 1)
    return (v * s[..., None]).view(n, rows, cols)


def _plain_moe(st):
    T, H, I, E, k = (st[n] for n in ("T", "H", "I", "E", "k"))
    x = st["x"].float()
    if st["routed"]:
        ids = st["ids"].long() - st["start"]
        p = torch.where((ids >= 0) & (ids < E), st["p"], 0.0)
        ids = ids.clamp(0, E - 1)
    else:
        top = st["logits"].sort(dim=1, descending=True, stable=True)
        ids = top.indices[:, :k]
        p = torch.softmax(top.values[:, :k], 1)
    share = torch.zeros(T, E, device=x.device).scatter_add_(1, ids, p)
    which = (share != 0).any(0).nonzero().view(-1)
    gu = x @ _decode(*st["w13"], which, 2 * I, H).transpose(1, 2)  # [experts, T, 2I]
    gate, up = gu[..., :I].clamp(max=GATE_LIMIT), gu[..., I:].clamp(-UP_LIMIT, UP_LIMIT)
    h = gate / (1 + torch.exp(-gate)) * up
    y = h @ _decode(*st["w2"], which, H, I).transpose(1, 2)
    return (share.T[which][..., None] * y).sum(0).bfloat16()


# ------------------------------------------------------------------ 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "linear": _exact_linear, "moe": _exact_moe}[case["op"]](st)


def _exact_norm(st):
    s = st["x"].double()
    if st["res"] is not None:
        s = s + st["res"].double()
    y = s / torch.sqrt(s.pow(2).sum(1) / st["H"] + EPS)[:, None] * st["w"].double()
    parts = [y[:, c:c + BLOCK] for c in range(0, st["H"], BLOCK)]
    tops = [torch.clamp(p.abs().max(dim=1).values, min=MIN_AMAX) for p in parts]
    q = torch.cat([p * (FP8_MAX / t)[:, None] for p, t in zip(parts, tops)], 1)
    return dict(q=q, scale=torch.stack(tops, 1) / FP8_MAX, y=y if st["normed"] else None,
                s=s if st["res"] is not None else None)


def _exact_linear(st):
    out = torch.zeros(st["M"], st["N"], dtype=torch.float64, device="cuda")
    by_row = st["w_scale"].double()[torch.arange(st["N"], device="cuda") // BLOCK]
    for c in range(st["a_scale"].shape[1]):
        cols = slice(c * BLOCK, min(st["K"], (c + 1) * BLOCK))
        part = torch.mm(st["a"][:, cols].float().double(), st["w"][:, cols].float().double().t())
        out += part * st["a_scale"][:, c].double()[:, None] * by_row[:, c][None, :]
    return out


def _exact_matrix(packed, sf, gs, e, rows, cols):
    """One expert's matrix from the formats' definitions, in FP64."""
    b = packed[e].to(torch.int32)
    n = torch.stack((b & 15, b >> 4), 2).view(rows, cols)
    exp, man = ((n >> 1) & 3).double(), (n & 1).double()
    mag = torch.where(exp > 0, torch.exp2(exp - 1) * (1 + man / 2), man / 2)
    v = torch.where(n >= 8, -mag, mag)
    r = torch.arange(rows, device="cuda")[:, None]
    c = torch.arange(cols // 16, device="cuda")[None, :]
    at = ((r // 128) * (cols // 64) + c // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + c % 4
    code = sf[e][at].to(torch.int32)
    se, sm = (code >> 3).double(), (code & 7).double()
    s = torch.where(se > 0, torch.exp2(se - 7) * (1 + sm / 8), sm / 512)
    return v * s.repeat_interleave(16, 1) / gs[e].double()


def _exact_moe(st):
    T, H, I, E, k = (st[n] for n in ("T", "H", "I", "E", "k"))
    if st["routed"]:
        ids, p = st["ids"].long().cpu() - st["start"], st["p"].double().cpu()
    else:
        logits = st["logits"].double().cpu()
        ids = torch.tensor([sorted(range(E), key=lambda e: (-row[e], e))[:k] for row in logits.tolist()])
        z = torch.exp(logits.gather(1, ids) - logits.max(1, keepdim=True).values)
        p = z / z.sum(1, keepdim=True)
    x = st["x"].double()
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        g, u = torch.mm(_exact_matrix(*st["w13"], e, 2 * I, H), x[t.cuda()].t()).chunk(2)
        g, u = torch.clamp(g, max=GATE_LIMIT), torch.clamp(u, -UP_LIMIT, UP_LIMIT)
        y = torch.mm(_exact_matrix(*st["w2"], e, H, I), g * torch.sigmoid(g) * u)
        out.index_add_(0, t.cuda(), (y * p[t, j].cuda()).t())
    return out


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        per = 2 + 1 + (4 if case["residual"] else 0) + (2 if case["normed"] else 0)
        return {"bytes": T * H * per + 4 * T * -(-H // BLOCK) + H * (2 if case["weight"] == "bf16" else 4),
                "flops": 8 * T * H}
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        cb = -(-K // BLOCK)
        return {"bytes": M * K + N * K + 4 * cb * (M + -(-N // BLOCK)) + M * N * (4 if case["out"] == "f32" else 2),
                "flops": 2 * M * N * K}
    T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
    share = k / (2 * E) if case["routed"] else k / E  # of the tokens, that choose a given expert
    active = E * (1 - (1 - share) ** T)
    return {"bytes": int(active * 3 * H * I * 9 / 16) + 4 * T * H + 8 * T * (k if case["routed"] else E),
            "flops": int(6 * T * E * share * H * I)}
