"""64-bit references of the FFN-block operators (norm with FP8 output, FP8
linear, few-token MoE layer) and the error bounds their tests hold them to.

Bounds: u32 = 2^-24 is FP32's unit roundoff, bf16 rounds within 2^-8 relative
(half a step of 7 bits at the bottom of a binade), E4M3 within 2^-4 relative or
2^-10 absolute.  A tensor-core product step may truncate instead of round: one
step costs at most 2 u32 of the sum of magnitudes."""
from __future__ import annotations

import torch

U32 = 2.0 ** -24
BF16 = 2.0 ** -8
MIN_AMAX = 2.0 ** -40


def norm(x, res, w, eps):
    """(s, y, scale, y / scale) in FP64; the last two per blocks of 128 columns."""
    s = x.double() + (res.double() if res is not None else 0)
    y = s / torch.sqrt((s * s).mean(1, keepdim=True) + eps) * w.double()
    H = y.shape[1]
    cols = torch.arange(H, device=y.device) // 128
    scale = torch.stack([y[:, cols == c].abs().amax(1) for c in range(int(cols[-1]) + 1)], 1)
    scale = scale.clamp_min(MIN_AMAX) / 448
    return s, y, scale, y / scale[:, cols]


def linear(a, a_scale, w, w_scale):
    """The product in FP64 and the same sum of magnitudes."""
    K, N = a.shape[1], w.shape[0]
    k = torch.arange(K, device=a.device) // 128
    n = torch.arange(N, device=a.device) // 128
    A = a.float().double() * a_scale.double()[:, k]
    W = w.float().double() * w_scale.double()[n][:, k]
    return A @ W.T, A.abs() @ W.abs().T


def decode_nvfp4(packed, sf, gs, rows, cols):
    """FP64 values of one expert's packed matrix (128 x 4 scale tiles)."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64,
                         device=packed.device)
    b = packed.reshape(rows, cols // 2).long()
    v = torch.stack((table[b & 15], table[b >> 4]), 2).reshape(rows, cols)
    r = torch.arange(rows, device=packed.device)[:, None]
    c = torch.arange(cols // 16, device=packed.device)[None, :]
    at = ((r // 128) * (cols // 64) + c // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + c % 4
    s = sf.reshape(-1).view(torch.float8_e4m3fn)[at].float().double()
    return v * s.repeat_interleave(16, 1) / gs.double()


def route(logits, k):
    """(ids, p) of the routing; p = 0 where the logit is -inf."""
    top = logits.double().sort(dim=1, descending=True, stable=True)
    v, ids = top.values[:, :k], top.indices[:, :k]
    z = torch.where(torch.isinf(v) & (v < 0), 0.0, torch.exp(v - v[:, :1]))
    total = z.sum(1, keepdim=True)
    return ids, torch.where(total > 0, z / total.clamp_min(1e-300), 0.0)


def moe(x, ids, p, w, E, H, I, gate_limit=10.0, up_limit=10.0):
    """The layer in FP64 and a bound on the kernel's error before its rounding to
    bf16.  ids outside [0, E) are not held here."""
    x = x.double()
    out = torch.zeros(x.shape[0], H, dtype=torch.float64, device=x.device)
    tol = torch.zeros_like(out)
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        keep = p[t, j] != 0
        t, j = t[keep], j[keep]
        if not t.numel():
            continue
        w13 = decode_nvfp4(w.w13[e], w.w13_sf[e], w.w13_gs[e], 2 * I, H)
        w2 = decode_nvfp4(w.w2[e], w.w2_sf[e], w.w2_gs[e], H, I)
        g, u = (x[t] @ w13.T).chunk(2, 1)
        # H / 16 product steps in the worst order, then the joins and the scalings
        dg, du = ((x[t].abs() @ w13.abs().T) * ((H / 16 * 2 + 40) * U32)).chunk(2, 1)
        gc, uc = g.clamp(max=gate_limit), u.clamp(-up_limit, up_limit)
        silu = gc * torch.sigmoid(gc)
        h = silu * uc
        dh = 1.1 * uc.abs() * dg + silu.abs() * du + 1.1 * dg * du + h.abs() * (2.0 ** -11 + 16 * U32)
        pt = p[t, j].double()[:, None]
        out.index_add_(0, t, pt * (h @ w2.T))
        tol.index_add_(0, t, pt.abs() * ((dh + h.abs() * ((I / 16 * 2 + 40) * U32)) @ w2.abs().T))
    return out, tol
