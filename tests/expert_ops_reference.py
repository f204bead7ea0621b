"""64-bit references of the token sort and combine, the linear with an epilogue
and the expert linear, with the error bounds their tests hold the kernels to.

Bounds: u32 = 2^-24 is FP32's unit roundoff; rounding to a type is off by half a
step, finfo.eps / 2 relative (and half of the smallest subnormal).  A sum of n
FP32 additions is off by n u32 of the sum of magnitudes.  A tensor-core product
step of 16 may truncate instead of round: 2 u32 of the magnitudes each; joins of
partial sums and the bias are below 40 more."""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


def rounded(ref, tol, dtype):
    """tol, and the rounding of what it allows to dtype."""
    return tol + (ref.abs() + tol) * half_step(dtype) + tiny(dtype)


def check(got, ref, tol):
    assert got.shape == ref.shape, (got.shape, ref.shape)
    d = (got.double() - ref).abs()
    bad = ~(d <= tol)  # a NaN fails
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), float(d[bad][0]), float(tol.expand_as(d)[bad][0]))


# ------------------------------------------------------------------ order


def order(ids, E, start=0, align=1):
    """(offsets, counts, source, inverse) as lists and tensors on the CPU."""
    T, k = ids.shape
    members = [[] for _ in range(E)]
    for f, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e - start < E:
            members[e - start].append(f)
    n = T * k
    offsets, inverse = [0], [-1] * n
    source = [-1] * (n + min(n, E) * (align - 1))
    for m in members:
        for i, f in enumerate(m):
            inverse[f] = offsets[-1] + i
            source[offsets[-1] + i] = f
        offsets.append(offsets[-1] + -(-len(m) // align) * align)
    as_t = lambda v: torch.tensor(v, dtype=torch.int32)
    return as_t(offsets), as_t([len(m) for m in members]), as_t(source), as_t(inverse).view(T, k)


def combine(rows, weights, inverse, residual=None):
    """(out, the sum of magnitudes)."""
    inv = inverse.long()
    out = residual.double() if residual is not None else 0.0
    mag = out.abs() if residual is not None else 0.0
    for j in range(inv.shape[1]):
        w = weights[:, j, None].double() if weights is not None else 1.0
        v = torch.where((inv[:, j] >= 0)[:, None], w * rows.double()[inv[:, j].clamp(min=0)], 0.0)
        out, mag = out + v, mag + v.abs()
    return out, mag


# ------------------------------------------------------------------ linear


def act(z, name, limits=(math.inf, math.inf)):
    if name is None:
        return z
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    g, u = z.chunk(2, 1)
    g, u = g.clamp(max=limits[0]), u.clamp(-limits[1], limits[1])
    return g * torch.sigmoid(g) * u


def linear(x, w, bias, name, residual, limits, out_dtype):
    """(z, its tolerance in FP32, out, its tolerance)."""
    X, W = x.double(), w.double()
    z = X @ W.T + (bias.double() if bias is not None else 0)
    mag = X.abs() @ W.abs().T + (bias.double().abs() if bias is not None else 0)
    dz = mag * ((X.shape[1] / 16 * 2 + 40) * U32)
    y = act(z, name, limits)
    if name == "swiglu":
        (g, u), (dg, du) = z.chunk(2, 1), dz.chunk(2, 1)
        gc, uc = g.clamp(max=limits[0]), u.clamp(-limits[1], limits[1])
        dy = 1.1 * dg * uc.abs() + (gc * torch.sigmoid(gc)).abs() * du + 1.1 * dg * du + 16 * U32 * (y.abs() + U32)
    elif name is None:
        dy = dz
    else:  # slopes up to 1.13; the functions within a few u32 of 1 + |z|
        dy = 1.2 * dz + 16 * U32 * (1 + z.abs()) * (name != "relu")
    if residual is not None:
        y = y + residual.double()
        dy = dy + U32 * (y.abs() + dy)
    return z, dz, y, rounded(y, dy, out_dtype)


def linear_grad(dy, x, w, z, name, limits, dtype, out_dtype=None):
    """((dx, tolerance), (dw, tolerance), (dbias, tolerance)) for dz rounded to dtype."""
    out_dtype = out_dtype or dtype
    D, X, W = dy.double(), x.double(), w.double()
    if name is None:
        dz, err, exact = D, torch.zeros_like(D), D
    else:
        Z = z.double().requires_grad_()
        act(Z, name, limits).backward(D)
        exact = dz = Z.grad
        if name == "relu":
            err = torch.zeros_like(dz)
        else:
            wide = torch.cat((D, D), 1) if name == "swiglu" else D
            other = 1.0
            if name == "swiglu":
                g, u = z.double().chunk(2, 1)
                other = torch.cat((u.clamp(-limits[1], limits[1]).abs(), 1 + 0 * u), 1)
            err = 16 * U32 * wide.abs() * (1 + z.double().abs().clamp(max=1e4)) * other
    rnd = err if name is None else err + (dz.abs() + err) * half_step(dtype) + tiny(dtype)
    top = dz.abs() + rnd
    dx, dw, db = dz @ W, dz.T @ X, exact.sum(0)
    steps = lambda n: (n / 16 * 2 + 40) * U32
    return ((dx, rounded(dx, rnd @ W.abs() + (top @ W.abs()) * steps(W.shape[0]), out_dtype)),
            (dw, rounded(dw, rnd.T @ X.abs() + (top.T @ X.abs()) * steps(X.shape[0]), out_dtype)),
            (db, (err.sum(0) + exact.abs().sum(0) * ((X.shape[0] / 64 + 24) * U32)) + 1e-30))
