"""Plain 64-bit forms of the 8-bit operators and of the balance loss, for the
tests: written from the definitions in include/moe.h, in torch fp64."""
from __future__ import annotations

import math

import torch

BLOCK = 128


def two_to(n: torch.Tensor) -> torch.Tensor:
    """2^n for integers n, exactly."""
    return ((n.to(torch.int64) + 1023) << 52).view(torch.float64)


def scale_bytes(amax: torch.Tensor) -> torch.Tensor:
    """Smallest b >= 0 with amax <= 448 * 2^(b - 127)."""
    m, e = torch.frexp(amax.double())          # amax = m 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    b = e.long() - 9 + (m > 0.875).long() + 127
    return torch.where(amax == 0, torch.zeros_like(b), b).clamp(min=0)


def e4m3(v: torch.Tensor) -> torch.Tensor:
    """Nearest e4m3 value (ties to even) of |v| <= 448; NaN where v is not finite."""
    fin = torch.isfinite(v)
    _, e = torch.frexp(torch.where(fin, v, torch.ones_like(v)))
    ulp = two_to((e.long() - 1).clamp(min=-6) - 3)
    return torch.where(fin, torch.round(v / ulp) * ulp, torch.full_like(v, math.nan))


def quantize_rows(x: torch.Tensor):
    """[R, K] -> (values as e4m3 holds them, before the scale; bytes)."""
    v = x.double().reshape(x.shape[0], -1, BLOCK)
    b = scale_bytes(torch.where(torch.isfinite(v), v.abs(), torch.zeros_like(v)).amax(2))
    return e4m3(v / two_to(b - 127)[:, :, None]).reshape(x.shape), b


def quantize_weights(W: torch.Tensor):
    E, N, K = W.shape
    v = W.double().reshape(E, N // BLOCK, BLOCK, K // BLOCK, BLOCK)
    b = scale_bytes(torch.where(torch.isfinite(v), v.abs(), torch.zeros_like(v)).amax((2, 4)))
    return e4m3(v / two_to(b - 127)[:, :, None, :, None]).reshape(W.shape), b


def rows_value(q, b):
    return q.double() * two_to(b.long() - 127).repeat_interleave(BLOCK, 1)


def matrix_value(q, b):
    s = two_to(b.long() - 127).repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)
    return q.double() * s


def product(x, xs, offsets, W, Ws):
    """(y, sum of |terms|), both fp64 [rows, N]."""
    X = rows_value(x, xs)
    y = torch.zeros((x.shape[0], W.shape[1]), dtype=torch.float64, device=x.device)
    a = torch.zeros_like(y)
    o = offsets.tolist()
    for e in range(len(o) - 1):
        if o[e + 1] > o[e]:
            M = matrix_value(W[e], Ws[e])
            y[o[e]:o[e + 1]] = X[o[e]:o[e + 1]] @ M.T
            a[o[e]:o[e + 1]] = X[o[e]:o[e + 1]].abs() @ M.abs().T
    return y, a


def expert(x, We):
    """One 8-bit expert on fp64 rows of quantised input."""
    g, u = x @ matrix_value(We[0], We[1]).T, x @ matrix_value(We[2], We[3]).T
    h, b = quantize_rows(g * torch.sigmoid(g) * u)
    return rows_value(h, b) @ matrix_value(We[4], We[5]).T


def layer(x, idx, gates, W):
    """Outputs fp64 [T, H] and y [T, k, H] of the routed 8-bit experts."""
    T, k = idx.shape
    xv = rows_value(*quantize_rows(x))
    y = torch.zeros((T, k, x.shape[1]), dtype=torch.float64, device=x.device)
    for e in idx.unique().tolist():
        t, j = (idx == e).nonzero(as_tuple=True)
        y[t, j] = expert(xv[t], [w[e] for w in W])
    return (y * gates.double()[:, :, None]).sum(1), y


def balance(logits, idx, off, coef):
    """Loss as a differentiable fp64 scalar of `logits`, and counts [S, E]."""
    E, k = logits.shape[1], idx.shape[1]
    total = max(1, off[-1] - off[0])
    p = torch.where(torch.isinf(logits).all(1, keepdim=True), torch.zeros_like(logits),
                    torch.softmax(logits, 1))
    loss, counts = logits.new_zeros(()), []
    for a, z in zip(off[:-1], off[1:]):
        c = torch.bincount(idx[a:z].flatten().long(), minlength=E)
        counts.append(c)
        if z > a:
            f = E * c.double() / (k * (z - a))
            loss = loss + (z - a) / total * (f * p[a:z].mean(0)).sum()
    return coef * loss, torch.stack(counts).int()
