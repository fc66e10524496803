"""Plain 64-bit forms of the experts' training passes and of the product with
an epilogue, for the tests: written from the definitions in include/moe.h."""
from __future__ import annotations

import math

import torch

import fp8_plain

U = 2.0 ** -8          # a rounding to bf16, relative to the value
ADD = 2.0 ** -23       # a sum of K terms is off by at most K ADD times the sum of their magnitudes:
#                        half a step per addition in fp32, twice that for truncating adders


def routing(T, E, k, seed, skew=1.0, device="cpu"):
    """Route lists of a skewed routing: (perm, offsets, inv_perm, gates fp32 [T, k])."""
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn((T, E), generator=g) - skew * torch.log(torch.randperm(E, generator=g) + 1.0)
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    idx = order.indices[:, :k]
    counts = torch.bincount(idx.flatten(), minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    perm = torch.sort(idx.flatten(), stable=True).indices
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(T * k)
    gates = torch.softmax(order.values[:, :k], 1)
    return (*(v.to(torch.int32).to(device) for v in (perm, offsets, inv)), gates.contiguous().to(device))


def groups(offsets, rows):
    if offsets is None:
        return [(0, slice(0, rows))]
    off = offsets.tolist()
    return [(e, slice(off[e], off[e + 1])) for e in range(len(off) - 1) if off[e + 1] > off[e]]


def held(v):
    """fp64 rows as an 8-bit checkpoint stands for them."""
    return fp8_plain.rows_value(*fp8_plain.quantize_rows(v))


def forward(x, tokens, offsets, Wg, Wu, Wd):
    """y, g, u by sorted row, and for each the sum of its terms' magnitudes."""
    P, x = len(tokens), x.double()
    new = lambda n: torch.zeros((P, n), dtype=torch.float64, device=x.device)  # noqa: E731
    I, H = Wg.shape[1:]
    y, g, u, gm, um, ym = new(H), new(I), new(I), new(I), new(I), new(H)
    for e, r in groups(offsets, P):
        a, (wg, wu, wd) = x[tokens[r]], (m[e].double() for m in (Wg, Wu, Wd))
        g[r], u[r] = a @ wg.T, a @ wu.T
        gm[r], um[r] = a.abs() @ wg.abs().T, a.abs() @ wu.abs().T
        h = g[r] * torch.sigmoid(g[r]) * u[r]
        y[r], ym[r] = h @ wd.T, h.abs() @ wd.abs().T
    return dict(y=y, g=g, u=u, g_mag=gm, u_mag=um, y_mag=ym)


def backward(d_out, gates, x, g, u, perm, offsets, k, Wg, Wu, Wd):
    """The gradients, for each the sum of its terms' magnitudes, and the same
    with the magnitudes of q's own terms in the place of q."""
    T, H = d_out.shape
    P, I, E, dev = T * k, Wg.shape[1], Wg.shape[0], d_out.device
    slot = perm.long() if perm is not None else torch.arange(P, device=dev)
    tok = slot // k
    w = gates.double().flatten()[slot][:, None] if gates is not None else torch.ones((P, 1), dtype=torch.float64, device=dev)
    x, g, u, d = x.double()[tok], g.double(), u.double(), d_out.double()[tok]
    new = lambda *s: torch.zeros(s, dtype=torch.float64, device=dev)  # noqa: E731
    r = {n: new(*s) for n, s in dict(d_x=(T, H), d_gates=(P,), dWg=(E, I, H), dWu=(E, I, H), dWd=(E, H, I)).items()}
    m, mq = ({n: torch.zeros_like(v) for n, v in r.items()} for _ in range(2))
    s = torch.sigmoid(g)
    h = g * s * u
    for e, rows in groups(offsets, P):
        wg, wu, wd = (t[e].double() for t in (Wg, Wu, Wd))
        q, qm = d[rows] @ wd, d[rows].abs() @ wd.abs()
        to_u, to_g = w[rows] * g[rows] * s[rows], w[rows] * u[rows] * s[rows] * (1 + g[rows] * (1 - s[rows]))
        du, dg, dum, dgm = q * to_u, q * to_g, qm * to_u.abs(), qm * to_g.abs()
        for to, a in ((r, q * h[rows]), (m, (q * h[rows]).abs()), (mq, qm * h[rows].abs())):
            to["d_gates"][slot[rows]] = a.sum(1)
        for to, a, b, c, v in ((r, dg, du, wg, wu), (m, dg.abs(), du.abs(), wg.abs(), wu.abs()),
                               (mq, dgm, dum, wg.abs(), wu.abs())):
            to["d_x"].index_add_(0, tok[rows], a @ c + b @ v)
        for n, a, b, am in (("dWg", dg, x[rows], dgm), ("dWu", du, x[rows], dum), ("dWd", d[rows], w[rows] * h[rows], None)):
            r[n][e], m[n][e] = a.T @ b, a.abs().T @ b.abs()
            if am is not None:
                mq[n][e] = am.T @ b.abs()
    for to in (r, m, mq):
        to["d_gates"] = to["d_gates"].view(T, k)
    return r, m, mq


def product(x, W, offsets, bias, act, residual):
    """(y, the argument of the activation, the sum of its terms' magnitudes)."""
    x = x.double()
    v = torch.zeros((x.shape[0], W.shape[1]), dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(v)
    for e, r in groups(offsets, x.shape[0]):
        v[r], mag[r] = x[r] @ W[e].double().T, x[r].abs() @ W[e].double().abs().T
        if bias is not None:
            v[r] += bias[e].double()
            mag[r] += bias[e].double().abs()
    y = {"none": lambda: v, "relu": lambda: v.clamp(min=0), "silu": lambda: v * torch.sigmoid(v),
         "gelu": lambda: 0.5 * v * (1 + torch.special.erf(v * math.sqrt(0.5)))}[act]()
    return (y if residual is None else y + residual.double()), v, mag


def rel_rms(got, want):
    got, want = got.double(), want.double()
    n = want.square().sum().sqrt().item()
    d = (got - want).square().sum().sqrt().item()
    return d / n if n else d
