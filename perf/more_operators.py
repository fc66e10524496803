"""Cases of training the experts, of their 8-bit activation checkpoints, and of
the bf16 product with an epilogue.

Three operators of the routed mixture-of-experts layer:

  train     the experts' gated feed-forward block y = W_down (silu(W_gate x) *
            (W_up x)) over rows grouped by expert, which also keeps what its
            backward pass needs: the two projections, in bf16, or in 8 bits
            together with x;
  backward  the gradients of that block and of the gated sum of its rows: of
            x, of the gates and of the three matrices;
  product   y[p] = act(x[p] . W[e]^T + bias[e]) + residual[p] over rows grouped
            by expert (one expert: a dense product).

run() computes an operator in its plain form (32-bit torch operations), or,
where `own` is true, through the package's entry points.  exact() restates
each definition in 64 bits.

An 8-bit checkpoint holds rows as 8-bit floating point (e4m3) with one
power-of-two scale per block of 128: byte b stands for 2^(b - 127), the
smallest such power, at least 2^-127, for which no finite value of the block
exceeds 448 times it.  It is returned as the values that it stands for, which
bf16 holds exactly.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = 128


# ---- cases ---------------------------------------------------------------

def listed():
    return [
        # train: the small layer of the tests (latency).
        dict(name="train_64", op="train", T=64, E=16, k=2, H=512, I=256, kept="bf16"),
        # train: a dense block (a shared expert) over one chunk of tokens.
        dict(name="train_dense_8192", op="train", T=8192, E=1, k=1, H=4096, I=2048, kept="bf16"),
        # train: a rank's share of the experts, 8-bit checkpoints.
        dict(name="train_fp8_8192", op="train", T=8192, E=64, k=8, H=4096, I=2048, kept="fp8"),
        # backward: the small layer of the tests, 8-bit checkpoints (latency).
        dict(name="backward_fp8_64", op="backward", T=64, E=16, k=2, H=512, I=256, kept="fp8"),
        # backward: ragged groups of a layer of middle size, an odd token count.
        dict(name="backward_1999", op="backward", T=1999, E=32, k=4, H=2048, I=1024, kept="bf16"),
        # backward: the dense block, one chunk of tokens, 8-bit checkpoints.
        dict(name="backward_dense_fp8_8192", op="backward", T=8192, E=1, k=1, H=4096, I=2048, kept="fp8"),
        # backward: the benchmark's prefill chunk over all of its experts.
        dict(name="backward_16384", op="backward", T=16384, E=384, k=8, H=4096, I=2048, kept="bf16"),
        # product: one token through one matrix (latency, bandwidth).
        dict(name="product_1", op="product", rows=1, E=1, N=4096, K=4096, act="silu", bias=True, residual=True, out="bf16"),
        # product: a router's logits with their bias for a decode batch, fp32.
        dict(name="product_router_24", op="product", rows=24, E=1, N=384, K=4096, act="none", bias=True, residual=False, out="fp32"),
        # product: ragged groups of odd sizes, some of them empty.
        dict(name="product_ragged_777", op="product", rows=777, E=48, N=650, K=1160, act="gelu", bias=True, residual=False, out="bf16"),
        # product: odd rows and columns, fp32 result.
        dict(name="product_odd_5001", op="product", rows=5001, E=1, N=1001, K=1000, act="relu", bias=False, residual=True, out="fp32"),
        # product: a prefill chunk through one matrix with everything fused.
        dict(name="product_16384", op="product", rows=16384, E=1, N=4096, K=4096, act="silu", bias=True, residual=True, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, step, lo, hi):
    return max(lo, _log(rng, lo, hi) // step * step)


def draw(rng):
    """One more case of the listed ranges: sizes spread over their logarithm."""
    op = rng.choice(["train", "backward", "product"])
    if op == "product":
        return dict(op=op, rows=_log(rng, 1, 16384), E=rng.choice([1, _log(rng, 2, 64)]),
                    N=_log(rng, 16, 4096), K=_mult(rng, 8, 64, 4096),
                    act=rng.choice(["none", "relu", "gelu", "silu"]), bias=rng.random() < 0.7,
                    residual=rng.random() < 0.5, out=rng.choice(["bf16", "bf16", "fp32"]))
    dense = rng.random() < 0.3
    E = 1 if dense else _log(rng, 2, 128)
    return dict(op=op, T=_log(rng, 1, 8192), E=E, k=1 if dense else rng.randint(1, min(8, E)),
                H=_mult(rng, 256, 512, 4096), I=_mult(rng, 256, 256, 2048),
                kept=rng.choice(["bf16", "fp8"]))


# ---- inputs --------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _matrices(E, N, K, g):
    W = torch.empty((E, N, K), dtype=torch.bfloat16, device=DEV)
    step = max(1, (1 << 29) // (N * K))
    for e in range(0, E, step):   # in parts, to bound the temporary memory
        W[e:e + step] = torch.randn((min(step, E - e), N, K), generator=g, device=DEV).mul_(K ** -0.5)
    return W


def _skewed(T, E, skew, g):
    """Router logits with expert popularity falling off like rank^-skew."""
    rank = torch.randperm(E, generator=g, device=DEV).float() + 1.0
    return torch.randn((T, E), generator=g, device=DEV) - skew * torch.log(rank)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case, kept={})
    if case["op"] == "product":
        rows, E, N, K = (case[n] for n in ("rows", "E", "N", "K"))
        s["x"] = torch.randn((rows, K), generator=g, device=DEV).to(torch.bfloat16)
        s["W"] = _matrices(E, N, K, g)
        s["bias"] = torch.randn((E, N), generator=g, device=DEV) if case["bias"] else None
        s["residual"] = (torch.randn((rows, N), generator=g, device=DEV).to(torch.bfloat16)
                         if case["residual"] else None)
        counts = torch.bincount(_skewed(rows, E, 1.1, g).argmax(1), minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["groups"] = s["offsets"].tolist()      # the caller's own copy on the host
        return s
    T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
    s["W"] = (_matrices(E, I, H, g), _matrices(E, I, H, g), _matrices(E, H, I, g))
    x = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
    logits = _skewed(T, E, 0.5, g)
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    idx = order.indices[:, :k]
    counts = torch.bincount(idx.flatten(), minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    perm = torch.sort(idx.flatten(), stable=True).indices
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(T * k, device=DEV)
    s["groups"] = offsets.tolist()               # the caller's own copy on the host
    s["offsets"], s["perm"], s["inv"] = (v.to(torch.int32) for v in (offsets, perm, inv))
    s["x"] = x
    if case["op"] == "train":
        return s
    s["gates"] = torch.softmax(order.values[:, :k], dim=1).contiguous() if E > 1 else None
    s["d_out"] = (torch.randn((T, H), generator=g, device=DEV) * 1e-2).to(torch.bfloat16)
    # the projections of such x and matrices, as a forward pass kept them
    kept = [x] + [torch.randn((T * k, I), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]
    if case["kept"] == "fp8":
        kept = [p for v in kept for p in _quantize_rows(v.float())]
        s["x"] = None
    s["saved"] = kept
    return s


# ---- plain forms -----------------------------------------------------------

def _pow2(b):
    """2^(b - 127) for bytes b, exactly: the exponent field of an fp32 number
    (2^-127 is subnormal)."""
    b = b.to(torch.int32)
    return torch.where(b > 0, b << 23, 1 << 22).view(torch.float32)


def _quantize_rows(x):
    """fp32 [R, K] -> codes [R, K], bytes [R, K/128]."""
    v = x.view(x.shape[0], -1, BLOCK)
    bits = torch.where(torch.isfinite(v), v.abs(), 0.0).amax(2).view(torch.int32)
    up = ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)     # 448 = 1.75 * 2^8
    b = ((bits >> 23) - 8 + up).clamp(min=0)
    return (v / _pow2(b)[:, :, None]).to(torch.float8_e4m3fn).view(x.shape), b.to(torch.uint8)


def _rows_value(q, b):
    return (q.float().view(q.shape[0], -1, BLOCK) * _pow2(b)[:, :, None]).view(q.shape)


def _held(v, kept):
    """fp32 rows as a checkpoint of that kind stands for them."""
    return (_rows_value(*_quantize_rows(v)) if kept == "fp8" else v).to(torch.bfloat16)


def _plain_block(x, Wg, Wu, Wd):
    g = x @ Wg.float().t()
    u = x @ Wu.float().t()
    return (g / (1 + torch.exp(-g)) * u) @ Wd.float().t(), g, u


def _plain_train(s):
    k, kept, at = s["case"]["k"], s["case"]["kept"], s["groups"]
    x = s["x"].float()
    xs = x[s["perm"].long() // k]
    # one expert after the other, those that hold rows
    parts = [_plain_block(xs[at[e]:at[e + 1]], *(m[e] for m in s["W"]))
             for e in range(len(at) - 1) if at[e + 1] > at[e]]
    y, g, u = (torch.cat(p) for p in zip(*parts))
    return (y.to(torch.bfloat16), _held(g, kept), _held(u, kept)) + ((_held(x, kept),) if kept == "fp8" else ())


def _plain_block_grad(x, d, w, g, u, Wg, Wu, Wd, d_xs, dWg, dWu, dWd):
    """One expert's gradients, written into the last four; returns d_gates."""
    sg = 1 / (1 + torch.exp(-g))
    h = g * sg * u
    dh = d @ Wd.float()
    d_gate = (dh * h).sum(1)
    dh = dh * w
    du = dh * g * sg
    dg = dh * u * sg * (1 + g * (1 - sg))
    d_xs.copy_(dg @ Wg.float() + du @ Wu.float())
    dWg.copy_(dg.t() @ x)
    dWu.copy_(du.t() @ x)
    dWd.copy_((d * w).t() @ h)
    return d_gate


def _plain_backward(s):
    T, k, at = s["case"]["T"], s["case"]["k"], s["groups"]
    if s["case"]["kept"] == "fp8":
        x, g, u = (_rows_value(*s["saved"][i:i + 2]) for i in (0, 2, 4))
    else:
        x, g, u = (v.float() for v in s["saved"])
    slot, inv = s["perm"].long(), s["inv"].long()
    xs, ds = x[slot // k], s["d_out"].float()[slot // k]
    w = s["gates"].flatten()[slot][:, None] if s["gates"] is not None else torch.ones((T * k, 1), device=DEV)
    d_xs = torch.empty_like(xs)
    dW = tuple(torch.zeros_like(m) for m in s["W"])
    # one expert after the other, those that hold rows
    d_gates = torch.cat([_plain_block_grad(*(v[at[e]:at[e + 1]] for v in (xs, ds, w, g, u)), *(m[e] for m in s["W"]),
                                           d_xs[at[e]:at[e + 1]], *(m[e] for m in dW))
                         for e in range(len(at) - 1) if at[e + 1] > at[e]])
    d_x = d_xs[inv].view(T, k, -1).sum(1).to(torch.bfloat16)
    return d_x, d_gates[inv].view(T, k) if s["gates"] is not None else None, *dW


def _plain_act(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    return v / (1 + torch.exp(-v)) if act == "silu" else v


def _plain_product(s):
    c, x, at = s["case"], s["x"].float(), s["groups"]
    # one matrix product per expert that holds rows: the groups are ragged
    y = torch.cat([x[at[e]:at[e + 1]] @ s["W"][e].float().t() + (s["bias"][e] if c["bias"] else 0.0)
                   for e in range(len(at) - 1) if at[e + 1] > at[e]])
    y = _plain_act(y, c["act"])
    if c["residual"]:
        y = y + s["residual"].float()
    return y.to(torch.bfloat16) if c["out"] == "bf16" else y


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"train": _plain_train, "backward": _plain_backward, "product": _plain_product}[op](s)
    import routed_expert_ffn_02_gb300 as moe
    kept = s["kept"]
    if op == "product":
        if not kept:      # the workspace that a program keeps between calls
            kept["ws"] = moe.Workspace(moe.grouped_gemm_workspace_size(*(case[n] for n in ("rows", "E", "N", "K"))))
        return moe.moe_grouped_gemm(s["x"], s["W"], s["offsets"] if case["E"] > 1 else None, bias=s["bias"],
                                    activation=case["act"], residual=s["residual"],
                                    out_dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32,
                                    ws=kept["ws"])
    if not kept:
        kept["shape"] = moe.Shape(*(case[n] for n in ("T", "E", "k", "H", "I")))
        size = moe.expert_ffn_train_workspace_size if op == "train" else moe.expert_ffn_backward_workspace_size
        kept["ws"] = moe.Workspace(size(kept["shape"]))
    routed = case["E"] > 1       # a dense block has no route lists
    perm, offsets = (s["perm"], s["offsets"]) if routed else (None, None)
    if op == "train":
        y, saved = moe.moe_expert_ffn_train(kept["shape"], s["x"], perm, offsets, *s["W"], checkpoint=case["kept"],
                                            ws=kept["ws"])
        if case["kept"] == "bf16":
            return y, saved.gate, saved.up
        return (y, moe.moe_dequantize_rows(saved.gate, saved.gate_scales),
                moe.moe_dequantize_rows(saved.up, saved.up_scales), moe.moe_dequantize_rows(saved.x, saved.x_scales))
    names = ("x", "x_scales", "gate", "gate_scales", "up", "up_scales") if case["kept"] == "fp8" else ("x", "gate", "up")
    if "saved" not in kept:      # the forward pass's record
        kept["saved"] = moe.SavedFfn(**dict(zip(names, s["saved"])))
    return moe.moe_expert_ffn_backward(kept["shape"], s["d_out"], kept["saved"], perm, offsets, s["inv"] if routed else None,
                                       *s["W"], gates=s["gates"], ws=kept["ws"])


# ---- work --------------------------------------------------------------------

def _touched(P, E, skew):
    """Experts that hold slots, expected for P independent slots of that skew."""
    w = np.arange(1, E + 1, dtype=np.float64) ** -skew
    w /= w.sum()
    return float((1 - np.exp(P * np.log1p(-np.minimum(w, 1 - 1e-12)))).sum())


def work(case):
    if case["op"] == "product":
        rows, E, N, K = (case[n] for n in ("rows", "E", "N", "K"))
        out = rows * N * ((4 if case["out"] == "fp32" else 2) + (2 if case["residual"] else 0))
        W = _touched(rows, E, 1.1)
        return {"bytes": W * (2 * N * K + (4 * N if case["bias"] else 0)) + 2 * rows * K + out, "flops": 2 * rows * N * K}
    T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
    P, fp8 = T * k, case["kept"] == "fp8"
    one = 1 + 1 / BLOCK if fp8 else 2                # bytes of a kept value
    touched = max(min(k, E), min(E, _touched(P, E, 0.5)))
    W, lists = 6 * touched * H * I, 4 * P if E > 1 else 0
    if case["op"] == "train":
        return {"bytes": W + 2 * T * H + (one * T * H if fp8 else 0) + 2 * one * P * I + 2 * P * H + lists,
                "flops": 6 * P * H * I}
    return {"bytes": W + 6 * E * H * I + one * (T * H + 2 * P * I) + 4 * T * H + 4 * lists, "flops": 12 * P * H * I}


# ---- the definitions in 64 bits ----------------------------------------------

def _two_to(n):
    """2^n in fp64 for whole numbers n, exactly."""
    return ((n.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_held(x):
    """fp64 rows as an 8-bit checkpoint stands for them, by its definition."""
    v = x.reshape(x.shape[0], -1, BLOCK)
    m, e = torch.frexp(v.abs().amax(2, keepdim=True))
    s = (e.to(torch.int64) - 9 + (m > 0.875).to(torch.int64))    # amax = m 2^e <= 448 * 2^s
    s = _two_to(torch.where(m == 0, torch.full_like(s, -127), s).clamp(min=-127))
    # e4m3: 3 bits after the leading one, the smallest exponent is -6
    _, ve = torch.frexp(v / s)
    ulp = _two_to((ve.to(torch.int64) - 1).clamp(min=-6) - 3) * s
    return (torch.round(v / ulp) * ulp).reshape(x.shape)


def _exact_values(q, b):
    return q.double() * _two_to(b.to(torch.int64) - 127).repeat_interleave(BLOCK, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "product":
        x, off = s["x"].double(), s["offsets"].cpu().numpy()
        y = torch.empty((case["rows"], case["N"]), dtype=torch.float64, device=DEV)
        for e in np.flatnonzero(np.diff(off)):
            r = slice(int(off[e]), int(off[e + 1]))
            y[r] = torch.matmul(x[r], s["W"][e].double().T)
            if case["bias"]:
                y[r] += s["bias"][e].double()
        if case["act"] == "relu":
            y = torch.maximum(y, torch.zeros_like(y))
        elif case["act"] == "gelu":      # v times the normal distribution's mass below v
            y *= torch.special.ndtr(y)
        elif case["act"] == "silu":
            y *= torch.sigmoid(y)
        return y + s["residual"].double() if case["residual"] else y
    T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
    if (6 if case["op"] == "train" else 12) * T * k * H * I > 8e12:      # over about 20 seconds in 64 bits
        return None
    off, slot = s["offsets"].cpu().numpy(), s["perm"].long()
    token = torch.div(slot, k, rounding_mode="floor")
    filled = [(e, slice(int(off[e]), int(off[e + 1]))) for e in np.flatnonzero(np.diff(off))]
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device=DEV)  # noqa: E731
    if case["op"] == "train":
        x = s["x"].double()
        y, g, u = new(T * k, H), new(T * k, I), new(T * k, I)
        for e, r in filled:
            Wg, Wu, Wd = (m[e].double() for m in s["W"])
            g[r], u[r] = x[token[r]] @ Wg.T, x[token[r]] @ Wu.T
            y[r] = (g[r] * torch.sigmoid(g[r]) * u[r]) @ Wd.T
        return (y, _exact_held(g), _exact_held(u), _exact_held(x)) if case["kept"] == "fp8" else (y, g, u)
    x, g, u = ([_exact_values(*s["saved"][i:i + 2]) for i in (0, 2, 4)] if case["kept"] == "fp8"
               else [v.double() for v in s["saved"]])
    d_out = s["d_out"].double()
    gates = s["gates"].double() if s["gates"] is not None else new(T, k) + 1
    d_x, d_gates = new(T, H), new(T * k)
    dW = tuple(new(*m.shape) for m in s["W"])
    for e, r in filled:
        Wg, Wu, Wd = (m[e].double() for m in s["W"])
        d, w, ge, ue = d_out[token[r]], gates.flatten()[slot[r]], g[r], u[r]
        act, slope = ge * torch.sigmoid(ge), torch.sigmoid(ge) + ge * torch.sigmoid(ge) * torch.sigmoid(-ge)
        per_h = d @ Wd
        d_gates[slot[r]] = torch.einsum("ri,ri->r", per_h, act * ue)
        per_h = torch.einsum("ri,r->ri", per_h, w)
        d_g, d_u = per_h * ue * slope, per_h * act
        d_x.index_add_(0, token[r], d_g @ Wg + d_u @ Wu)
        dW[0][e], dW[1][e] = d_g.T @ x[token[r]], d_u.T @ x[token[r]]
        dW[2][e] = torch.einsum("rh,r->rh", d, w).T @ (act * ue)
    return d_x, d_gates.view(T, k) if s["gates"] is not None else None, *dW
