"""Cases of the 8-bit expert operators and of the router's balance loss.

Four operators of the routed mixture-of-experts layer:

  quantize   rows of activations, or expert matrices, to 8-bit floating point
             (e4m3) with one power-of-two scale per block of 128;
  product    y[p] = x[p] . W[e]^T over rows grouped by expert, both operands
             8-bit with block scales, bf16 output;
  layer      the routed layer (route, experts, combine) on 8-bit experts;
  balance    the router's balance loss over packed sequences, its per-expert
             counts, and the gradient of the logits from the loss and from
             the gates.

run() computes an operator in its plain form (32-bit torch operations), or,
where `own` is true, through the package's entry points.  exact() restates
each definition in 64 bits.

Block scales are held as one byte b standing for 2^(b - 127).  A block's
scale is the smallest such power of two, at least 2^-127, for which no finite
value of the block exceeds 448 (the largest e4m3 value) times it; values are
rounded to nearest, ties to even; a value that is not finite becomes NaN.
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
        # quantize: the activations of a decode step of 4 tokens (latency).
        dict(name="quantize_rows_4", op="quantize", what="rows", rows=4, K=4096),
        # quantize: the activations of one prefill chunk.
        dict(name="quantize_rows_16384", op="quantize", what="rows", rows=16384, K=4096),
        # quantize: 64 experts' gate matrices, as a checkpoint is converted.
        dict(name="quantize_weights_64", op="quantize", what="weights", E=64, N=2048, K=4096),
        # product: one token through one dense 8-bit matrix (a shared expert
        # while decoding).
        dict(name="product_dense_1", op="product", rows=1, E=1, N=4096, K=2048, skew=0.0),
        # product: ragged small groups with odd sizes, some of them empty.
        dict(name="product_ragged_777", op="product", rows=777, E=48, N=640, K=1152, skew=1.1),
        # product: a prefill chunk through one dense matrix.
        dict(name="product_dense_16384", op="product", rows=16384, E=1, N=4096, K=4096, skew=0.0),
        # layer: one decode step of one token at full size (latency, bandwidth).
        dict(name="layer_decode_1", op="layer", T=1, E=384, k=8, H=4096, I=2048, skew=1.1),
        # layer: the largest decode batch of the benchmark's sweep.
        dict(name="layer_decode_24", op="layer", T=24, E=384, k=8, H=4096, I=2048, skew=1.1),
        # layer: the benchmark's prefill chunk with its skewed routing.
        dict(name="layer_prefill_16384", op="layer", T=16384, E=384, k=8, H=4096, I=2048, skew=1.1),
        # balance: the small layer of the tests (latency).
        dict(name="balance_64", op="balance", T=64, E=16, k=2, S=1),
        # balance: odd sizes, packed sequences of different lengths, one of
        # them empty, tokens of padding after the last.
        dict(name="balance_packed_5001", op="balance", T=5001, E=1000, k=6, S=7),
        # balance: one prefill-sized chunk as one sequence.
        dict(name="balance_16384", op="balance", T=16384, E=384, k=8, S=1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, step, lo, hi):
    return max(lo, _log(rng, lo, hi) // step * step)


def draw(rng):
    """One more case of the listed ranges: sizes spread over their logarithm."""
    op = rng.choice(["quantize", "product", "layer", "balance"])
    if op == "quantize" and rng.random() < 0.6:
        return dict(op=op, what="rows", rows=_log(rng, 1, 16384), K=_mult(rng, 128, 256, 8192))
    if op == "quantize":
        N, K = _mult(rng, 128, 256, 4096), _mult(rng, 128, 256, 4096)
        return dict(op=op, what="weights", E=_log(rng, 1, max(1, (1 << 29) // (N * K))), N=N, K=K)
    if op == "product":
        E = rng.choice([1, _log(rng, 2, 384)])
        return dict(op=op, rows=_log(rng, 1, 16384), E=E, N=_mult(rng, 128, 256, 4096),
                    K=_mult(rng, 128, 256, 4096), skew=rng.choice([0.0, 0.5, 1.1]))
    if op == "layer":
        E = _log(rng, 8, 384)
        return dict(op=op, T=_log(rng, 1, 16384), E=E, k=rng.randint(1, 8),
                    H=_mult(rng, 256, 512, 4096), I=_mult(rng, 256, 256, 2048),
                    skew=rng.choice([0.0, 0.5, 1.1]))
    T, E = _log(rng, 1, 16384), _log(rng, 8, 1024)
    return dict(op=op, T=T, E=E, k=rng.randint(1, 8), S=rng.randint(1, min(32, T)))


# ---- inputs --------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _codes(shape, g):
    """8-bit expert matrices [E, N, K] as a conversion leaves them: codes of
    normal weights whose block maximum lies in (224, 448], and scales around
    the size of weights of deviation 0.02, differing from block to block."""
    E, N, K = shape
    q = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
    step = max(1, (1 << 29) // (N * K))
    for e in range(0, E, step):   # in parts, to bound the temporary memory
        part = torch.randn((min(step, E - e), N, K), generator=g, device=DEV, dtype=torch.bfloat16)
        q[e:e + step] = part.mul_(82.0).clamp_(-448, 448).to(torch.float8_e4m3fn)
    s = torch.randint(114, 117, (E, N // BLOCK, K // BLOCK), generator=g, device=DEV)
    return q, s.to(torch.uint8)


def _skewed(T, E, skew, g):
    """Router logits with expert popularity falling off like rank^-skew."""
    rank = torch.randperm(E, generator=g, device=DEV).float() + 1.0
    return torch.randn((T, E), generator=g, device=DEV) - skew * torch.log(rank)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case, kept={})
    if op == "quantize":
        if case["what"] == "rows":
            # activations with a few large channels, as trained layers have
            x = torch.randn((case["rows"], case["K"]), generator=g, device=DEV)
            x *= torch.exp(torch.randn((1, case["K"]), generator=g, device=DEV))
            s["x"] = x.to(torch.bfloat16)
        else:
            shape = (case["E"], case["N"], case["K"])
            s["x"] = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16).mul_(0.02)
    elif op == "product":
        rows, E, N, K = (case[n] for n in ("rows", "E", "N", "K"))
        s["q"] = (torch.randn((rows, K), generator=g, device=DEV) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
        s["sq"] = torch.randint(118, 122, (rows, K // BLOCK), generator=g, device=DEV).to(torch.uint8)
        s["W"], s["sW"] = _codes((E, N, K), g)
        e = _skewed(rows, E, case["skew"], g).argmax(1)
        counts = torch.bincount(e, minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["groups"] = s["offsets"].tolist()      # the caller's own copy on the host
    elif op == "layer":
        T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
        s["logits"] = _skewed(T, E, case["skew"], g)
        s["x"] = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
        s["W"] = (*_codes((E, I, H), g), *_codes((E, I, H), g), *_codes((E, H, I), g))
        counts = torch.bincount(s["logits"].topk(k, dim=1).indices.flatten(), minlength=E)
        s["groups"] = [0] + counts.cumsum(0).tolist()
    else:
        T, E, k, S = (case[n] for n in ("T", "E", "k", "S"))
        s["logits"] = _skewed(T, E, 1.1, g)
        idx = torch.sort(s["logits"], dim=1, descending=True, stable=True).indices[:, :k]
        s["idx"] = idx.to(torch.int32).contiguous()
        s["gates"] = torch.softmax(s["logits"].gather(1, idx), dim=1)
        s["d_gates"] = torch.randn((T, k), generator=g, device=DEV) * 1e-3
        s["d_loss"] = torch.rand((), generator=g, device=DEV) + 0.5
        if S == 1:
            off = torch.tensor([0, T], device=DEV)
        else:                                    # packed: one empty, padding at the end
            off = torch.sort(torch.randint(0, T + 1, (S + 1,), generator=g, device=DEV)).values
            off[0] = 0
            off[S // 2 + 1] = off[S // 2]
            off = torch.sort(off).values
        s["off"] = off.to(torch.int32)
        s["coef"] = 1e-2
    return s


# ---- plain forms -----------------------------------------------------------

def _pow2(b):
    """2^(b - 127) for bytes b, exactly: the exponent field of an fp32 number
    (2^-127 is subnormal)."""
    b = b.to(torch.int32)
    return torch.where(b > 0, b << 23, 1 << 22).view(torch.float32)


def _scale_byte(amax):
    """Byte of the smallest power of two >= amax / 448 (fp32 amax, >= 0)."""
    bits = amax.contiguous().view(torch.int32)
    up = ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)     # 448 = 1.75 * 2^8
    return ((bits >> 23) - 8 + up).clamp(min=0)


def _quantize_rows(x):
    """fp32 [R, K] -> codes [R, K], bytes [R, K/128]."""
    v = x.view(x.shape[0], -1, BLOCK)
    b = _scale_byte(torch.where(torch.isfinite(v), v.abs(), 0.0).amax(2))
    return (v / _pow2(b)[:, :, None]).to(torch.float8_e4m3fn).view(x.shape), b.to(torch.uint8)


def _rows_value(q, b):
    return (q.float().view(q.shape[0], -1, BLOCK) * _pow2(b)[:, :, None]).view(q.shape)


def _matrix_value(q, b):
    N, K = q.shape
    v = q.float().view(N // BLOCK, BLOCK, K // BLOCK, BLOCK)
    return (v * _pow2(b)[:, None, :, None]).view(N, K)


def _plain_quantize(s):
    x = s["x"].float()
    if x.dim() == 2:
        return _quantize_rows(x)
    E, N, K = x.shape
    v = x.view(E, N // BLOCK, BLOCK, K // BLOCK, BLOCK)
    b = _scale_byte(torch.where(torch.isfinite(v), v.abs(), 0.0).amax((2, 4)))
    return (v / _pow2(b)[:, :, None, :, None]).to(torch.float8_e4m3fn).view(E, N, K), b.to(torch.uint8)


def _plain_product(s):
    x = _rows_value(s["q"], s["sq"])
    at = s["groups"]
    # one matrix product per expert that holds rows: the groups are ragged
    parts = [x[at[e]:at[e + 1]] @ _matrix_value(s["W"][e], s["sW"][e]).t()
             for e in range(len(at) - 1) if at[e + 1] > at[e]]
    return torch.cat(parts).to(torch.bfloat16)


def _plain_expert(x, Wg, Sg, Wu, Su, Wd, Sd):
    g = x @ _matrix_value(Wg, Sg).t()
    u = x @ _matrix_value(Wu, Su).t()
    h = _rows_value(*_quantize_rows(g / (1 + torch.exp(-g)) * u))
    return h @ _matrix_value(Wd, Sd).t()


def _plain_layer(s):
    k = s["case"]["k"]
    order = torch.sort(s["logits"], dim=1, descending=True, stable=True)
    idx, top = order.indices[:, :k], order.values[:, :k]
    w = torch.exp(top - top[:, :1])
    gates = w / w.sum(1, keepdim=True)
    x = _rows_value(*_quantize_rows(s["x"].float()))
    perm = torch.sort(idx.flatten(), stable=True).indices
    xs = x[perm // k]
    at, W = s["groups"], s["W"]
    # one expert after the other, those that hold slots
    y = torch.cat([_plain_expert(xs[at[e]:at[e + 1]], *(m[e] for m in W))
                   for e in range(len(at) - 1) if at[e + 1] > at[e]])
    slots = torch.empty_like(y)
    slots[perm] = y
    out = (slots.view(-1, k, y.shape[1]) * gates[:, :, None]).sum(1)
    return out.to(torch.bfloat16), idx.to(torch.int32), gates


def _plain_balance(s):
    l, idx, off, k = s["logits"], s["idx"].long(), s["off"].long(), s["case"]["k"]
    T, E = l.shape
    t = torch.arange(T, device=DEV)
    inside = (t[None] >= off[:-1, None]) & (t[None] < off[1:, None])      # [S, T]
    S = inside.shape[0]
    e = torch.exp(l - l.amax(1, keepdim=True))
    p = e / e.sum(1, keepdim=True)
    hot = (idx[:, :, None] == torch.arange(E, device=DEV)).sum(1).float()
    counts = inside.float() @ hot
    n = inside.sum(1).float()
    total = n.sum().clamp(min=1)
    a = s["coef"] * E / (k * total) * counts / n.clamp(min=1)[:, None]     # [S, E]
    loss = (a * (inside.float() @ p)).sum()
    at = inside.float().t() @ a                                            # [T, E], 0 outside
    d = s["d_loss"] * p * (at - (p * at).sum(1, keepdim=True))
    g, dg = s["gates"], s["d_gates"]
    d = d.scatter_add(1, idx, g * (dg - (g * dg).sum(1, keepdim=True)))
    return loss, counts.to(torch.int32), d


def run(s):
    op = s["case"]["op"]
    if not own:
        plain = {"quantize": _plain_quantize, "product": _plain_product,
                 "layer": _plain_layer, "balance": _plain_balance}[op]
        return plain(s)
    import routed_expert_ffn_02_gb300 as moe
    kept, case = s["kept"], s["case"]
    if op == "quantize":
        return (moe.moe_quantize_rows if case["what"] == "rows" else moe.moe_quantize_weights)(s["x"])
    if op == "product":
        if not kept:      # the workspace that a program keeps between calls
            kept["ws"] = moe.Workspace(moe.grouped_gemm_fp8_workspace_size(case["rows"], case["E"]))
        return moe.moe_grouped_gemm_fp8(s["q"], s["sq"], s["offsets"], s["W"], s["sW"], ws=kept["ws"])
    if op == "layer":
        if not kept:
            shape = moe.Shape(*(case[n] for n in ("T", "E", "k", "H", "I")))
            kept.update(shape=shape, experts=moe.Fp8Experts(*s["W"]),
                        ws=moe.Workspace(moe.fp8_workspace_size(shape)))
        idx = torch.empty((case["T"], case["k"]), dtype=torch.int32, device=DEV)
        gates = torch.empty((case["T"], case["k"]), dtype=torch.float32, device=DEV)
        out = moe.moe_forward_fp8(kept["shape"], s["logits"], s["x"], kept["experts"],
                                  topk_idx=idx, gates=gates, ws=kept["ws"])
        return out, idx, gates
    if not kept:
        kept["ws"] = moe.Workspace(moe.balance_workspace_size(case["T"], case["E"], case["S"]))
    loss, counts, stats = moe.moe_balance(s["logits"], s["idx"], s["off"], s["coef"], ws=kept["ws"])
    d = moe.moe_balance_backward(s["logits"], stats, counts, case["k"], s["off"], s["coef"],
                                 s["d_loss"], topk_idx=s["idx"], gates=s["gates"],
                                 d_gates=s["d_gates"])
    return loss, counts, d


# ---- work --------------------------------------------------------------------

def _touched(P, E, skew):
    """Experts that hold slots, expected for P independent slots of that skew."""
    w = np.arange(1, E + 1, dtype=np.float64) ** -skew
    w /= w.sum()
    return float((1 - np.exp(P * np.log1p(-np.minimum(w, 1 - 1e-12)))).sum())


def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["K"] if case["what"] == "rows" else case["E"] * case["N"] * case["K"]
        per = BLOCK if case["what"] == "rows" else BLOCK * BLOCK
        return {"bytes": 3 * n + n / per, "flops": 2 * n}
    if op == "product":
        rows, N, K = case["rows"], case["N"], case["K"]
        W = _touched(rows, case["E"], case["skew"]) * N * K * (1 + BLOCK ** -2)
        return {"bytes": W + rows * K * (1 + 1 / BLOCK) + 2 * rows * N, "flops": 2 * rows * N * K}
    if op == "layer":
        T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
        # a token's experts differ, so one token touches min(k, E) of them
        touched = max(min(k, E), min(E, _touched(T * k, E, case["skew"])))
        W = touched * 3 * H * I * (1 + BLOCK ** -2)
        return {"bytes": W + 4 * T * E + 4 * T * H + 8 * T * k, "flops": 6 * T * k * H * I}
    T, E, k, S = (case[n] for n in ("T", "E", "k", "S"))
    return {"bytes": 8 * T * E + 12 * T * k + 4 * S * E, "flops": 12 * T * E}


# ---- the definitions in 64 bits ----------------------------------------------

def _two_to(n):
    """2^n in fp64 for whole numbers n, exactly."""
    return ((n.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_round(x, whole):
    """(codes' values, bytes) of fp64 x by its definition; `whole`: the axes
    of a block in the blocked view that it comes in."""
    fin = torch.isfinite(x)
    m, e = torch.frexp(torch.where(fin, x.abs(), torch.zeros_like(x)).amax(whole, keepdim=True))
    s = (e.to(torch.int64) - 9 + (m > 0.875).to(torch.int64))    # amax = m 2^e <= 448 * 2^s
    s = torch.where(m == 0, torch.full_like(s, -127), s).clamp(min=-127)
    v = x / _two_to(s)
    # e4m3: 3 bits after the leading one, the smallest exponent is -6
    _, ve = torch.frexp(torch.where(fin, v, torch.ones_like(v)))
    ulp = _two_to((ve.to(torch.int64) - 1).clamp(min=-6) - 3)
    q = torch.round(v / ulp) * ulp
    return torch.where(fin, q, torch.full_like(q, math.nan)), s + 127


def _exact_rows(x):
    q, b = _exact_round(x.double().reshape(x.shape[0], -1, BLOCK), 2)
    return q.reshape(x.shape), b[:, :, 0]


def _wide(q, b):
    """Values of 8-bit codes [.., K] whose bytes b have one entry per block."""
    b = b.to(torch.int64) - 127
    if b.shape[0] != q.shape[0]:
        b = b.repeat_interleave(BLOCK, 0)
    return q.double() * _two_to(b).repeat_interleave(BLOCK, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = s["x"]
        if x.dim() == 2:
            q, b = _exact_rows(x)
            return q, b.to(torch.uint8)
        q = torch.empty(x.shape, dtype=torch.float32, device=DEV)    # e4m3 values are exact in it
        b = torch.empty((x.shape[0], x.shape[1] // BLOCK, x.shape[2] // BLOCK), dtype=torch.uint8, device=DEV)
        for e in range(x.shape[0]):
            blocks = x[e].double().reshape(x.shape[1] // BLOCK, BLOCK, -1, BLOCK)
            qe, be = _exact_round(blocks, (1, 3))
            q[e], b[e] = qe.reshape(x[e].shape).float(), be[:, 0, :, 0].to(torch.uint8)
        return q, b
    if op == "product":
        y = torch.empty((case["rows"], case["N"]), dtype=torch.float64, device=DEV)
        off = s["offsets"].cpu().numpy()
        for e in np.flatnonzero(np.diff(off)):
            rows = slice(int(off[e]), int(off[e + 1]))
            y[rows] = _wide(s["q"][rows], s["sq"][rows]) @ _wide(s["W"][e], s["sW"][e]).T
        return y
    if op == "layer":
        T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
        if 6 * T * k * H * I > 8e12:      # over about 20 seconds in 64 bits
            return None
        l = s["logits"].double().cpu().numpy()
        idx = np.lexsort((np.broadcast_to(np.arange(E), l.shape), -l), axis=1)[:, :k]
        top = np.take_along_axis(l, idx, 1)
        gates = np.exp(top) / np.exp(top).sum(1, keepdims=True)
        x, b = _exact_rows(s["x"])
        x = _wide(x, b)
        out = torch.zeros((T, H), dtype=torch.float64, device=DEV)
        Wg, Sg, Wu, Su, Wd, Sd = s["W"]
        for e in np.unique(idx):
            t, j = np.nonzero(idx == e)
            xe = x[torch.from_numpy(t).to(DEV)]
            g = xe @ _wide(Wg[e], Sg[e]).T
            h = g * torch.sigmoid(g) * (xe @ _wide(Wu[e], Su[e]).T)
            ye = _wide(*_exact_rows(h)) @ _wide(Wd[e], Sd[e]).T
            out[torch.from_numpy(t).to(DEV)] += ye * torch.from_numpy(gates[t, j]).to(DEV)[:, None]
        return out, torch.from_numpy(idx.astype(np.int32)), torch.from_numpy(gates)
    l, idx = s["logits"].double().cpu().numpy(), s["idx"].cpu().numpy()
    off, k, E = s["off"].cpu().numpy(), case["k"], case["E"]
    p = np.exp(l - np.logaddexp.reduce(l, axis=1)[:, None])
    d = np.zeros_like(l)
    counts = np.zeros((len(off) - 1, E), dtype=np.int32)
    total, loss = max(1, int(off[-1] - off[0])), 0.0
    for i in range(len(off) - 1):
        a, z = int(off[i]), int(off[i + 1])
        if z == a:
            continue
        counts[i] = np.bincount(idx[a:z].ravel(), minlength=E)
        f = counts[i] * E / (k * (z - a))
        loss += (z - a) / total * float(f @ p[a:z].mean(0))
        d[a:z] = p[a:z] * (f - (p[a:z] @ f)[:, None]) / total
    d *= s["coef"] * float(s["d_loss"])
    g, dg = s["gates"].double().cpu().numpy(), s["d_gates"].double().cpu().numpy()
    np.add.at(d, (np.arange(len(l))[:, None], idx), g * (dg - (g * dg).sum(1, keepdims=True)))
    return torch.tensor(loss * s["coef"], dtype=torch.float64), torch.from_numpy(counts), torch.from_numpy(d)
