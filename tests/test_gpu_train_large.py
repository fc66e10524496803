"""GPU: the experts' training passes over route lists where buffers hold more
than 2^31 values: sorted and padded rows, kept projections and their scales, the
fp32 parts of d_x, the weights and their gradients.  Sampled tokens and features
against the 64-bit forms, with test_gpu_train's bounds."""
import pytest
import torch

import fp8_plain
import train_plain as plain
from parity import REL_RMS_TOL
from test_gpu_train import Case, check_backward, check_forward, moe  # noqa: F401  (moe: the fixture)

pytestmark = pytest.mark.gpu


def lists(idx, E):
    """(perm, offsets, inv_perm, tokens) of routed experts idx [T, k]."""
    perm = torch.sort(idx.flatten(), stable=True).indices
    counts = torch.bincount(idx.flatten(), minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(len(perm), device=perm.device)
    return perm.to(torch.int32), offsets, inv.to(torch.int32), perm // idx.shape[1]


def of_tokens(moe, case, saved, at, experts):  # noqa: F811
    """The same layer over the tokens `at`, with the experts numbered from
    experts.start on alone: (case, record, sorted rows of the whole)."""
    T, E, k, H, I = case.sizes
    part = Case(1, 1, 1, 256, 256)
    part.sizes, part.dense = (len(at), len(range(E)[experts]), k, H, I), False
    part.x, part.d_out, part.gates, part.W = case.x[at], case.d_out[at], case.gates[at], tuple(w[experts] for w in case.W)
    slots = (at[:, None] * k + torch.arange(k, device="cuda")).flatten()
    rows = case.inv.long()[slots]
    idx = (torch.searchsorted(case.offsets.long(), rows, right=True) - 1 - (experts.start or 0)).view(-1, k)
    part.perm, part.offsets, part.inv, part.tokens = lists(idx, part.sizes[1])
    rows = rows[part.perm.long()]
    take = lambda t, r: None if t is None else t.view(torch.uint8)[r].view(t.dtype)  # noqa: E731
    kept = [take(t, r) for t, r in ((saved.gate, rows), (saved.up, rows), (saved.x_scales, at),
                                    (saved.gate_scales, rows), (saved.up_scales, rows))]
    x = part.x if saved.gate_scales is None else take(saved.x, at)
    return part, moe.SavedFfn(x, *kept), rows


def weight_gradients(case, saved, feats):
    """dWg, dWu [E, feats, H] and dWd [E, H, feats] in 64 bits, of features inside one block of 128."""
    T, E, k, H, I = case.sizes
    if saved.gate_scales is None:
        x, g, u = saved.x.double(), saved.gate[:, feats].double(), saved.up[:, feats].double()
    else:
        x, b = fp8_plain.rows_value(saved.x, saved.x_scales), feats.start // 128
        g, u = (q[:, feats].double() * fp8_plain.two_to(s[:, b:b + 1].long() - 127)
                for q, s in ((saved.gate, saved.gate_scales), (saved.up, saved.up_scales)))
    d, n = case.d_out.double(), feats.stop - feats.start
    out = [torch.zeros(s, dtype=torch.float64, device="cuda") for s in ((E, n, H), (E, n, H), (E, H, n))]
    for e, r in plain.groups(case.offsets, T * k):
        tok, s = case.tokens[r], torch.sigmoid(g[r])
        w = case.gates.double().flatten()[case.perm[r].long()][:, None]
        q = (d @ case.W[2][e][:, feats].double())[tok] * w
        by_token = lambda v: torch.zeros((T, n), dtype=torch.float64, device="cuda").index_add_(0, tok, v)  # noqa: E731
        out[0][e] = by_token(q * u[r] * s * (1 + g[r] * (1 - s))).T @ x
        out[1][e] = by_token(q * g[r] * s).T @ x
        out[2][e] = d.T @ by_token(w * g[r] * s * u[r])
    return out


@pytest.mark.parametrize("checkpoint", ["bf16", "fp8"])
@pytest.mark.parametrize("H,I", [(16384, 256), (256, 16384)])
def test_rows_beyond_32_bits(moe, H, I, checkpoint):  # noqa: F811
    T, E, k = 70_000, 3, 2
    case = Case(T, E, k, H, I, seed=28)
    y, saved = case.forward(moe, checkpoint)
    d_x, d_gates, *dW = case.backward(moe, saved)
    P, mid = T * k, 2 ** 31 // 16384
    pos = torch.cat([torch.arange(0, 3), torch.arange(mid - 3, mid + 3), torch.arange(P - 20, P)]).cuda()
    at = torch.unique(case.tokens[pos])
    part, kept, rows = of_tokens(moe, case, saved, at, slice(0, E))
    check_forward(part, y[rows], kept, moe)
    want, _, _ = part.plain_backward(moe, kept)
    assert plain.rel_rms(d_x[at], want["d_x"]) <= REL_RMS_TOL
    assert plain.rel_rms(d_gates[at], want["d_gates"]) <= 2e-5
    for feats in (slice(0, 16), slice(I - 16, I)):
        g, u, d = weight_gradients(case, saved, feats)
        for got, ref in ((dW[0][:, feats], g), (dW[1][:, feats], u), (dW[2][:, :, feats], d)):
            assert all(plain.rel_rms(got[e], ref[e]) <= REL_RMS_TOL for e in range(E))


@pytest.mark.parametrize("checkpoint", ["bf16", "fp8"])
def test_weights_beyond_32_bits(moe, checkpoint):  # noqa: F811
    """130 x 4096 x 4096 values a matrix: the last two experts, and those without rows."""
    T, E, k, H, I = 40, 130, 2, 4096, 4096
    case = Case(T, E, k, H, I, seed=29)
    t = torch.arange(T, device="cuda")
    idx = torch.where((t < 20)[:, None], torch.stack([t, t + 20], 1), torch.tensor([[128, 129]], device="cuda"))
    case.perm, case.offsets, case.inv, case.tokens = lists(idx, E)
    y, saved = case.forward(moe, checkpoint)
    dW = tuple(torch.full_like(w, float("nan")) for w in case.W)
    d_x, d_gates, *_ = case.backward(moe, saved, dW=dW)
    part, kept, rows = of_tokens(moe, case, saved, t[20:], slice(128, 130))
    check_forward(part, y[rows], kept, moe)
    check_backward(part, (d_x[20:], d_gates[20:], *(w[128:] for w in dW)), kept, moe)
    assert all((w[40:128] == 0).all() for w in dW)


@pytest.mark.parametrize("rows,K", [(5, 16384), (131_080, 16384)])
def test_quantised_and_widened_rows(moe, rows, K):  # noqa: F811
    """A checkpoint's rows and their values, below and beyond 2^31 of them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(30)
    x = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    at = torch.cat([torch.arange(0, 2), torch.arange(rows - 3, rows)]).cuda()
    got = moe.moe_dequantize_rows(*moe.moe_quantize_rows(x))
    assert torch.equal(got[at].double(), plain.held(x[at]))
