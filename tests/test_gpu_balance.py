"""GPU: the router's balance loss, counts and logits gradient against the
definition in 64 bits (gradient by fp64 autograd and by differences).

Tolerances.  Counts are exact.  A probability carries a few fp32 roundings
(exp, the row sum over at most 32 terms per lane and 5 levels, the product):
under 40 * 2^-24 relative, and a sum over T tokens in chunks adds at most
(8 + 64 / 8 + T / 64) roundings of a running sum of positive terms; the bound
used, (64 + T / 64) * 2^-23, covers both.  A gradient value is the difference
of two such quantities, so its error is held against p (|a| + sum p |a|)."""
import pytest
import torch

import fp8_plain as plain
import synth

pytestmark = pytest.mark.gpu
MOE_ERR_BAD_INDEX = 6


@pytest.fixture(scope="module")
def moe():
    import routed_expert_ffn_02_gb300 as m
    return m


def case(moe, T, E, k, seed=0):
    lg = synth.make_logits(T, E, seed=seed, zipf_s=1.1).cuda()
    idx, gates = moe.moe_route(lg, k)
    return lg, idx, gates


def check(moe, lg, idx, gates, off, coef, d_loss=1.7, with_gates=True):
    T, E = lg.shape
    k = idx.shape[1]
    offs = off if off is not None else [0, T]
    seq = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    ws = moe.Workspace(moe.balance_workspace_size(T, E, len(offs) - 1))
    loss, counts, stats = moe.moe_balance(lg, idx, seq, coef, ws=ws)
    assert ws.status() == 0
    l64 = lg.double().requires_grad_()
    want, c = plain.balance(l64, idx, offs, coef)
    tol = (64 + T / 64) * 2.0 ** -23
    assert torch.equal(counts, c.cuda())
    assert abs(loss.item() - want.item()) <= tol * want.item()
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    dg = torch.randn((T, k), generator=g, device="cuda") * 1e-3
    extra = dict(topk_idx=idx, gates=gates, d_gates=dg) if with_gates else {}
    d = moe.moe_balance_backward(lg, stats, counts, k, seq, coef,
                                 torch.tensor(d_loss, device="cuda"), **extra)
    if want.requires_grad:
        (grad,) = torch.autograd.grad(want * d_loss, l64)
        grad = grad.nan_to_num(0.0)      # rows of -inf alone
    else:                                # every sequence is empty
        grad = torch.zeros_like(lg, dtype=torch.float64)
    # magnitude of what cancels in a gradient value
    p = torch.softmax(l64.detach(), 1).nan_to_num(0.0)
    total = max(1, offs[-1] - offs[0])
    a = torch.zeros_like(p)
    for s, (b, z) in enumerate(zip(offs[:-1], offs[1:])):
        if z > b:
            a[b:z] = coef * E * c[s].double().cuda() / (k * (z - b) * total)
    size = abs(d_loss) * p * (a + (p * a).sum(1, keepdim=True))
    if with_gates:
        gd, dgd = gates.double(), dg.double()
        mine = gd * (dgd - (gd * dgd).sum(1, keepdim=True))
        grad = grad.scatter_add(1, idx.long(), mine)
        size = size.scatter_add(1, idx.long(), gd * (dgd.abs() + (gd * dgd.abs()).sum(1, keepdim=True)))
    over = (d.double() - grad).abs() - tol * size
    assert bool((over <= 0).all()), over.max().item()
    again = moe.moe_balance(lg, idx, seq, coef, ws=ws)
    assert torch.equal(again[0], loss) and torch.equal(again[1], counts)
    return loss, counts, d


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 8), (5, 33, 3), (64, 16, 2), (65, 256, 8),
                                   (1000, 384, 8), (200, 1000, 6), (130, 1024, 1), (16384, 100, 8)])
@pytest.mark.parametrize("with_gates", [True, False])
def test_one_sequence(moe, T, E, k, with_gates):
    check(moe, *case(moe, T, E, k), None, 1e-2, with_gates=with_gates)


@pytest.mark.parametrize("off", [[0, 500], [0, 0, 500], [0, 3, 3, 3, 64, 65, 200, 200], [7, 100, 400],
                                 [0, 1, 2, 3, 4, 5, 499, 500], [0, 0, 0], [500, 500], [63, 64, 65, 128, 129]])
def test_packed_sequences(moe, off):
    lg, idx, gates = case(moe, 500, 70, 4, seed=1)
    loss, counts, d = check(moe, lg, idx, gates, off, 0.5)
    outside = torch.ones(500, dtype=torch.bool)
    outside[off[0]:off[-1]] = False
    d0 = moe.moe_balance_backward(lg, moe.moe_balance(lg, idx, torch.tensor(off, dtype=torch.int32).cuda(), 0.5)[2],
                                  counts, 4, torch.tensor(off, dtype=torch.int32).cuda(), 0.5)
    assert not d0[outside.cuda()].any()


def test_many_sequences(moe):
    lg, idx, gates = case(moe, 900, 40, 2, seed=2)
    check(moe, lg, idx, gates, list(range(0, 901)), 1.0)


def test_masked_experts_and_empty_rows(moe):
    lg, idx, gates = case(moe, 200, 50, 4, seed=3)
    lg[:, 10:20] = float("-inf")
    idx, gates = moe.moe_route(lg, 4)
    lg[17] = float("-inf")           # no expert left: no probability, no gradient
    check(moe, lg, idx, gates, [0, 100, 200], 1.0)
    loss, counts, stats = moe.moe_balance(lg, idx)
    assert torch.isfinite(loss)
    d = moe.moe_balance_backward(lg, stats, counts, 4)
    assert torch.isfinite(d).all() and not d[17].any() and not d[:, 10:20].any()


def test_even_routing_gives_coef(moe):
    """Slots spread evenly: loss = coef, and no gradient."""
    T, E, k = 64, 16, 4
    idx = ((torch.arange(T)[:, None] * k + torch.arange(k)) % E).int().cuda()
    lg = torch.randn((T, E), device="cuda")
    loss, counts, stats = moe.moe_balance(lg, idx, coef=0.25)
    assert bool((counts == T * k // E).all())
    assert abs(loss.item() - 0.25) <= 0.25 * 65 * 2.0 ** -23
    d = moe.moe_balance_backward(lg, stats, counts, k, coef=0.25)
    assert d.abs().max().item() <= 0.25 / T * 65 * 2.0 ** -23


def test_gradient_by_differences(moe):
    """Central differences of the kernel's own loss along random directions
    (counts held): step 0.5 % of unit logits; the third-order term is under
    h^2 and the loss's rounding under 2^-20 / h of its size."""
    lg, idx, gates = case(moe, 300, 24, 3, seed=4)
    off = torch.tensor([0, 120, 300], dtype=torch.int32, device="cuda")
    loss, counts, stats = moe.moe_balance(lg, idx, off, 1.0)
    d = moe.moe_balance_backward(lg, stats, counts, 3, off, 1.0).double()
    h = 0.02
    for seed in range(4):
        v = torch.randn(lg.shape, generator=torch.Generator().manual_seed(seed)).cuda()
        lo, hi = (moe.moe_balance(lg + s * h * v, idx, off, 1.0)[0].double().item() for s in (-1, 1))
        slope = (d * v.double()).sum().item()
        assert abs((hi - lo) / (2 * h) - slope) <= 2 * h * h + 2.0 ** -20 / h


def test_bad_index_and_offsets(moe):
    lg, idx, gates = case(moe, 100, 8, 2, seed=5)
    bad = idx.clone()
    bad[3, 1], bad[50, 0] = 8, -1
    ws = moe.Workspace(moe.balance_workspace_size(100, 8))
    loss, counts, stats = moe.moe_balance(lg, bad, ws=ws)
    assert ws.status(clear=True) == MOE_ERR_BAD_INDEX
    assert counts.sum().item() == 198
    # offsets out of [0, T] are held inside it
    off = torch.tensor([-5, 40, 1000], dtype=torch.int32, device="cuda")
    a = moe.moe_balance(lg, idx, off, ws=moe.Workspace(moe.balance_workspace_size(100, 8, 2)))
    b = moe.moe_balance(lg, idx, torch.tensor([0, 40, 100], dtype=torch.int32, device="cuda"))
    assert torch.equal(a[1], b[1]) and torch.equal(a[0], b[0])


def test_no_tokens(moe):
    z = torch.empty((0, 8), device="cuda")
    loss, counts, stats = moe.moe_balance(z, torch.empty((0, 2), dtype=torch.int32, device="cuda"))
    assert loss.item() == 0 and not counts.any()
    assert moe.moe_balance_backward(z, stats, counts, 2).shape == (0, 8)
