"""GPU: the balance loss at the ends of its range of tokens and offsets, and its
gradient against extrapolated differences."""
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


@pytest.mark.parametrize("E,k", [(1, 1), (8, 8)])
def test_as_many_slots_as_fit_31_bits(moe, E, k):
    """T k at the largest value that is taken.  Every token is routed evenly, so
    the loss is coef and no logit has a gradient; the sums are of equal powers
    of two, exact within a chunk of tokens, and at most 512 chunks are added up:
    2^-15 of rounding, twice that is allowed."""
    T = (2**31 - 129) // k
    lg = torch.zeros((T, E), device="cuda")
    idx = torch.arange(k, dtype=torch.int32, device="cuda").repeat(T, 1)
    loss, counts, stats = moe.moe_balance(lg, idx, coef=0.5)
    assert (counts == T).all()
    assert abs(loss.item() - 0.5) <= 0.5 * 2.0 ** -14
    del idx
    d = torch.full((T, E), 7.0, device="cuda")
    moe.moe_balance_backward(lg, stats, counts, k, coef=0.5, d_logits=d)
    assert not d.any()


def poisoned(moe, T, E, S):
    """A workspace whose scratch holds large numbers."""
    ws = moe.Workspace(moe.balance_workspace_size(T, E, S))
    ws.tensor[256:].view(torch.float32).fill_(1e6)
    return ws


@pytest.mark.parametrize("T", [100, 3000])
@pytest.mark.parametrize("off", [[0, 80, 40, 100], [90, 10], [0, 50, 50, 49], [0, 2000, 30, 100]])
def test_descending_offsets(moe, T, off):
    """Recorded, and no token takes part: nothing of the scratch's former
    contents reaches the outputs."""
    E, k, S = 40, 4, len(off) - 1
    lg = torch.randn((T, E), device="cuda")
    idx, gates = moe.moe_route(lg, k)
    seq = torch.tensor(off, dtype=torch.int32, device="cuda")
    ws = poisoned(moe, T, E, S)
    stats = torch.full((T, 2), float("nan"), device="cuda")
    loss, counts, _ = moe.moe_balance(lg, idx, seq, 1.0, stats=stats, ws=ws)
    assert ws.status(clear=True) == MOE_ERR_BAD_INDEX
    assert loss.item() == 0 and not counts.any()
    d = moe.moe_balance_backward(lg, stats, counts, k, seq, 1.0)
    assert not d.any()
    dg = torch.randn((T, k), device="cuda")
    both = moe.moe_balance_backward(lg, stats, counts, k, seq, 1.0, topk_idx=idx, gates=gates, d_gates=dg)
    ok = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    _, c1, s1 = moe.moe_balance(lg, idx, ok, 0.0)
    assert torch.equal(both, moe.moe_balance_backward(lg, s1, c1, k, ok, 0.0, topk_idx=idx, gates=gates,
                                                      d_gates=dg))


@pytest.mark.parametrize("off,held", [([-5, 40, 1000], [0, 40, 100]), ([0, 101], [0, 100]), ([-1, 100], [0, 100])])
def test_offsets_out_of_range_are_held_and_recorded(moe, off, held):
    lg = torch.randn((100, 8), device="cuda")
    idx, _ = moe.moe_route(lg, 2)
    a, b = (torch.tensor(o, dtype=torch.int32, device="cuda") for o in (off, held))
    ws = poisoned(moe, 100, 8, len(off) - 1)
    loss, counts, stats = moe.moe_balance(lg, idx, a, ws=ws)
    assert ws.status(clear=True) == MOE_ERR_BAD_INDEX
    want = moe.moe_balance(lg, idx, b, ws=ws)
    assert ws.status() == 0
    assert torch.equal(loss, want[0]) and torch.equal(counts, want[1]) and torch.equal(stats, want[2])


def test_no_tokens_with_offsets(moe):
    z, i = torch.empty((0, 8), device="cuda"), torch.empty((0, 2), dtype=torch.int32, device="cuda")
    ws = poisoned(moe, 0, 8, 2)
    loss, counts, _ = moe.moe_balance(z, i, torch.zeros(3, dtype=torch.int32, device="cuda"), ws=ws)
    assert ws.status() == 0 and loss.item() == 0 and not counts.any()
    moe.moe_balance(z, i, torch.tensor([0, 1, 0], dtype=torch.int32, device="cuda"), ws=ws)
    assert ws.status(clear=True) == MOE_ERR_BAD_INDEX


def fixed_slots(lg, idx, off, coef, d_loss, dg):
    """d_loss * loss + sum of dg * gates over the selected slots, in 64 bits."""
    loss, _ = plain.balance(lg, idx, off, coef)
    gates = torch.softmax(lg.gather(1, idx.long()), 1)
    return (d_loss * loss + (dg.double() * gates).sum()).item()


@pytest.mark.parametrize("T,E,k,off", [(300, 24, 3, [0, 120, 300]), (130, 200, 8, [10, 10, 77, 130])])
def test_gradient_against_extrapolated_differences(moe, T, E, k, off):
    """Along random directions the kernel's gradient has to give the slope of the
    definition in 64 bits: central differences at h and h / 2, extrapolated, are
    off by about h^4 of the fifth derivative (h = 0.01: 1e-9 of the slope).  The
    gradient's own rounding is held as in test_gpu_balance.py, and is under a
    hundredth of the slope, so that no term of it can be missing."""
    coef, d_loss = 1.0, 1.7
    lg = synth.make_logits(T, E, seed=4, zipf_s=1.1).cuda()
    idx, gates = moe.moe_route(lg, k)
    seq = torch.tensor(off, dtype=torch.int32, device="cuda")
    dg = torch.randn((T, k), generator=torch.Generator().manual_seed(1)).cuda() * 1e-2
    loss, counts, stats = moe.moe_balance(lg, idx, seq, coef)
    d = moe.moe_balance_backward(lg, stats, counts, k, seq, coef, torch.tensor(d_loss, device="cuda"),
                                 topk_idx=idx, gates=gates, d_gates=dg).double()
    tol = (64 + T / 64) * 2.0 ** -23
    p, g, b = torch.softmax(lg.double(), 1), gates.double(), dg.double().abs()
    a = torch.zeros_like(p)
    for s, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        if hi > lo:
            a[lo:hi] = coef * E * counts[s].double() / (k * (hi - lo) * (off[-1] - off[0]))
    size = d_loss * p * (a + (p * a).sum(1, keepdim=True))
    size = size.scatter_add(1, idx.long(), g * (b + (g * b).sum(1, keepdim=True)))
    for seed in range(4):
        v = torch.randn((T, E), generator=torch.Generator().manual_seed(seed), dtype=torch.float64).cuda()
        v += 2 * torch.sign(d)      # a slope that does not cancel

        def slope(h):
            f = [fixed_slots(lg.double() + s * h * v, idx, off, coef, d_loss, dg) for s in (-1, 1)]
            return (f[1] - f[0]) / (2 * h)
        want = slope(0.005) + (slope(0.005) - slope(0.01)) / 3
        held = tol * (size * v.abs()).sum().item() + 1e-6 * abs(want)
        assert held <= 0.01 * abs(want)
        assert abs((d * v).sum().item() - want) <= held
