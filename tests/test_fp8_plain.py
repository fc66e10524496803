"""CPU: the tests' plain 64-bit forms of the 8-bit format and of the balance
loss against independent facts, and the binding's refusal of host tensors."""
import math

import pytest
import torch

import fp8_plain as plain


def all_bf16():
    return torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)


def test_e4m3_is_torchs_cast():
    """Every bf16 value inside the range rounds as torch's cast does."""
    v = all_bf16()
    v = v[torch.isfinite(v) & (v.float().abs() <= 448)]
    assert torch.equal(plain.e4m3(v.double()), v.float().to(torch.float8_e4m3fn).double())


def test_scale_is_the_smallest_power_of_two():
    a = all_bf16()
    a = a[torch.isfinite(a) & (a.float() > 0)].double()
    b = plain.scale_bytes(a)
    fits = lambda b: a <= 448 * plain.two_to(b - 127)      # noqa: E731
    assert bool(fits(b).all()) and bool((~fits(b - 1) | (b == 0)).all())
    assert b.max() < 255


def test_one_bad_value_leaves_its_block_alone():
    x = torch.randn(2, 256, dtype=torch.float64)
    y = x.clone()
    y[1, 5], y[1, 200] = math.inf, math.nan
    (q, b), (r, c) = plain.quantize_rows(x), plain.quantize_rows(y)
    keep = torch.isfinite(y)
    x0 = x.clone()
    x0[~keep] = 0
    q0, b0 = plain.quantize_rows(x0)
    assert torch.equal(c, b0) and torch.equal(r[keep], q0[keep]) and torch.isnan(r[~keep]).all()
    assert torch.equal(q[0], r[0]) and torch.equal(b[0], c[0])


def test_balance_loss_closed_forms():
    T, E, k = 24, 6, 2
    even = (torch.arange(T)[:, None] * k + torch.arange(k)) % E
    lg = torch.randn(T, E, dtype=torch.float64)
    loss, counts = plain.balance(lg, even, [0, T], 0.5)
    assert abs(loss.item() - 0.5) < 1e-12 and (counts == T * k // E).all()
    # all tokens on one expert with certainty: f = E / 1, P = 1 -> loss = E coef
    sure = torch.full((T, E), -100.0, dtype=torch.float64)
    sure[:, 3] = 100
    loss, _ = plain.balance(sure, torch.full((T, 1), 3), [0, T], 1.0)
    assert abs(loss.item() - E) < 1e-9
    # a split into sequences of one distribution each is the token-weighted mean
    a, _ = plain.balance(lg[:10], even[:10], [0, 10], 1.0)
    b, _ = plain.balance(lg[10:], even[10:], [0, T - 10], 1.0)
    both, _ = plain.balance(lg, even, [0, 10, 10, T], 1.0)
    assert abs(both.item() - (10 * a.item() + (T - 10) * b.item()) / T) < 1e-12


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import routed_expert_ffn_02_gb300 as m
    return m


def test_host_tensors_and_wrong_types_are_refused(moe):
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    with pytest.raises(AssertionError, match="CUDA tensor"):
        moe.moe_quantize_rows(x)
    with pytest.raises(AssertionError):
        moe.moe_balance(torch.zeros((4, 8)), torch.zeros((4, 2), dtype=torch.int32),
                        torch.tensor([0], dtype=torch.int32))
    z = torch.zeros((2, 256, 256), dtype=torch.float8_e4m3fn)
    s = torch.zeros((2, 2, 2), dtype=torch.uint8)
    with pytest.raises(AssertionError):
        moe.Fp8Experts(z, s, z, s, z, s)
