"""GPU: the balance loss at the ends of its range of tokens and offsets."""
import pytest
import torch

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
