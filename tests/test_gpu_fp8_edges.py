"""GPU: the quantiser on blocks without a finite value.  Exact."""
import pytest
import torch

import fp8_plain as plain
from test_gpu_fp8 import randn, same

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def moe():
    import routed_expert_ffn_02_gb300 as m
    return m


@pytest.mark.parametrize("fill", [[NAN], [-NAN], [INF], [-INF], [NAN, INF], [-INF, NAN, NAN]],
                         ids=lambda f: "_".join(map(str, f)))
def test_block_without_finite_values(moe, fill):
    """No finite value, no part in the scale: the smallest one, byte 0."""
    def values(*shape):
        return torch.tensor(fill, device="cuda").repeat(128 * 128)[:shape[0] * shape[1]].view(shape)
    x = randn((5, 384), 1)
    x[1, :128], x[2, 256:], x[4] = values(1, 128), values(1, 128), values(1, 384)
    q, s = moe.moe_quantize_rows(x)
    want, b = plain.quantize_rows(x)
    assert torch.equal(s.long(), b) and same(q, want)
    assert s[1, 0] == 0 and s[2, 2] == 0 and not s[4].any()
    W = randn((2, 256, 256), 2, 0.02)
    W[0, :128, 128:], W[1, 128:, 128:] = values(128, 128), values(128, 128)
    W[1, :128, :128], W[1, 3, 5] = values(128, 128), 0.5     # one finite value in it
    q, s = moe.moe_quantize_weights(W)
    want, b = plain.quantize_weights(W)
    assert torch.equal(s.long(), b) and same(q, want)
    assert s[0, 0, 1] == 0 and s[1, 1, 1] == 0 and s[1, 0, 0] > 0


@pytest.mark.parametrize("T", [3, 40, 300])
def test_token_without_finite_values(moe, T):
    """In the layer: NaN outputs for that token alone, whichever launch quantises."""
    from test_gpu_fp8 import layer_case
    shape, lg, x, ex, _ = layer_case(moe, T, 8, 2, 512, 256)
    ref = moe.moe_forward_fp8(shape, lg, x, ex)
    x[1] = NAN
    out = moe.moe_forward_fp8(shape, lg, x, ex)
    assert torch.isnan(out[1]).all()
    rest = [t for t in range(T) if t != 1]
    assert torch.equal(out[rest], ref[rest])
