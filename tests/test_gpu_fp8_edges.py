"""GPU: the 8-bit operators on blocks without a finite value and on route lists of
bad indices.  The quantiser is exact; tolerances else as in test_gpu_fp8.py."""
import pytest
import torch

import fp8_plain as plain
from parity import REL_RMS_TOL
from test_gpu_fp8 import layer_case, randn, rel_rms, same

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
    shape, lg, x, ex, _ = layer_case(moe, T, 8, 2, 512, 256)
    ref = moe.moe_forward_fp8(shape, lg, x, ex)
    x[1] = NAN
    out = moe.moe_forward_fp8(shape, lg, x, ex)
    assert torch.isnan(out[1]).all()
    rest = [t for t in range(T) if t != 1]
    assert torch.equal(out[rest], ref[rest])


@pytest.mark.parametrize("T,E,k", [(200, 8, 2), (3000, 16, 4)])
def test_experts_after_bad_indices(moe, T, E, k):
    """Slots of bad indices are skipped; the tail of perm that nobody writes holds
    slots of other tokens here, whose rows must come out right all the same."""
    shape, lg, x, ex, parts = layer_case(moe, T, E, k, 512, 256)
    idx, gates = moe.moe_route(lg, k)
    bad = torch.zeros((T, k), dtype=torch.bool, device="cuda")
    bad[T // 2:, 1] = True
    n_bad, P = int(bad.sum()), T * k
    sent = torch.where(bad, E + 3, idx).int()
    out = tuple(torch.arange(n, dtype=torch.int32, device="cuda") for n in (E, E + 1, P, P))
    out[2][-n_bad:] = torch.arange(n_bad, device="cuda")     # slots of the first tokens
    pws = moe.Workspace(moe.permute_workspace_size(T, E, k))
    _, offsets, perm, inv = moe.moe_permute(sent, E, ws=pws, out=out)
    assert pws.status(clear=True) == 6       # MOE_ERR_BAD_INDEX
    ws = moe.Workspace(moe.expert_ffn_fp8_workspace_size(shape))
    ws.tensor[256:].zero_()                  # as stale as a workspace can be: all positions 0
    ys = moe.moe_expert_ffn_fp8(shape, x, perm, offsets, ex, ws=ws)
    _, y = plain.layer(x, idx, gates, parts)
    good = ~bad.flatten()
    assert rel_rms(ys[inv[good].long()], y.view(P, 512)[good]) <= REL_RMS_TOL


def test_experts_whose_storage_is_replaced(moe):
    """The tensors of an Fp8Experts are used where they are at the call."""
    shape, lg, x, ex, _ = layer_case(moe, 40, 8, 2, 512, 256, seed=1)
    other = layer_case(moe, 40, 8, 2, 512, 256, seed=2)[3]
    first, second = (moe.moe_forward_fp8(shape, lg, x, e) for e in (ex, other))
    assert not torch.equal(first, second)
    kept = [t.data for t in ex._tensors()]       # so that the old places stay readable
    for a, b in zip(ex._tensors(), other._tensors()):
        a.data = b.data
    assert torch.equal(moe.moe_forward_fp8(shape, lg, x, ex), second)
    ex.up.data = ex.up.data[:, :128].contiguous()            # no longer these sizes: refused
    with pytest.raises(AssertionError):
        moe.moe_forward_fp8(shape, lg, x, ex)
    del kept


def test_experts_copy_and_pickle(moe):
    import copy
    import pickle
    shape, lg, x, ex, _ = layer_case(moe, 40, 8, 2, 512, 256)
    want = moe.moe_forward_fp8(shape, lg, x, ex)
    for e in (copy.copy(ex), copy.deepcopy(ex), pickle.loads(pickle.dumps(ex))):
        assert torch.equal(moe.moe_forward_fp8(shape, lg, x, e), want)
    deep = copy.deepcopy(ex)
    assert deep.gate.data_ptr() != ex.gate.data_ptr()
