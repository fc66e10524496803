"""GPU: the 8-bit layer and experts where the planner pads an expert's row tiles
with an empty one (257-384 rows, 513-640, ...) in batches whose every tile runs
on the one-CTA kernel, with more items than SMs, so that CTAs meet the empty
tile first and have other items after it.

Tolerance: the layer's, as in test_gpu_fp8.py, over all outputs; and a tenth for
each row alone.  A row's own rounding error is under a hundredth (bf16, and a
few values of h that round to the other neighbour, each at most 1/16 of one of
its I values), while a row multiplied with another tile's weights is off by
about its own size."""
import pytest
import torch

import fp8_plain as plain
from parity import REL_RMS_TOL
from test_gpu_fp8 import layer_case, rel_rms

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import routed_expert_ffn_02_gb300 as m
    return m


def check_rows(got, want):
    assert rel_rms(got, want) <= REL_RMS_TOL
    d = got.double() - want
    worst = (d.square().sum(1) / want.square().sum(1)).sqrt()
    assert worst.max().item() <= 0.1, f"row {worst.argmax().item()}: {worst.max().item():.3g}"


def check_layer(moe, T, E, k, H, I, zipf=None, seed=0, force=None):
    """force: {expert: tokens it is chosen by}, the rest as the logits fall."""
    shape, lg, x, ex, parts = layer_case(moe, T, E, k, H, I, zipf, seed)
    top = lg.amax(1)      # a little above the others, so that every gate counts
    for i, (e, n) in enumerate((force or {}).items()):
        lg[:n, e], lg[n:, e] = top[:n] + 0.1 * (i + 1), -50.0
    idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
    gates = torch.empty((T, k), dtype=torch.float32, device="cuda")
    ws = moe.Workspace(moe.fp8_workspace_size(shape))
    out = moe.moe_forward_fp8(shape, lg, x, ex, topk_idx=idx, gates=gates, ws=ws)
    assert ws.status() == 0
    counts = torch.bincount(idx.flatten().long(), minlength=E)
    for e, n in (force or {}).items():
        assert counts[e].item() == n
    want, y = plain.layer(x, idx, gates, parts)
    check_rows(out, want)
    _, offsets, perm, inv = moe.moe_permute(idx, E)
    ws = moe.Workspace(moe.expert_ffn_fp8_workspace_size(shape))
    ys = moe.moe_expert_ffn_fp8(shape, x, perm, offsets, ex, ws=ws)
    assert ws.status() == 0
    check_rows(ys[inv.long()], y.view(T * k, H))


def test_every_token_on_one_expert(moe):
    check_layer(moe, 300, 64, 2, 4096, 256, force={0: 300})


@pytest.mark.parametrize("rows", [257, 384, 385, 513, 640])
@pytest.mark.parametrize("expert", [0, 5])
def test_rows_of_one_expert(moe, rows, expert):
    check_layer(moe, 700, 64, 2, 2048, 512, force={expert: rows})


def test_many_padded_experts(moe):
    check_layer(moe, 512, 64, 8, 2048, 1024, force={0: 300, 1: 260, 2: 129, 7: 384, 63: 257})


@pytest.mark.parametrize("T,E,k,H,I", [(512, 64, 8, 2048, 256), (1000, 64, 4, 4096, 256),
                                       (2048, 64, 2, 4096, 512), (1365, 3, 3, 4096, 1280)])
@pytest.mark.parametrize("seed", range(3))
def test_skewed_layers(moe, T, E, k, H, I, seed):
    check_layer(moe, T, E, k, H, I, 1.1, seed)
