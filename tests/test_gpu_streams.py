"""GPU: calls on a stream other than the current one, with the outputs and the
workspace left to the call, beside work of the current stream that frees or
takes memory of the same sizes.

The current (or the side) stream is held back by a kernel that spins for a
bounded number of cycles, so that the order on the GPU is not the host's."""
import pytest
import torch

import synth
from test_gpu_fp8 import layer_case, randn

pytestmark = pytest.mark.gpu
HOLD = 100_000_000       # cycles, about 50 ms


@pytest.fixture(scope="module")
def moe():
    import routed_expert_ffn_02_gb300 as m
    return m


def calls(moe):
    """name -> call(stream) that allocates its outputs, returning them."""
    lg = synth.make_logits(4096, 64, seed=1).cuda()
    idx, gates = moe.moe_route(lg, 4)
    counts, offsets, perm, inv = moe.moe_permute(idx, 64)
    x, y = randn((4096, 4096), 1), randn((4 * 4096, 512), 2)
    W = randn((8, 1024, 1024), 3)
    bal = moe.Workspace(moe.balance_workspace_size(4096, 64))
    pws = moe.Workspace(moe.permute_workspace_size(4096, 64, 4))
    _, c, stats = moe.moe_balance(lg, idx)
    return {
        "route": lambda s: moe.moe_route(lg, 4, stream=s),
        "permute": lambda s: moe.moe_permute(idx, 64, ws=pws, stream=s),
        "combine": lambda s: (moe.moe_combine(y, inv, gates, 4096, 4, 512, stream=s),),
        "quantize_rows": lambda s: moe.moe_quantize_rows(x, stream=s),
        "quantize_weights": lambda s: moe.moe_quantize_weights(W, stream=s),
        "balance": lambda s: moe.moe_balance(lg, idx, ws=bal, stream=s),
        "balance_backward": lambda s: (moe.moe_balance_backward(lg, stats, c, 4, stream=s),),
    }


NAMES = ["route", "permute", "combine", "quantize_rows", "quantize_weights", "balance", "balance_backward"]


@pytest.mark.parametrize("name", NAMES)
def test_outputs_are_not_memory_that_another_stream_still_writes(moe, name):
    call = calls(moe)[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda._sleep(HOLD)
    for t in want:           # written late by the current stream, freed at once
        torch.empty_like(t).reshape(-1).view(torch.uint8).fill_(0x55)
    got = call(side)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g.reshape(-1).view(torch.uint8), w.reshape(-1).view(torch.uint8))


def layers(moe):
    """name -> (call(out, stream) that allocates its workspace, workspace bytes)."""
    shape, lg, x, ex, _ = layer_case(moe, 300, 16, 4, 512, 256)
    W = synth.make_weights(16, 512, 256, seed=0, device=torch.device("cuda"))
    idx, _ = moe.moe_route(lg, 4)
    _, offsets, perm, _ = moe.moe_permute(idx, 16)
    q, s = moe.moe_quantize_rows(randn((700, 512), 1))
    off = torch.tensor([0, 300, 700], dtype=torch.int32, device="cuda")
    Wq, Ws = moe.moe_quantize_weights(randn((2, 256, 512), 2))
    return {
        "forward_fp8": (lambda o, st: moe.moe_forward_fp8(shape, lg, x, ex, out=o, stream=st),
                        moe.fp8_workspace_size(shape), (300, 512)),
        "expert_ffn_fp8": (lambda o, st: moe.moe_expert_ffn_fp8(shape, x, perm, offsets, ex, y_sorted=o,
                                                                stream=st),
                           moe.expert_ffn_fp8_workspace_size(shape), (1200, 512)),
        "grouped_gemm_fp8": (lambda o, st: moe.moe_grouped_gemm_fp8(q, s, off, Wq, Ws, y=o, stream=st),
                             moe.grouped_gemm_fp8_workspace_size(700, 2), (700, 256)),
        "forward": (lambda o, st: moe.moe_forward(shape, lg, x, *W, out=o, stream=st),
                    moe.workspace_size(shape), (300, 512)),
    }


@pytest.mark.parametrize("name", ["forward_fp8", "expert_ffn_fp8", "grouped_gemm_fp8", "forward"])
def test_workspace_is_not_given_away_before_the_call_has_run(moe, name):
    call, nbytes, size = layers(moe)[name]
    out = torch.empty(size, dtype=torch.bfloat16, device="cuda")
    want = call(out, None).clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(HOLD)
    call(out, side)
    junk = [torch.full((nbytes + 256,), 0x55, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    del junk
