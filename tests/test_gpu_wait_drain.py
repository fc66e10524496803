"""GPU: expert kernels whose waits expire leave nothing behind, also where one
role had already issued all it had to (few blocks of K: the producer never
waits), so that only the others gave up.

Each round launches a call whose main-loop waits give up after one cycle and,
without a pause, the same call with the default bound: its CTAs take over the
shared memory and tensor memory at once, so a copy or MMA still on its way
would land in theirs.  Its outputs have to be the bits of an undisturbed call."""
import pytest
import torch

import synth
from test_gpu_fp8 import layer_case

pytestmark = pytest.mark.gpu
MOE_ERR_TIMEOUT = 5
ROUNDS = 20


@pytest.fixture(scope="module")
def moe():
    import routed_expert_ffn_02_gb300 as m
    return m


def check(moe, call, ws):
    ref = call().clone()
    torch.cuda.synchronize()
    assert ws.status() == 0
    outs = []
    for _ in range(ROUNDS):
        moe.debug_set_wait_limit(1)
        try:
            call()
        finally:
            moe.debug_set_wait_limit(0)
        outs.append(call().clone())
    torch.cuda.synchronize()
    assert ws.status(clear=True) == MOE_ERR_TIMEOUT
    assert all(torch.equal(o, ref) for o in outs)
    assert torch.equal(call(), ref) and ws.status() == 0


@pytest.mark.parametrize("T,E,k,H,I", [(4, 64, 8, 512, 256),       # thin tiles
                                       (40, 2, 2, 512, 512),       # 33-128 rows
                                       (300, 64, 2, 512, 512),     # padded pair tiles, early weights
                                       (700, 3, 2, 2048, 1024)])
def test_8bit_one_cta_kernel(moe, T, E, k, H, I):
    shape, lg, x, ex, _ = layer_case(moe, T, E, k, H, I, 1.1)
    ws = moe.Workspace(moe.fp8_workspace_size(shape))
    check(moe, lambda: moe.moe_forward_fp8(shape, lg, x, ex, ws=ws), ws)


def experts_case(moe, T, E, k, H, I, thr, mma):
    """moe_expert_ffn on bf16 experts, as a call."""
    d = {n: v.cuda() for n, v in synth.make_layer(synth.Shape(T=T, E=E, k=k, H=H, I=I), seed=7).items()}
    shape = moe.Shape(T, E, k, H, I, fat_threshold=thr, thin_mma_min=mma)
    counts, offsets, perm, _ = moe.moe_permute(moe.moe_route(d["logits"], k)[0], E)
    ws = moe.Workspace(moe.expert_ffn_workspace_size(shape))
    return (lambda: moe.moe_expert_ffn(shape, d["x"], perm, offsets, counts, d["Wg"], d["Wu"], d["Wd"],
                                       ws=ws)), ws


@pytest.mark.parametrize("H,I", [(256, 256), (2048, 512)])
def test_bf16_one_cta_gemm(moe, H, I):
    check(moe, *experts_case(moe, 64, 16, 2, H, I, 1, 0))


@pytest.mark.parametrize("H,I", [(256, 256), (2048, 1024)])
def test_tensor_core_streaming(moe, H, I):
    check(moe, *experts_case(moe, 64, 16, 2, H, I, 33, 1))


@pytest.mark.parametrize("H,I", [(256, 256), (2048, 1024)])
def test_cuda_core_streaming(moe, H, I):
    check(moe, *experts_case(moe, 64, 16, 2, H, I, 33, 33))


@pytest.mark.parametrize("T,H,I", [(2, 1024, 2048), (1, 2048, 1024), (2, 2048, 1024)])
def test_self_routed_decode(moe, T, H, I):
    """Two launches, or the whole layer in one."""
    Wg, Wu, Wd = synth.make_weights(16, H, I, seed=7, layer=0, device="cuda")
    shape = moe.Shape(T, 16, 8, H, I, fat_threshold=32, thin_mma_min=33)
    x, lg = synth.make_x(T, H, seed=7).cuda(), synth.make_logits(T, 16, seed=7).cuda()
    ws = moe.Workspace(moe.workspace_size(shape))
    check(moe, lambda: moe.moe_forward(shape, lg, x, Wg, Wu, Wd, ws=ws), ws)


@pytest.mark.parametrize("H,I", [(256, 256), (1024, 768)])
def test_bf16_pair_gemm(moe, H, I):
    check(moe, *experts_case(moe, 1000, 4, 2, H, I, 1, 0))


@pytest.mark.parametrize("T,E,k,H,I", [(300, 1, 1, 256, 256), (2500, 6, 2, 512, 256), (2500, 2, 2, 2048, 1024)])
def test_8bit_pair_kernel(moe, T, E, k, H, I):
    shape, lg, x, ex, _ = layer_case(moe, T, E, k, H, I, 1.1)
    ws = moe.Workspace(moe.fp8_workspace_size(shape))
    check(moe, lambda: moe.moe_forward_fp8(shape, lg, x, ex, ws=ws), ws)
