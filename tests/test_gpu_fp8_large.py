"""GPU: the 8-bit operators and the balance loss at sizes whose offsets pass
32 bits, on misaligned rows, over seeded random shapes, and the example.

Tolerances as in test_gpu_fp8.py and test_gpu_balance.py."""
import importlib.util
import os

import pytest
import torch

import fp8_plain as plain
from parity import REL_RMS_TOL
from test_gpu_balance import check as check_balance
from test_gpu_fp8 import check_product, layer_case, product_case, randn, rel_rms, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import routed_expert_ffn_02_gb300 as m
    return m


def test_quantize_beyond_32_bits(moe):
    rows, K = 270_000, 16384                 # 8.8 GB of bf16, 4.4 G codes
    x = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda").normal_()
    q, s = moe.moe_quantize_rows(x)
    for part in (slice(0, 64), slice(131_060, 131_090), slice(rows - 64, rows)):
        want, b = plain.quantize_rows(x[part])
        assert torch.equal(s[part].long(), b) and same(q[part], want)


@pytest.mark.parametrize("rows,N,K", [(270_000, 128, 16384), (140_000, 16384, 256)])
def test_product_beyond_32_bits(moe, rows, N, K):
    """Operand or output offsets past 2^32; two groups, the first small."""
    q = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda").normal_().mul_(100)
    q = q.clamp_(-448, 448).to(torch.float8_e4m3fn)
    sq = torch.randint(118, 122, (rows, K // 128), device="cuda").to(torch.uint8)
    W, sW = moe.moe_quantize_weights(randn((2, N, K), 1, 0.05))
    off = torch.tensor([0, 77, rows], dtype=torch.int32, device="cuda")
    y = moe.moe_grouped_gemm_fp8(q, sq, off, W, sW)
    tail = slice(rows - 100, rows)
    check_product(y[tail], q[tail], sq[tail], torch.tensor([0, 0, 100]), W, sW)
    check_product(y[:77], q[:77], sq[:77], torch.tensor([0, 77, 77]), W, sW)
    mid = slice(131_000, 131_200)
    check_product(y[mid], q[mid], sq[mid], torch.tensor([0, 0, 200]), W, sW)


def test_balance_beyond_32_bits(moe):
    T, E, k = 2_200_000, 1000, 2             # 8.8 GB of logits
    lg = torch.empty((T, E), device="cuda").normal_()
    idx, gates = moe.moe_route(lg, k)
    loss, counts, stats = moe.moe_balance(lg, idx, coef=0.5)
    assert counts.sum().item() == T * k
    assert abs(loss.item() - 0.5) < 0.01     # nearly even routing
    d = moe.moe_balance_backward(lg, stats, counts, k, coef=0.5)
    part = slice(T - 50, T)
    p = torch.softmax(lg[part].double(), 1)
    a = 0.5 * E * counts.double() / (k * T) / T
    want = p * (a - (p * a).sum(1, keepdim=True))
    size = p * (a + (p * a).sum(1, keepdim=True))
    assert bool(((d[part].double() - want).abs() <= 128 * 2.0 ** -23 * size).all())


def test_misaligned_rows(moe):
    """Inputs that start off the widest vectors' boundaries."""
    flat = randn((33 * 256 + 8,), 3)
    x = flat[8:].view(33, 256)               # 16 but not 32 bytes aligned
    q, s = moe.moe_quantize_rows(x)
    want, b = plain.quantize_rows(x)
    assert torch.equal(s.long(), b) and same(q, want)
    with pytest.raises(moe.MoeError):        # 2 bytes aligned: refused
        moe.moe_quantize_rows(randn((256 * 4 + 1,), 3)[1:].view(4, 256))
    with pytest.raises(AssertionError):      # not contiguous: refused
        moe.moe_quantize_rows(randn((4, 512), 3)[:, :256])
    lg = torch.randn(200 * 384 + 1, device="cuda")[1:].view(200, 384)   # 4 bytes aligned
    idx, gates = moe.moe_route(lg, 8)
    check_balance(moe, lg, idx, gates, [0, 150, 200], 1.0)


@pytest.mark.parametrize("seed", range(12))
def test_random_layers(moe, seed):
    g = torch.Generator().manual_seed(seed)
    pick = lambda *v: v[int(torch.randint(0, len(v), (1,), generator=g))]   # noqa: E731
    T, E = pick(1, 2, 7, 31, 33, 60, 129, 400), pick(1, 3, 16, 50)
    k, H, I = min(E, pick(1, 2, 5, 8)), pick(256, 768, 1280), pick(256, 512, 768)
    shape, lg, x, ex, parts = layer_case(moe, T, E, k, H, I, pick(None, 1.1), seed=seed)
    idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
    gates = torch.empty((T, k), dtype=torch.float32, device="cuda")
    out = moe.moe_forward_fp8(shape, lg, x, ex, topk_idx=idx, gates=gates)
    ridx, rgates = moe.moe_route(lg, k)
    assert torch.equal(idx, ridx) and torch.equal(gates, rgates)
    assert rel_rms(out, plain.layer(x, idx, gates, parts)[0]) <= REL_RMS_TOL


@pytest.mark.parametrize("seed", range(8))
def test_random_products(moe, seed):
    g = torch.Generator().manual_seed(100 + seed)
    E = int(torch.randint(1, 20, (1,), generator=g))
    counts = torch.randint(0, [40, 300][seed % 2], (E,), generator=g).tolist()
    counts[0] += 1
    N, K = (128 * int(torch.randint(1, 12, (1,), generator=g)) for _ in range(2))
    args = product_case(moe, counts, N, K, seed=seed)
    check_product(moe.moe_grouped_gemm_fp8(*args), *args)


def test_example_trains_the_router():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "router_on_fp8_experts.py")
    spec = importlib.util.spec_from_file_location("router_on_fp8_experts", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    seen = mod.run(T=1000, E=16, k=2, H=256, I=256, steps=40, verbose=False)
    first, last = seen[0], seen[-1]
    assert last[1] < first[1] and last[2] < first[2], (first, last)   # better balanced
    assert last[0] < 1.05 * first[0], (first, last)                   # and no worse a fit
