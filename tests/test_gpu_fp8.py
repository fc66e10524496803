"""GPU: the 8-bit operators (quantiser, grouped product, expert FFN, whole
layer) against plain 64-bit forms.

Tolerances.  The quantiser is exact.  A product's terms are exact in fp32, so
its error is the rounding of the sum (at most K 2^-24 times the sum of the
terms' magnitudes in any order; twice that allows for truncating adders) plus
the last rounding to bf16 (8 significant bits: at most 2^-8 of the value).  The expert layer rounds y and
out to bf16 (a relative RMS of 1.7e-3 each) and may round a few intermediate
values near a tie to the other neighbour: 5e-3 relative RMS, as for bf16."""
import ctypes

import numpy as np
import pytest
import torch

import fp8_plain as plain
import synth
from parity import REL_RMS_TOL

pytestmark = pytest.mark.gpu
MOE_ERR_TIMEOUT, MOE_ERR_BAD_INDEX = 5, 6


@pytest.fixture(scope="module")
def moe():
    import routed_expert_ffn_02_gb300 as m
    return m


def randn(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def same(q, want):
    a, b = q.double(), want.double()
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(7e9), b.nan_to_num(7e9))


# ---- quantiser --------------------------------------------------------------

@pytest.mark.parametrize("rows,K", [(1, 128), (3, 256), (7, 384), (1, 16384), (129, 1152), (2000, 512)])
def test_quantize_rows(moe, rows, K):
    x = randn((rows, K), rows + K)
    x *= torch.exp2(torch.randint(-30, 30, (rows, K // 128), device="cuda").float()).to(
        torch.bfloat16).repeat_interleave(128, 1)
    q, s = moe.moe_quantize_rows(x)
    want, b = plain.quantize_rows(x)
    assert torch.equal(s.long(), b) and same(q, want)


def test_quantize_special_values(moe):
    x = randn((8, 256), 5)
    x[0, 3] = float("inf")          # not finite: NaN, outside the block's maximum
    x[1, 7] = float("nan")
    x[2, 130] = float("-inf")
    x[3, :128] = 0                  # empty block: the smallest scale
    x[4] = 0
    x[4, 0] = torch.finfo(torch.bfloat16).tiny / 128      # subnormal
    x[5, :128] = torch.finfo(torch.bfloat16).max
    x[6, :128] = 448.0              # exactly the largest value: scale 1
    x[7, :128] = 450.0              # one bf16 step above: scale 2
    q, s = moe.moe_quantize_rows(x)
    want, b = plain.quantize_rows(x)
    assert torch.equal(s.long(), b) and same(q, want)
    assert s[6, 0] == 127 and s[7, 0] == 128 and s[3, 0] == 0


@pytest.mark.parametrize("E,N,K", [(1, 128, 128), (3, 256, 384), (2, 640, 1152)])
def test_quantize_weights(moe, E, N, K):
    W = randn((E, N, K), N, 0.02)
    W[0, 0, 0] = float("nan")
    W[-1, -1, -1] = float("inf")
    q, s = moe.moe_quantize_weights(W)
    want, b = plain.quantize_weights(W)
    assert torch.equal(s.long(), b) and same(q, want)


# ---- grouped product -------------------------------------------------------

def product_case(moe, counts, N, K, seed=0, wide=True):
    rows, E = sum(counts), len(counts)
    x, W = randn((rows, K), seed), randn((E, N, K), seed + 1, 0.05)
    if wide:    # blocks of very different sizes, so that a wrong scale shows
        x *= torch.exp2(torch.randint(-6, 7, (rows, K // 128), device="cuda").float()).to(
            torch.bfloat16).repeat_interleave(128, 1)
        s = torch.exp2(torch.randint(-6, 7, (E, N // 128, K // 128), device="cuda").float())
        W *= s.to(torch.bfloat16).repeat_interleave(128, 1).repeat_interleave(128, 2)
    q, sq = moe.moe_quantize_rows(x) if rows else (x.to(torch.float8_e4m3fn), None)
    Wq, sW = moe.moe_quantize_weights(W)
    off = torch.tensor([0, *np.cumsum(counts)], dtype=torch.int32, device="cuda")
    return q, sq, off, Wq, sW


def check_product(y, q, sq, off, Wq, sW):
    want, mag = plain.product(q, sq, off, Wq, sW)
    K = q.shape[1]
    tol = 2.0 ** -8 * want.abs() + K * 2.0 ** -23 * mag
    over = (y.double() - want).abs() - tol
    assert bool((over <= 0).all()), f"worst {over.max().item():.3e} over, {(over > 0).sum().item()} values"


@pytest.mark.parametrize("counts", [[1], [2, 0, 5], [31, 32, 33], [0, 127, 128, 129, 0],
                                    [255, 256, 257, 1], [300, 7, 0, 640], [1000]],
                         ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("N,K", [(128, 128), (256, 512), (384, 640), (640, 1152), (1024, 256)])
def test_product(moe, counts, N, K):
    args = product_case(moe, counts, N, K, seed=N + K)
    ws = moe.Workspace(moe.grouped_gemm_fp8_workspace_size(sum(counts), len(counts)))
    y = moe.moe_grouped_gemm_fp8(*args, ws=ws)
    assert ws.status() == 0
    check_product(y, *args)
    assert torch.equal(y, moe.moe_grouped_gemm_fp8(*args, ws=ws)), "repeated run differs"


@pytest.mark.parametrize("counts", [[255, 256, 257, 1, 3900], [129, 0, 385, 33, 4000, 128, 31], [4097, 512]],
                         ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("N,K", [(128, 128), (384, 640), (640, 1152), (1024, 256)])
def test_product_many_rows(moe, counts, N, K):
    """More than 4096 rows: the CTA-pair kernel beside the one-CTA kernel."""
    test_product(moe, counts, N, K)


@pytest.mark.parametrize("counts,N,K", [([1], 16384, 256), ([40], 256, 16384), ([200], 384, 16384),
                                        ([3] * 1024, 128, 256), ([0, 4097, 0, 12], 512, 2048)])
def test_product_limits(moe, counts, N, K):
    args = product_case(moe, counts, N, K, seed=3)
    check_product(moe.moe_grouped_gemm_fp8(*args), *args)


def test_product_nan_scale_stays_in_its_rows(moe):
    """A NaN scale or value reaches its own row (or column) only."""
    q, sq, off, Wq, sW = product_case(moe, [5, 140], 256, 384, wide=False)
    sq[3, 1] = 255
    sq[60, 0] = 255
    y = moe.moe_grouped_gemm_fp8(q, sq, off, Wq, sW)
    bad = torch.isnan(y).any(1).nonzero().flatten().tolist()
    assert bad == [3, 60]
    sW[1, 1, 2] = 255
    y = moe.moe_grouped_gemm_fp8(q, sq, off, Wq, sW)
    assert torch.isnan(y[5:, 128:]).all()
    assert torch.isnan(y).any(1).nonzero().flatten().tolist() == [3, *range(5, 145)]
    assert not torch.isnan(y[5:60, :128]).any()


@pytest.mark.parametrize("off,written", [([0, 5, 3, 10], 10), ([2, 4, 6, 10], None),
                                         ([0, 4, 6, 9], 9), ([0, 4, 6, 90], None),
                                         ([-3, 4, 6, 10], None), ([0, 2**30, -5, 10], None)])
def test_product_bad_offsets(moe, off, written):
    """Offsets that do not partition the rows are recorded; nothing is written
    out of range."""
    q, sq, _, Wq, sW = product_case(moe, [4, 2, 4], 128, 128)
    y = torch.zeros((12, 128), dtype=torch.bfloat16, device="cuda")
    y[10:] = 7
    ws = moe.Workspace(moe.grouped_gemm_fp8_workspace_size(10, 3))
    moe.moe_grouped_gemm_fp8(q, sq, torch.tensor(off, dtype=torch.int32, device="cuda"), Wq, sW,
                             y=y[:10], ws=ws)
    assert ws.status() == MOE_ERR_BAD_INDEX
    assert bool((y[10:] == 7).all())
    if written is not None:
        assert bool((y[written:10] == 0).all())


@pytest.mark.parametrize("rows", [10, 300])
@pytest.mark.parametrize("off,lo,hi", [([0, 7], 0, 7), ([2, 10**6], 2, None), ([-5, 4], 0, 4), ([9, 3], 0, 0)])
def test_product_bad_offsets_of_one_group(moe, rows, off, lo, hi):
    """One group takes no planner launch: the same rules hold."""
    q, sq, _, Wq, sW = product_case(moe, [rows], 256, 256)
    good = moe.moe_grouped_gemm_fp8(q, sq, torch.tensor([0, rows], dtype=torch.int32, device="cuda"), Wq, sW)
    y = torch.zeros((rows + 2, 256), dtype=torch.bfloat16, device="cuda")
    ws = moe.Workspace(moe.grouped_gemm_fp8_workspace_size(rows, 1))
    moe.moe_grouped_gemm_fp8(q, sq, torch.tensor(off, dtype=torch.int32, device="cuda"), Wq, sW,
                             y=y[:rows], ws=ws)
    assert ws.status() == MOE_ERR_BAD_INDEX
    hi = rows if hi is None else hi
    assert torch.equal(y[lo:hi], good[lo:hi])
    assert not y[:lo].any() and not y[hi:].any()


def test_product_as_input_gradient(moe):
    """dX = dY W by the same entry point on the transposed matrix, whose
    blocks keep their scales."""
    q, sq, off, Wq, sW = product_case(moe, [70, 9], 256, 384)
    dy, s_dy = moe.moe_quantize_rows(randn((79, 256), 9))
    Wt, sWt = Wq.transpose(1, 2).contiguous(), sW.transpose(1, 2).contiguous()
    dx = moe.moe_grouped_gemm_fp8(dy, s_dy, off, Wt, sWt)
    check_product(dx, dy, s_dy, off, Wt, sWt)


# ---- experts and layer ----------------------------------------------------

def layer_case(moe, T, E, k, H, I, zipf=None, seed=0):
    dev = torch.device("cuda")
    W = synth.make_weights(E, H, I, seed=seed, device=dev)
    x = synth.make_x(T, H, seed=seed).to(dev)
    lg = synth.make_logits(T, E, seed=seed, zipf_s=zipf).to(dev)
    ex = moe.quantize_experts(*W)
    parts = (ex.gate, ex.gate_scales, ex.up, ex.up_scales, ex.down, ex.down_scales)
    return moe.Shape(T, E, k, H, I), lg, x, ex, parts


def rel_rms(got, want):
    d = got.double() - want
    return float((d.square().mean() / want.square().mean()).sqrt())


@pytest.mark.parametrize("T,E,k,H,I,zipf", [
    (1, 16, 2, 512, 256, None), (3, 16, 2, 512, 256, None), (64, 16, 2, 512, 256, None),
    (1, 1, 1, 256, 256, None), (130, 1, 1, 256, 512, None), (300, 5, 3, 768, 512, None),
    (700, 6, 2, 512, 256, 1.1), (24, 64, 8, 1024, 768, 1.1), (2049, 32, 8, 512, 256, 1.1),
    (5, 1024, 8, 256, 256, None), (4, 64, 8, 2048, 1024, 1.1)])
def test_layer(moe, T, E, k, H, I, zipf):
    shape, lg, x, ex, parts = layer_case(moe, T, E, k, H, I, zipf)
    idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
    gates = torch.empty((T, k), dtype=torch.float32, device="cuda")
    ws = moe.Workspace(moe.fp8_workspace_size(shape))
    out = moe.moe_forward_fp8(shape, lg, x, ex, topk_idx=idx, gates=gates, ws=ws)
    assert ws.status() == 0
    ridx, rgates = moe.moe_route(lg, k)
    assert torch.equal(idx, ridx) and torch.equal(gates, rgates)
    want, y = plain.layer(x, idx, gates, parts)
    assert rel_rms(out, want) <= REL_RMS_TOL
    assert torch.equal(out, moe.moe_forward_fp8(shape, lg, x, ex, ws=ws)), "repeated run differs"
    # the separate entry points give the same bits (above 128 tokens)
    counts, offsets, perm, inv = moe.moe_permute(idx, E)
    ys = moe.moe_expert_ffn_fp8(shape, x, perm, offsets, ex)
    assert rel_rms(ys[inv.long()].view(T, k, H), y) <= REL_RMS_TOL
    combined = moe.moe_combine(ys, inv, gates, T, k, H)
    if T > 128:
        assert torch.equal(combined, out)
    else:    # y kept in fp32: one rounding to bf16 (1.7e-3) and not two
        assert rel_rms(out, want) <= 2e-3 and rel_rms(out, combined.double()) <= REL_RMS_TOL


def test_layer_against_bf16_experts(moe):
    """The 8-bit layer stays near the bf16 one: e4m3 rounds to 1 part in 16 at
    worst, a relative RMS of 2.6e-2 per operand for values spread over a
    binade; x, three weights and h add up to well under 0.1."""
    shape, lg, x, ex, _ = layer_case(moe, 200, 16, 4, 1024, 512)
    W = synth.make_weights(16, 1024, 512, seed=0, device=torch.device("cuda"))
    ref = moe.moe_forward(shape, lg, x, *W)
    assert rel_rms(moe.moe_forward_fp8(shape, lg, x, ex), ref.double()) < 0.1


def test_layer_special_values(moe):
    """A token with NaN or inf in x gives NaN outputs for itself alone."""
    shape, lg, x, ex, _ = layer_case(moe, 40, 4, 2, 512, 256)
    ref = moe.moe_forward_fp8(shape, lg, x, ex)
    x[7, 100] = float("inf")
    x[9, 0] = float("nan")
    out = moe.moe_forward_fp8(shape, lg, x, ex)
    assert torch.isnan(out).any(1).nonzero().flatten().tolist() == [7, 9]
    rest = [t for t in range(40) if t not in (7, 9)]
    assert torch.equal(out[rest], ref[rest])


def test_empty_and_other_stream(moe):
    shape, lg, x, ex, _ = layer_case(moe, 33, 8, 2, 512, 256)
    assert moe.moe_forward_fp8(moe.Shape(0, 8, 2, 512, 256), lg[:0], x[:0], ex).shape == (0, 512)
    q, s = moe.moe_quantize_rows(x[:0])
    assert q.shape == (0, 512) and s.shape == (0, 4)
    ref = moe.moe_forward_fp8(shape, lg, x, ex)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ws = moe.Workspace(moe.fp8_workspace_size(shape))
        out = moe.moe_forward_fp8(shape, lg, x, ex, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, ref)


def test_decode_step_in_a_graph(moe):
    shape, lg, x, ex, _ = layer_case(moe, 2, 64, 8, 1024, 512, 1.1)
    ws = moe.Workspace(moe.fp8_workspace_size(shape))
    out = torch.empty((2, 1024), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        moe.moe_forward_fp8(shape, lg, x, ex, out=out, ws=ws)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        moe.moe_forward_fp8(shape, lg, x, ex, out=out, ws=ws, stream=s)
    for seed in (5, 6):
        lg.copy_(synth.make_logits(2, 64, seed=seed))
        x.copy_(synth.make_x(2, 1024, seed=seed))
        g.replay()
        assert torch.equal(out.clone(), moe.moe_forward_fp8(shape, lg, x, ex))


@pytest.mark.parametrize("T,E,k,H,I", [(700, 6, 2, 512, 256), (64, 16, 2, 512, 256),
                                       (2500, 6, 2, 512, 256), (4, 16, 2, 512, 512)])
def test_wait_expiry(moe, T, E, k, H, I):
    """Waits given up after one cycle: the status says so, and the next call
    on the same workspace gives the outputs of the call before."""
    shape, lg, x, ex, _ = layer_case(moe, T, E, k, H, I, 1.1)
    ws = moe.Workspace(moe.fp8_workspace_size(shape))
    ref = moe.moe_forward_fp8(shape, lg, x, ex, ws=ws)
    assert ws.status() == 0
    moe.debug_set_wait_limit(1)
    try:
        moe.moe_forward_fp8(shape, lg, x, ex, ws=ws)
        torch.cuda.synchronize()
    finally:
        moe.debug_set_wait_limit(0)
    assert ws.status(clear=True) == MOE_ERR_TIMEOUT
    for _ in range(2):
        assert torch.equal(moe.moe_forward_fp8(shape, lg, x, ex, ws=ws), ref)
    assert ws.status() == 0
