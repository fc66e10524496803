"""GPU: the bf16 product with bias, activation and residual against its plain
64-bit form.

Tolerance.  The terms are exact in fp32; their sum, with the bias, is off by at
most K 2^-23 times the sum of the magnitudes (fp32 additions with truncating
adders, in any order).  An activation passes that on with a slope of at most
1.13 (gelu; silu 1.1) and is itself evaluated within (16 + 2|v|) 2^-23 of |v|:
the fast exponential's error is 2 + 1.2|v| units in the last place (2^-23), a
sigmoid passes on at most all of it, and the division, the products and erf add
a few units each.  The residual's addition rounds once in fp32 (2^-24), and a
bf16 result once more (2^-8)."""
import pytest
import torch

import train_plain as plain

pytestmark = pytest.mark.gpu
MOE_ERR_TIMEOUT, MOE_ERR_BAD_INDEX = 5, 6


@pytest.fixture(scope="module")
def moe():
    import routed_expert_ffn_02_gb300 as m
    return m


def make(rows, E, N, K, seed, bias=True, residual=True, skew=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, W = randn(rows, K).to(torch.bfloat16), (randn(E, N, K) * K ** -0.5).to(torch.bfloat16)
    b = randn(E, N) if bias else None
    r = randn(rows, N).to(torch.bfloat16) if residual else None
    counts = torch.bincount((randn(rows, E) - skew * torch.log(torch.randperm(E, generator=g, device="cuda") + 1.0)).argmax(1),
                            minlength=E)
    off = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    return x, W, off, b, r


def check(y, x, W, off, b, act, r):
    want, v, mag = plain.product(x, W, off, b, act, r)
    K = x.shape[1]
    tol = 1.13 * (K + 1) * plain.ADD * mag + (16 + 2 * v.abs()) * plain.ADD * v.abs() + 2.0 ** -24 * want.abs()
    if y.dtype is torch.bfloat16:
        tol = tol + plain.U * (want.abs() + tol)
    bad = (y.double() - want).abs() > tol + 1e-30
    assert not bad.any(), (bad.sum().item(), bad.nonzero()[0].tolist())


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,N,K", [(1, 256, 64), (5, 17, 8), (33, 300, 200), (300, 640, 1160)])
def test_dense(moe, rows, N, K, out, act):
    x, W, _, b, r = make(rows, 1, N, K, rows + N)
    y = moe.moe_grouped_gemm(x, W, bias=b, activation=act, residual=r, out_dtype=out)
    check(y, x, W, None, b, act, r)


@pytest.mark.parametrize("rows,E,N,K", [(1, 4, 64, 64), (777, 48, 650, 1160), (40, 30, 1000, 72), (2000, 7, 256, 128),
                                        (1500, 3, 31, 520), (300, 1024, 16, 16), (5000, 2, 1, 256), (64, 2, 4096, 4096)])
@pytest.mark.parametrize("bias,residual", [(True, False), (False, True)])
def test_groups(moe, rows, E, N, K, bias, residual):
    x, W, off, b, r = make(rows, E, N, K, rows + E, bias, residual)
    ws = moe.Workspace(moe.grouped_gemm_workspace_size(rows, E, N, K))
    y = moe.moe_grouped_gemm(x, W, off, bias=b, activation="silu", residual=r, ws=ws)
    assert ws.status() == 0
    check(y, x, W, off, b, "silu", r)


@pytest.mark.parametrize("rows", [15, 16, 17, 31, 32, 33, 255, 256, 257, 512, 513])
@pytest.mark.parametrize("listed", [False, True])
def test_row_counts_at_the_tiles_edges(moe, rows, listed):
    x, W, off, b, r = make(rows, 1, 272, 136, rows)
    y = moe.moe_grouped_gemm(x, W, off if listed else None, bias=b, residual=r, out_dtype=torch.float32)
    check(y, x, W, None, b, "none", r)


@pytest.mark.parametrize("rows", [1, 2, 3, 4])
@pytest.mark.parametrize("N,K", [(1, 8), (5, 520), (384, 4096), (1001, 1000), (130, 16384), (7, 65536)])
@pytest.mark.parametrize("act,out", [("silu", torch.bfloat16), ("relu", torch.float32)])
def test_single_tokens(moe, rows, N, K, act, out):
    """Up to three rows stream the weights on the CUDA cores."""
    x, W, _, b, r = make(rows, 1, N, K, rows + N)
    y = torch.full((rows + 2, N), 7.0, dtype=out, device="cuda")
    moe.moe_grouped_gemm(x, W, bias=b, activation=act, residual=r, out_dtype=out, y=y[1:1 + rows] if N % 8 == 0 else y[:rows])
    at = y[1:1 + rows] if N % 8 == 0 else y[:rows]
    check(at, x, W, None, b, act, r)
    assert (y[rows + 1:] == 7).all()


@pytest.mark.parametrize("rows,N,K", [(1, 4096, 4096), (24, 384, 4096), (4, 4096, 4096), (32, 1001, 1032), (2, 8, 65536), (17, 16640, 1024),
                                      (32, 9000, 2056), (5, 300, 1024)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_few_rows_of_long_k(moe, rows, N, K, out):
    """K split over the pairs of a cluster, or too many columns for that."""
    x, W, _, b, r = make(rows, 1, N, K, rows + N)
    ws = moe.Workspace(moe.grouped_gemm_workspace_size(rows, 1, N, K))
    y = torch.full((rows + 2, N), 7.0, dtype=out, device="cuda")
    moe.moe_grouped_gemm(x, W, bias=b, activation="gelu", residual=r, out_dtype=out, y=y[:rows], ws=ws)
    assert ws.status() == 0 and (y[rows:] == 7).all()
    check(y[:rows], x, W, None, b, "gelu", r)


@pytest.mark.parametrize("N,out", [(16400, torch.bfloat16), (16401, torch.float32)])
def test_offsets_beyond_32_bits(moe, N, out):
    rows = 140_000
    x, W, _, b, _ = make(rows, 1, N, 64, 11, residual=False)
    r = torch.ones((rows, N), dtype=torch.bfloat16, device="cuda")
    y = moe.moe_grouped_gemm(x, W, bias=b, residual=r, out_dtype=out)
    at = torch.cat([torch.arange(0, 3), torch.arange(130_900, 130_960), torch.arange(rows - 70, rows)]).cuda()
    check(y[at], x[at], W, None, b, "none", r[at])


def test_no_rows(moe):
    x, W, off, b, _ = make(0, 3, 64, 64, 1, residual=False, skew=0.0)
    assert moe.moe_grouped_gemm(x, W, off, bias=b).shape == (0, 64)


@pytest.mark.parametrize("rows", [3, 300])
def test_rows_outside_are_left_alone(moe, rows):
    """A result inside a larger tensor: what is before and behind it stays."""
    x, W, off, b, _ = make(rows, 1, 200, 64, 3)
    whole = torch.full((rows + 40, 200), 7.0, dtype=torch.bfloat16, device="cuda")
    y = whole[20:20 + rows]
    moe.moe_grouped_gemm(x, W, bias=b, y=y)
    check(y, x, W, None, b, "none", None)
    assert (whole[:20] == 7).all() and (whole[20 + rows:] == 7).all()


def test_result_over_its_residual(moe):
    x, W, _, b, r = make(200, 1, 512, 256, 4)
    want = moe.moe_grouped_gemm(x, W, bias=b, activation="gelu", residual=r)
    assert moe.moe_grouped_gemm(x, W, bias=b, activation="gelu", residual=r, y=r) is r
    assert torch.equal(r, want)


def test_infinities_and_nan_stay_in_their_rows_and_columns(moe):
    x, W, _, b, r = make(70, 1, 300, 96, 5)
    x[3, 5], x[40, 0] = float("nan"), float("inf")
    b[0, 7], r[9, 11] = float("inf"), float("nan")
    y = moe.moe_grouped_gemm(x, W, bias=b, activation="relu", residual=r).float()
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[3], want[:, 7], want[9, 11] = True, True, True
    bad[40] = want[40] = False                 # each of +-inf, relu takes -inf to 0
    assert torch.equal(bad, want)
    assert torch.isnan(y[3]).all() and not torch.isnan(y[40]).any()


def test_offsets_that_are_no_offsets(moe):
    """Recorded; the rows of the groups that are left are right, none is written twice."""
    x, W, _, b, _ = make(100, 4, 64, 64, 6)
    ws = moe.Workspace(moe.grouped_gemm_workspace_size(100, 4, 64, 64))
    y = torch.full((100, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 30, 20, 60, 80], dtype=torch.int32, device="cuda")
    moe.moe_grouped_gemm(x, W, off, bias=b, y=y, ws=ws)
    assert ws.status() == MOE_ERR_BAD_INDEX
    fixed = torch.tensor([0, 30, 30, 60, 80], dtype=torch.int32, device="cuda")
    check(y[:80], x[:80], W, fixed, b, "none", None)
    assert (y[80:] == 7).all()
    moe.moe_grouped_gemm(x, W, torch.tensor([-5, 30, 2 ** 30, 7, 100], dtype=torch.int32, device="cuda"), bias=b, y=y, ws=ws)
    assert ws.status() == MOE_ERR_BAD_INDEX
    fixed = torch.tensor([0, 30, 100, 100, 100], dtype=torch.int32, device="cuda")
    check(y, x, W, fixed, b, "none", None)


def test_another_stream_and_a_graph(moe):
    x, W, off, b, r = make(500, 6, 384, 256, 7)
    want = moe.moe_grouped_gemm(x, W, off, bias=b, activation="silu", residual=r)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = moe.moe_grouped_gemm(x, W, off, bias=b, activation="silu", residual=r, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    ws = moe.Workspace(moe.grouped_gemm_workspace_size(500, 6, 384, 256))
    y = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_grouped_gemm(x, W, off, bias=b, activation="silu", residual=r, y=y, ws=ws)
    x2, _, off2, _, _ = make(500, 6, 384, 256, 8)
    x.copy_(x2), off.copy_(off2)
    graph.replay()
    torch.cuda.synchronize()
    check(y, x2, W, off2, b, "silu", r)
    assert ws.status() == 0


@pytest.mark.parametrize("rows,E", [(20, 1), (300, 1), (2000, 3), (40, 30)])
def test_waits_that_expire_leave_nothing_behind(moe, rows, E):
    x, W, off, b, r = make(rows, E, 1024, 2048, 9)
    ws = moe.Workspace(moe.grouped_gemm_workspace_size(rows, E, 1024, 2048))
    call = lambda: moe.moe_grouped_gemm(x, W, off, bias=b, residual=r, ws=ws)  # noqa: E731
    want = call()
    outs = []
    for _ in range(10):
        moe.debug_set_wait_limit(1)
        try:
            call()
        finally:
            moe.debug_set_wait_limit(0)
        outs.append(call())
    torch.cuda.synchronize()
    assert ws.status(clear=True) == MOE_ERR_TIMEOUT
    assert all(torch.equal(o, want) for o in outs)
