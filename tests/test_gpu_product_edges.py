"""GPU: the bf16 product at the ends of its ranges, against its plain 64-bit
form with test_gpu_product's bounds."""
import math

import pytest
import torch

import train_plain as plain
from test_gpu_product import check, make, moe  # noqa: F401  (moe: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ends", [None, (0, 2 ** 31 - 129), (0, 5, 2 ** 31 - 132, 2 ** 31 - 129)], ids=str)
def test_most_rows(moe, ends):  # noqa: F811
    """2^31 - 129 rows: a group's count and its number of chunks add up to more
    than 32 bits hold.  Every row is there."""
    rows, K = 2 ** 31 - 129, 8
    E = 1 if ends is None else len(ends) - 1
    g = torch.Generator(device="cuda")
    g.manual_seed(41)
    x = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=g)
    W = torch.randn((E, 1, K), generator=g, device="cuda").to(torch.bfloat16)
    b = torch.randn((E, 1), generator=g, device="cuda")
    off = None if ends is None else torch.tensor(ends, dtype=torch.int32, device="cuda")
    ws = moe.Workspace(moe.grouped_gemm_workspace_size(rows, E, 1, K))
    y = torch.full((rows, 1), float("nan"), dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm(x, W, off, bias=b, y=y, ws=ws)
    assert ws.status() == 0
    step = 1 << 27
    for r in range(0, rows, step):
        part = slice(r, min(r + step, rows))
        inside = None if ends is None else torch.tensor(ends).clamp(r, part.stop) - r
        check(y[part], x[part], W, inside, b, "none", None)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("by_bias", [False, True])
@pytest.mark.parametrize("rows,K", [(1, 8), (3, 8), (4, 8), (24, 1024), (300, 72)])
def test_gelu_keeps_its_digits(moe, rows, K, by_bias, out):  # noqa: F811
    """Arguments that are exact (one term, or the bias alone), down to -12.5: the
    relative error is that of the form in act_dev.cuh, at most 10.4 units of
    2^-23 (its comment adds them up); a bf16 result is rounded once more."""
    N = 1001
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + K)
    v = torch.rand((N, K), generator=g, device="cuda") * 12.49 - 12.5
    v[::4] = v[::4] + 11                               # some of them positive
    x = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
    if by_bias:
        W, b = torch.zeros((1, N, K), dtype=torch.bfloat16, device="cuda"), v[:, :1].t().contiguous()
        at = v[:, :1].double().t().expand(rows, N)
    else:
        x[torch.arange(rows), torch.arange(rows) % K] = 1
        W, b = v.to(torch.bfloat16)[None].contiguous(), None
        at = W[0].double().t()[torch.arange(rows, device="cuda") % K]
    y = moe.moe_grouped_gemm(x, W, bias=b, activation="gelu", out_dtype=out)
    want = at * 0.5 * torch.special.erfc(-at * math.sqrt(0.5))      # (torch's ndtr cancels, in 64 bits too)
    tol = 10.5 * 2.0 ** -23 + (2.0 ** -8 if out is torch.bfloat16 else 0.0)
    assert ((y.double() - want).abs() <= tol * want.abs()).all(), ((y.double() - want) / want).abs().max()


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
def test_an_activation_is_the_same_at_any_number_of_rows(moe, act):  # noqa: F811
    """Arguments that are exact: the kernel of up to three rows, the split one
    and the others give the same bits."""
    N, K = 8192, 1024
    v = torch.linspace(-90, 30, N, device="cuda")[None]
    W = torch.zeros((1, N, K), dtype=torch.bfloat16, device="cuda")
    out = [moe.moe_grouped_gemm(torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda"), W, bias=v, activation=act,
                                out_dtype=torch.float32) for rows in (1, 2, 3, 4, 40, 200)]
    for y in out[1:]:
        assert torch.equal(y, out[0][:1].expand_as(y))


@pytest.mark.parametrize("rows", [1, 40])
def test_silu_keeps_its_digits(moe, rows):  # noqa: F811
    """Arguments that are exact, from -87 on: |v| 2^-23 for 2^x's argument (its
    rounding and that of 1 / ln 2, half a unit each), 2^-22 for 2^x, 2^-24 for 1 + 2^x,
    2^-23 for the reciprocal, 2^-24 for the product."""
    v = torch.linspace(-87, 40, 8192, device="cuda")[None]
    y = moe.moe_grouped_gemm(torch.zeros((rows, 64), dtype=torch.bfloat16, device="cuda"),
                             torch.zeros((1, 8192, 64), dtype=torch.bfloat16, device="cuda"), bias=v, activation="silu",
                             out_dtype=torch.float32)
    want = v.double() * torch.sigmoid(v.double())
    assert ((y.double() - want).abs() <= (4 + v.abs()) * 2.0 ** -23 * want.abs()).all()


@pytest.mark.parametrize("rows", [1, 3, 5, 40, 300])
@pytest.mark.parametrize("K", [4096, 16392, 65536])
def test_long_sums_lose_nothing(moe, rows, K):  # noqa: F811
    """Beside the bound per element, which grows with K as the terms' magnitudes
    do: over the whole result, K additions of at most 2^-23 of the sum so far (no
    larger than the sum itself, in the mean over independent terms).  A block of
    128 that is left out is sqrt(128 / K) of the result: six times the bound at
    65536, more below."""
    x, W, _, _, _ = make(rows, 1, 96, K, rows, False, False)
    y = moe.moe_grouped_gemm(x, W, out_dtype=torch.float32)
    assert plain.rel_rms(y, plain.product(x, W, None, None, "none", None)[0]) <= K * 2.0 ** -23
