"""GPU: the bf16 product at the ends of its ranges, against its plain 64-bit
form with test_gpu_product's bounds."""
import pytest
import torch

from test_gpu_product import check, moe  # noqa: F401  (moe: the fixture)

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
