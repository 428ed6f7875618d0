"""cvx_linear_grouped's sums of e4m3 values where groups have 64 rows or fewer on average.

Operands whose products are integers: in every eight channels one of 448*448 or its negative
(of the first 1024 channels), the others between -9 and 9.  All partial sums, in any order, are
integers below 2^24, which fp32 holds, and a whole sum of at most 256 is held by both output types:
there results are equal.  Sums that drop what lies 2^-13 below the largest of eight products lose the small ones,
which lie up to 2^-17.6 below."""
import pytest
import torch

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

from conv2d_batchnorm_activation_amd import cvx  # noqa: E402

F16, BF16, E4M3 = cvx.CVX_DT_F16, cvx.CVX_DT_BF16, cvx.CVX_DT_E4M3


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def rows_and_weights(seed, rows, n, ci, co):
    """x [rows][ci] and w [n][co][ci] whose products sum to small integers."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(1, 4, (rows, ci), generator=g).float()
    w = torch.randint(-3, 4, (n, co, ci), generator=g).float()
    x[:, ::8], w[:, :, ::8] = 448, 0
    m = min(ci, 1024) // 16 * 16  # as many of either sign as leave every partial sum below 2^24
    w[:, :, 0:m:16], w[:, :, 8:m:16] = 448, -448
    return x, w


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("sizes,ci,co,gather", [
    ([7, 9, 0, 64, 13] * 13, 2048, 644, False),  # the kind of tile that most shapes of few rows a group take
    ([8] * 128, 512, 768, True), ([1] * 80, 1040, 516, True), ([64, 1, 63] * 3, 272, 2052, False),
    ([33, 30, 64, 60], 1008, 1284, True), ([40, 2], 144, 8196, False), ([60] * 40, 528, 2052, True), ([5, 3], 4096, 64, False),
    ([64] * 3, 272, 1284, False), ([1, 127], 1040, 2052, True), ([32, 32], 8192, 2048, False), ([64, 0, 128], 8192, 1024, True)])
def test_small_products_beside_large_ones(sizes, ci, co, gather, dt):
    rows, n = sum(sizes), len(sizes)
    assert rows <= 64 * n
    x, w = rows_and_weights(rows + ci, rows, n, ci, co)
    want = torch.empty(rows, co, dtype=torch.float64)
    a = 0
    for d, k in enumerate(sizes):
        want[a:a + k] = x[a:a + k].double() @ w[d].double().t()
        a += k
    offset = torch.cat([torch.zeros(1), torch.tensor(sizes).cumsum(0)]).to(torch.int32)
    ids = torch.randperm(rows, generator=torch.Generator().manual_seed(1)) if gather else None
    xs = x[torch.argsort(ids)] if gather else x
    y = torch.full((rows, co), float("nan"), device=DEV, dtype=torch.bfloat16 if dt == BF16 else torch.float16)
    d = cvx.make_grouped_desc(rows, rows, n, ci, co, dt, E4M3)
    say(f"{cvx.cvx_linear_grouped_plan(d)} rows={rows} ci={ci} co={co}")
    e4m3 = torch.float8_e4m3fn
    cvx.cvx_linear_grouped(d, xs.to(DEV).to(e4m3), w.to(DEV).to(e4m3), offset.to(DEV), y, torch.ones(rows, device=DEV),
                           row_id=None if ids is None else ids.to(torch.int32).to(DEV))
    got = y.cpu().double()
    small = want.abs() <= 256
    assert small.double().mean() > 0.3
    assert torch.equal(got[small], want[small]), f"{int((got != want)[small].sum())} of {int(small.sum())} differ"
