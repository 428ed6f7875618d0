"""Sums of 8-bit integers are exact 32-bit integers, in cvx_linear and cvx_linear_grouped.

Every row of x and of w is `half` channels of 64 to 127, the same values in another order (one order for all
rows, and negated in w), and sixteen channels of -3 to 3.  A sum climbs to some 2^28 by odd values and comes
back to one of at most 144, which bf16 holds: results are equal, while fp32 sums, which have even
values only from 2^24 up, are off by some hundreds.  Where eight waves share a row each still passes
2^25, and fp32 sums of theirs are off by some ten.

The longest rows there are, of -128 throughout, sum to 131056 * 2^14 = 2^31 - 2^18, a multiple of 2^18 below
2^31 that fp32 holds; times a power of two the output is its rounding to the output's type."""
import pytest
import torch

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

from conv2d_batchnorm_activation_amd import cvx  # noqa: E402

BF16, I8 = cvx.CVX_DT_BF16, cvx.CVX_DT_I8
LONGEST = (1 << 17) - 16


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def there_and_back(seed, half, *rows):
    """Tensors of rows [..., 2 * half + 16] whose products, of the first's rows with another's, sum to at most 144."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    order = torch.randperm(half, generator=g, device=DEV)
    out = []
    for i, r in enumerate(rows):
        up = torch.randint(64, 128, (*r, half), generator=g, device=DEV, dtype=torch.int8)
        end = torch.randint(-3, 4, (*r, 16), generator=g, device=DEV, dtype=torch.int8)
        out.append(torch.cat([up, up[..., order] if i == 0 else -up[..., order], end], -1))
    return out


def project(x, w, sx=1.0, plan=None):
    (t, ci), co = x.shape, w.shape[0]
    d = cvx.make_linear_desc(t, ci, co, BF16, I8)
    y = torch.full((t, co), float("nan"), dtype=torch.bfloat16, device=DEV)
    say(f"{cvx.cvx_linear_plan(d)} t={t} ci={ci} co={co}")
    assert plan is None or cvx.cvx_linear_plan(d).split()[1:3] == plan.split()
    cvx.cvx_linear(d, x, w, y, torch.full((t,), sx, device=DEV))
    torch.cuda.synchronize()
    return y.double()


def by_group(x, w, sizes, sx=1.0, plan=None, row_id=None):
    (t, ci), (n, co, _) = x.shape, w.shape
    rows = sum(sizes)
    offset = torch.cat([torch.zeros(1), torch.tensor(sizes).cumsum(0)]).to(torch.int32).to(DEV)
    d = cvx.make_grouped_desc(rows, t, n, ci, co, BF16, I8)
    y = torch.full((rows, co), float("nan"), dtype=torch.bfloat16, device=DEV)
    say(f"{cvx.cvx_linear_grouped_plan(d)} rows={rows} ci={ci} co={co}")
    assert plan is None or cvx.cvx_linear_grouped_plan(d).split()[1:3] == plan.split()
    cvx.cvx_linear_grouped(d, x, w, offset, y, torch.full((t,), sx, device=DEV), row_id=row_id)
    torch.cuda.synchronize()
    return y.double()


@pytest.mark.parametrize("t,co,plan", [
    (1, 68, "few 16x16"), (8, 4100, "few 32x16"), (16, 132, "few 16x16"), (13, 4100, "few 32x16"), (30, 260, "few 16x32"),
    (30, 4100, "few 32x32"), (60, 132, "few 16x64"), (60, 4100, "few 32x64"), (200, 516, "few 16x64"), (60, 8260, "tile 128x64"),
    (300, 1284, "tile 128x64"), (1500, 2564, "tile 128x128"), (2000, 8192, "tile 256x256")])
def test_projection(t, co, plan):
    x, w = there_and_back(t + co, 32760, (t,), (co,))
    got = project(x, w, plan=plan)
    want = torch.cat([x[a:a + 256].double() @ w.double().t() for a in range(0, t, 256)])
    assert want.abs().max() <= 144 and torch.equal(got, want)


@pytest.mark.parametrize("sizes,co,plan", [
    ([1], 68, "few 16x16"), ([5, 0, 3], 260, "few 16x16"), ([13, 1], 132, "few 16x16"), ([70], 516, "few 16x16"),
    ([30, 40, 0, 9], 1028, "tile 128x64"), ([100, 3, 160], 8188, "tile 128x128"), ([700, 30, 900], 8188, "tile 256x256"),
    ([2, 5] * 30, 1028, "tile 128x64")])
@pytest.mark.parametrize("gather", [False, True])
def test_by_group(sizes, co, plan, gather):
    rows, n = sum(sizes), len(sizes)
    x, w = there_and_back(rows + co, 32760, (rows,), (n, co))
    ids = torch.randperm(rows, generator=torch.Generator().manual_seed(rows)).to(DEV)
    got = by_group(x, w, sizes, plan=plan, row_id=ids.to(torch.int32) if gather else None)
    a = 0
    for d, k in enumerate(sizes):
        xs = x[ids[a:a + k]] if gather else x[a:a + k]
        want = xs.double() @ w[d].double().t()
        assert (k == 0 or want.abs().max() <= 144) and torch.equal(got[a:a + k], want), d
        a += k


@pytest.mark.parametrize("t,co", [(1, 20), (20, 36), (64, 8260), (100, 260), (400, 2052)])
def test_the_longest_rows(t, co):
    x = torch.full((t, LONGEST), -128, dtype=torch.int8, device=DEV)
    w = torch.full((co, LONGEST), -128, dtype=torch.int8, device=DEV)
    w[1::2] = 127
    w[2::4, 5] = -127
    want = torch.full((co,), LONGEST * 128 * 128.0, dtype=torch.float64)
    want[1::2] = -LONGEST * 128 * 127.0
    want[2::4] -= 128
    want = (want.float() * 2.0 ** -24).bfloat16().double().to(DEV)  # an integer, rounded to fp32, then to the type
    got = project(x, w, 2.0 ** -24)
    assert torch.equal(got, want.expand(t, co))
    got = by_group(x, w[None], [t], 2.0 ** -24)
    assert torch.equal(got, want.expand(t, co))
