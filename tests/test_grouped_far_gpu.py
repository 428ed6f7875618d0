"""cvx_linear_grouped with x at the limit of rows found by their number: 2^31 bytes from first to last.  All of
x but the rows that are named holds NaN, or a large number where integers have none."""
import pytest
import torch

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

from conv2d_batchnorm_activation_amd import cvx  # noqa: E402

BF16, E4M3, I8 = cvx.CVX_DT_BF16, cvx.CVX_DT_E4M3, cvx.CVX_DT_I8
DT = {BF16: torch.bfloat16, E4M3: torch.float8_e4m3fn, I8: torch.int8}


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# tokens, stride and channels of an x of exactly 2^31 bytes
LIMIT = {BF16: (1024, 1049600, 1024), E4M3: (2048, 1049088, 512), I8: (2048, 1049088, 512)}


@pytest.mark.parametrize("held", [BF16, E4M3, I8])
@pytest.mark.parametrize("sizes,co,kind", [([3, 0, 4], 36, "few"), ([16, 20], 68, "few"), ([40, 9, 0, 30], 1284, "tile"),
                                           ([300, 80], 2052, "tile")])
def test_rows_at_the_limit(held, sizes, co, kind):
    tokens, stride, ci = LIMIT[held]
    es = 2 if held == BF16 else 1
    assert ((tokens - 1) * stride + ci) * es == 1 << 31
    g = torch.Generator(device=DEV).manual_seed(co)
    buf = torch.full(((1 << 31) // es,), 127 if held == I8 else 0, dtype=torch.int8 if held == I8 else torch.uint8 if es == 1 else torch.int16,
                     device=DEV)
    if held != I8:
        buf.view(torch.uint8).fill_(255)  # NaN in either type
    x = torch.as_strided(buf.view(DT[held]), (tokens, ci), (stride, 1))
    near = [0, 1, tokens // 2 - 1, tokens // 2, tokens - 2, tokens - 1]
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    values = rnd(len(near), ci)
    values = (values * 40).round().clamp(-127, 127) if held == I8 else values
    for i, r in enumerate(near):
        x[r].copy_(values[i])
    rows, n = sum(sizes), len(sizes)
    w = rnd(n, co, ci)
    w = ((w * 40).round().clamp(-127, 127) if held == I8 else w / ci ** 0.5).to(DT[held])
    pick = torch.randint(0, len(near), (rows,), generator=g, device=DEV)
    pick[-1] = len(near) - 1
    ids = torch.tensor(near, device=DEV)[pick].to(torch.int32)
    none = torch.zeros(rows, dtype=torch.bool, device=DEV)
    for i, r in enumerate((tokens, -1, 2 ** 31 - 1, -2 ** 31)):  # name no row
        ids[i % (rows - 1)], none[i % (rows - 1)] = r, True
    offset = torch.cat([torch.zeros(1), torch.tensor(sizes).cumsum(0)]).to(torch.int32).to(DEV)
    bias = rnd(n, co)
    sx = None if held == BF16 else torch.full((tokens,), 2.0 ** -8, device=DEV)
    y = torch.full((rows, co), 7.0, dtype=torch.bfloat16, device=DEV)
    d = cvx.make_grouped_desc(rows, tokens, n, ci, co, BF16, held, x_stride=stride)
    say(f"{cvx.cvx_linear_grouped_plan(d)} rows={rows} x of 2^31 bytes, held={held}")
    assert cvx.cvx_linear_grouped_plan(d).split()[1] == kind
    cvx.cvx_linear_grouped(d, x, w, offset, y, sx, None, bias, ids)
    torch.cuda.synchronize()
    xs = torch.stack([x[r] for r in near]).double()[pick] * ~none[:, None] * (1.0 if sx is None else 2.0 ** -8)
    a = 0
    for i, k in enumerate(sizes):
        wd = w[i].double()
        z, mag = xs[a:a + k] @ wd.t() + bias[i].double(), xs[a:a + k].abs() @ wd.abs().t() + bias[i].double().abs()
        # sums in fp32, each of whose steps rounds, and the output's rounding; e4m3 in the larger tiles loses 7*2^-13
        # of the largest product of eight, which is at most their sum
        tol = ((ci + 4) * 2.0 ** -24 + (7 * 2.0 ** -13 if held == E4M3 and rows > 64 * n else 0)) * mag
        tol = tol + 2.0 ** -8 * (z.abs() + tol)
        assert ((y[a:a + k].double() - z).abs() <= tol).all(), i
        a += k
