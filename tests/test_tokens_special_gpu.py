"""Infinities and NaN through the operators on tokens.  Through cvx_linear's epilogue: a
NaN sum is a NaN output under every activation, in each of the kernels, and touches
only the outputs whose definition holds it; finite outputs beside them keep the
tolerance of their case.  Through cvx_rmsnorm: sums that leave fp32's range."""
import pytest
import torch

from gpu_util import DEV, say
from test_linear_gpu import BF16, E4M3, F16, NONE, RELU, SILU, Case
from test_rmsnorm_gpu import F32, compare, inputs, run

pytestmark = pytest.mark.gpu

from conv2d_batchnorm_activation_amd import cvx  # noqa: E402

NAN, INF = float("nan"), float("inf")

SHAPES = [
    # tokens, c_in, c_out: one token; 8, 16, 32 and 64 a workgroup, of 16 and of 32 channels; blocks of 64
    # (16 bits; tiles in 8); the three tiles
    (1, 144, 100), (7, 144, 100), (12, 144, 100), (20, 144, 100), (60, 144, 100), (60, 64, 4100), (100, 2064, 132),
    (100, 144, 100), (1000, 80, 4092), (4097, 48, 3588),
]


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def poison(c):
    """Plants NaN and infinities in what the case reads."""
    last = c.t - 1
    if c.t > 3:
        if c.x8:
            c.x.view(torch.uint8)[last, 9] = 0x7f  # e4m3's NaN
            c.sx[2] = NAN                          # a row that the norm marked
        else:
            c.x[last, 9] = NAN
    c.bias[5] = NAN
    c.bias[9] = -INF
    c.bias[17] = INF
    if c.res is not None:
        c.res[0, 30] = NAN
    if c.rank:
        c.ids[0] = 1 if c.t > 1 else 0
        c.a[2 % c.n, 3, 5] = NAN
        c.b[2 % c.n, 40, 1] = INF


@pytest.mark.parametrize("x8", [False, True], ids=["x16", "x8"])
@pytest.mark.parametrize("act", [NONE, RELU, SILU], ids=["none", "relu", "silu"])
@pytest.mark.parametrize("shape", SHAPES, ids=["x".join(map(str, s)) for s in SHAPES])
def test_linear_keeps_nan_through_the_activation(shape, act, x8):
    t, ci, co = shape
    for dt, rank, res in ((BF16, 8, 1), (F16, 0, 0), (F16, 16, 2)):
        c = Case(t + act + rank, t, ci, co, dt, x8, rank, 3 if rank else 0, act, res)
        poison(c)
        got = c.run()
        want, tol = c.definition()
        nan = torch.isnan(want)
        assert nan.any() and not nan.all()
        assert torch.equal(torch.isnan(got), nan), f"{c.plan}: NaN in other places than the definition's"
        exact = ~nan & ~(torch.isfinite(want) & torch.isfinite(tol))
        assert torch.equal(got[exact], want[exact]), f"{c.plan}: infinities"
        rest = ~nan & ~exact
        assert ((got - want).abs() <= tol)[rest].all(), c.plan


@pytest.mark.parametrize("c", [40, 5000, 30000])
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_rmsnorm_sums_that_leave_fp32(dt, c):
    # h is the fp32 sum of x and the residual, an infinity here, and so is `sum`; in the one
    # form that takes h in 64 bits the row is like any other
    x, r, g = inputs(c, 3, c, dt)
    x[1] *= 2.0 ** 100
    r[1] *= 2.0 ** 100
    x[1, 7] = r[1, 7] = 3e38
    fine = [0, 2]
    for out8 in (False, True):
        s, y, q = run(x, r, g, dt, out8)
        compare(x[fine], r[fine], g, dt, out8, (s[fine], y[fine], q[fine]), "rows beside")
        assert s[1, 7] == INF
        if out8 and dt == F32:
            compare(x, r, g, dt, out8, (s, y, q), "h in 64 bits")
        else:
            assert torch.isnan(y[1, 7]) and not y[1, :7].any() and not y[1, 8:].any()
            assert torch.isnan(q[1]) or not out8


@pytest.mark.parametrize("outliers", [1, 100], ids=["normal", "outliers"])
@pytest.mark.parametrize("tokens", [64, 65, 1000, 4097], ids=["few", "tile128x64", "tile128x128", "tile256x256"])
def test_linear_e4m3_sums_before_they_are_rounded(tokens, outliers):
    # every token is the same and the bias takes its sum away, so that what comes out is the
    # error of the sum itself.  Up to 64 tokens it is that of fp32 sums of exact products; beyond,
    # of eight consecutive channels' products up to seven may each lose 2^-13 of the largest,
    # itself at most the largest x times the largest w.  The bias is rounded to fp32, the output
    # once.
    ci, co, f = 1024, 3588, torch.float64
    g = torch.Generator().manual_seed(outliers)
    x = torch.randn(1, ci, generator=g) * 4
    x[:, ::64] *= outliers
    x = x.clamp(-448, 448).to(torch.float8_e4m3fn)
    w = (torch.randn(co, ci, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    xd, wd = x.to(f), w.to(f)
    z, mag = (xd @ wd.t())[0], (xd.abs() @ wd.abs().t())[0]
    bias = (-z).float()
    y = torch.full((tokens, co), NAN, dtype=torch.bfloat16, device=DEV)
    d = cvx.make_linear_desc(tokens, ci, co, BF16, E4M3)
    say(cvx.cvx_linear_plan(d))
    cvx.cvx_linear(d, x.view(torch.uint8).repeat(tokens, 1).to(DEV), w.to(DEV), y, torch.ones(tokens, device=DEV), None,
                   bias.to(DEV))
    err = y.cpu().to(f) - (z + bias.to(f))[None, :]
    tol = (ci + 2) * 2.0 ** -24 * mag
    if tokens > 64:
        tol = tol + 7 * 2.0 ** -13 * (xd.abs().view(-1, 8).amax(1) @ wd.abs().view(co, -1, 8).amax(2).t())
    tol = tol * (1 + 2.0 ** -8)
    say(f"error of the sums, of their size: {float(err.square().mean().sqrt() / z.square().mean().sqrt()):.3g}")
    assert (err.abs() <= tol).all()
