"""cvx_rmsnorm against its definition in 64 bits, element by element.

Tolerances, for a value v of the definition.  The kernel rounds h = x + r and the
product h*gamma*q to fp32, at most 2^-24 each, and the output once to its type,
at most eps/2 (or half the smallest subnormal): eps/2 + 5*2^-24 of |v| covers
them and their products.  `sum` is h rounded twice.  A code is the nearest e4m3 value of u*(448/t): off by half a
step (2^-4 of the value, 2^-10 below 2^-6) plus four fp32 roundings; its scale
takes three."""
import pytest
import torch

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

from conv2d_batchnorm_activation_amd import cvx  # noqa: E402

F32, F16, BF16, E4M3 = cvx.CVX_DT_F32, cvx.CVX_DT_F16, cvx.CVX_DT_BF16, cvx.CVX_DT_E4M3
DT = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16, E4M3: torch.float8_e4m3fn}
EPS = 1e-5
U = 2.0 ** -24


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def half(dt):
    return torch.finfo(dt).eps / 2


def smallest(dt):
    return torch.finfo(dt).smallest_normal * torch.finfo(dt).eps


def definition(x, r, g, eps=EPS):
    h = x.double() + (r.double() if r is not None else 0.0)
    q = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    return h, q, h * g.double()


def strided(rows, c, stride, dt, fill, head=64):
    """A [rows][c] view with rows `stride` apart inside a buffer filled with `fill`."""
    buf = torch.full((head + rows * stride + head,), 0.0, dtype=torch.float32).fill_(fill).to(dt).to(DEV)
    return buf, buf[head:head + rows * stride].view(rows, stride)[:, :c]


def untouched(buf, view_rows, c, stride, head=64):
    """Everything outside the view still holds its fill (NaN)."""
    b = buf.float().cpu()
    inner = b[head:-head].view(view_rows, stride)[:, c:]
    return bool(torch.isnan(b[:head]).all() and torch.isnan(b[-head:]).all() and torch.isnan(inner).all())


def check(got, want, tol, what):
    # infinities and NaN of the definition (rows whose input holds one) have to be there as they are
    same = (torch.isnan(got) & torch.isnan(want)) | (got == want)
    bad = ~(((got - want).abs() <= tol) & torch.isfinite(want)) & ~same
    assert not bad.any(), f"{what}: {int(bad.sum())} out of bound, first at {bad.nonzero()[0].tolist()}: " \
                          f"{got[bad][0].item()!r} for {want[bad][0].item()!r}"


def run(x, r, g, dt, out8, pads=(0, 0, 0, 0), eps=EPS, in_place=None, want_sum=True):
    """pads: extra elements between the rows of x, residual, sum, y.  in_place: "x" or "r" for the sum."""
    rows, c = x.shape
    tdt, odt = DT[dt], DT[E4M3] if out8 else DT[dt]
    _, xv = strided(rows, c, c + pads[0], tdt, float("nan"))
    xv.copy_(x)
    rv = None
    if r is not None:
        _, rv = strided(rows, c, c + pads[1], tdt, float("nan"))
        rv.copy_(r)
    ss = c + pads[2]
    if in_place:
        sv = xv if in_place == "x" else rv
        sbuf, ss = None, sv.stride(0)
    elif want_sum:
        sbuf, sv = strided(rows, c, ss, tdt, float("nan"))
    else:
        sbuf = sv = None
    ybuf, yv = strided(rows, c, c + pads[3], odt, float("nan"))
    qbuf = torch.full((rows + 32,), float("nan"), device=DEV)
    d = cvx.make_rmsnorm_desc(rows, c, dt, E4M3 if out8 else dt, eps, x_stride=xv.stride(0) if rows > 1 else 0,
                              res_stride=(rv.stride(0) if rows > 1 else 0) if rv is not None else 0,
                              sum_stride=(ss if rows > 1 else 0), y_stride=c + pads[3])
    say(f"rmsnorm rows={rows} c={c} dt={dt} out8={out8} res={r is not None} pads={pads} in_place={in_place}")
    cvx.cvx_rmsnorm(d, xv, rv, g.to(DEV), sv, yv, qbuf[16:16 + rows] if out8 else None)
    torch.cuda.synchronize()
    assert untouched(ybuf, rows, c, c + pads[3])
    if sbuf is not None:
        assert untouched(sbuf, rows, c, ss)
    q = qbuf.cpu()
    assert torch.isnan(q[:16]).all() and torch.isnan(q[16 + rows:]).all()
    return (sv.cpu().double() if sv is not None else None), yv.cpu().float().double(), q[16:16 + rows].double()


def compare(x, r, g, dt, out8, got, what):
    s, y, scale = got
    h, q, u = definition(x, r, g)
    tdt = DT[dt]
    if s is not None:
        # rounding to nearest takes what is at least half a step past the largest value to infinity
        top = torch.finfo(tdt).max
        over = h.abs() >= top * (1 + half(tdt) / 2)
        assert torch.equal(s[over], torch.sign(h[over]) * float("inf"))
        check(s[~over], h[~over], ((half(tdt) + U) * h.abs() + smallest(tdt))[~over], f"{what} sum")
    if out8:
        t = u.abs().amax(1, keepdim=True)
        check(scale[:, None], t * q / 448, 3 * U * t * q / 448, f"{what} scale")
        v = torch.where(t > 0, u * 448 / torch.where(t > 0, t, 1.0), 0.0)
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
        check(y, v, step / 2 + 4 * U * v.abs(), f"{what} codes")
        assert not (y.abs() > 448).any()
    else:
        v = u * q
        check(y, v, (half(tdt) + 5 * U) * v.abs() + smallest(tdt), what)


def inputs(seed, rows, c, dt, residual=True, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, c, generator=g) * scale).to(DT[dt])
    r = (torch.randn(rows, c, generator=g) * 3 * scale).to(DT[dt]) if residual else None
    gamma = 1 + 0.3 * torch.randn(c, generator=g)
    return x, r, gamma


CASES = [
    # rows, c, residual, pads (x, residual, sum, y)
    (1, 1, True, (0, 0, 0, 0)), (3, 2, False, (1, 0, 0, 3)), (5, 7, True, (0, 0, 0, 0)), (2, 8, True, (8, 8, 8, 8)),
    (9, 31, True, (2, 1, 3, 5)), (4, 255, False, (0, 0, 0, 1)), (6, 512, True, (0, 0, 0, 0)),
    (5, 513, True, (0, 0, 0, 0)), (7, 1025, False, (7, 0, 0, 0)), (2, 2048, True, (0, 0, 0, 0)),
    (3, 2049, True, (3, 1, 0, 0)), (2, 4096, True, (0, 0, 16, 0)), (3, 5003, True, (0, 0, 0, 0)),
    (2, 8192, True, (0, 0, 0, 0)), (2, 8200, False, (0, 0, 0, 0)), (3, 16387, True, (0, 5, 0, 1)),
    (2, 32768, True, (0, 0, 0, 0)), (2, 32777, True, (0, 0, 3, 0)), (1, 70001, False, (0, 0, 0, 0)),
    (1030, 64, True, (0, 0, 0, 0)),
]


@pytest.mark.parametrize("out8", [False, True], ids=["same", "e4m3"])
@pytest.mark.parametrize("dt", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}x{c[1]}" for c in CASES])
def test_rmsnorm(case, dt, out8):
    rows, c, residual, pads = case
    x, r, g = inputs(rows * 100003 + c, rows, c, dt, residual)
    compare(x, r, g, dt, out8, run(x, r, g, dt, out8, pads), f"{rows}x{c}")


@pytest.mark.parametrize("out8", [False, True], ids=["same", "e4m3"])
@pytest.mark.parametrize("dt", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,c", [(257, 1500), (260, 4091), (514, 4004), (515, 8190)])
def test_rmsnorm_rows_that_fill_the_device(rows, c, dt, out8):
    # of so many rows each is fewer threads'
    x, r, g = inputs(rows + c, rows, c, dt)
    compare(x, r, g, dt, out8, run(x, r, g, dt, out8, (3, 0, 0, 1)), f"{rows}x{c}")


@pytest.mark.parametrize("out8", [False, True], ids=["same", "e4m3"])
@pytest.mark.parametrize("where", ["x", "r"])
@pytest.mark.parametrize("c", [40, 2051, 40000])
def test_rmsnorm_sum_in_place(c, where, out8):
    x, r, g = inputs(c, 3, c, BF16)
    compare(x, r, g, BF16, out8, run(x, r, g, BF16, out8, (5, 5, 0, 0), in_place=where), f"in place {where}")


def test_rmsnorm_without_a_sum():
    x, r, g = inputs(5, 4, 100, F16)
    compare(x, r, g, F16, False, run(x, r, g, F16, False, want_sum=False), "no sum")


@pytest.mark.parametrize("dt,scale", [(F32, 1e30), (F32, 1e-30), (BF16, 1e30), (BF16, 1e-30), (F16, 1e4), (F16, 1e-5)])
def test_rmsnorm_large_and_small_values(dt, scale):
    # squares beyond fp32's range on either side; eps decides the small ones
    x, r, g = inputs(7, 4, 300, dt, scale=scale)
    compare(x, r, g, dt, False, run(x, r, g, dt, False), f"scale {scale}")
    compare(x, r, g, dt, True, run(x, r, g, dt, True), f"scale {scale} e4m3")


@pytest.mark.parametrize("out8", [False, True], ids=["same", "e4m3"])
def test_rmsnorm_zero_rows(out8):
    x, r, g = inputs(8, 4, 200, BF16)
    x[1] = 0
    r[1] = 0
    got = run(x, r, g, BF16, out8)
    compare(x, r, g, BF16, out8, got, "zero row")
    assert not got[1][1].any()


@pytest.mark.parametrize("c", [100, 3001, 40000])
def test_rmsnorm_infinities_and_nans_stay_in_their_rows(c):
    x, r, g = inputs(9, 6, c, BF16)
    x[1, 5] = float("nan")
    x[3, c - 1] = float("inf")
    fine = [0, 2, 4, 5]
    for out8 in (False, True):
        s, y, q = run(x, r, g, BF16, out8)
        compare(x[fine], r[fine], g, BF16, out8, (s[fine], y[fine], q[fine]), "rows beside")
        if out8:
            assert torch.isnan(q[1]) and torch.isnan(q[3])
        else:
            assert torch.isnan(y[1]).all()
            assert torch.isnan(y[3, c - 1]) and not y[3, :c - 1].any()


def test_rmsnorm_an_infinity_that_gamma_hides():
    x, r, g = inputs(10, 3, 72, BF16)
    x[1, 7] = float("-inf")
    g[7] = 0
    s, y, q = run(x, r, g, BF16, True)
    assert torch.isnan(q[1]) and torch.isfinite(q[0]) and torch.isfinite(q[2])
    y = run(x, r, g, BF16, False)[1]
    assert torch.isnan(y[1, 7]) and not y[1, :7].any() and not y[1, 8:].any()


def test_rmsnorm_many_rows():
    # more rows than one launch takes
    rows, c = (1 << 20) + 37, 8
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(rows, c, generator=g, device=DEV, dtype=torch.float32).to(torch.float16)
    gamma = torch.ones(c, device=DEV)
    y = torch.full((rows, c), float("nan"), device=DEV, dtype=torch.float16)
    say("rmsnorm many rows")
    cvx.cvx_rmsnorm(cvx.make_rmsnorm_desc(rows, c, F16, eps=EPS), x, None, gamma, None, y)
    h, q, u = definition(x.cpu(), None, gamma.cpu())
    check(y.cpu().double(), u * q, (half(torch.float16) + 5 * U) * (u * q).abs() + smallest(torch.float16), "many rows")
