"""cvx_gate against its definition in 64 bits, element by element.

Tolerances.  16- and 32-bit output: the activation is good to 8 units of fp32 (an exponential,
an addition, a quotient) where its exponent is small, and its exponential to |g|*2^-23 more of
the value; the product is rounded once more, and the output once, eps/2 or half the smallest
subnormal of its type.  Codes are the integers, or e4m3 values, nearest to u*(M*(1/t)), which both
sides take in 64 bits: equal for the activations that are exact.  Where an exponential comes in,
the two sides' u may differ by some 2^-50 of it, and a code where u*f lies that near to a
border: where another value's gate is the same and its factor a simple multiple, so that u/t
is a ratio of small integers.  The test of many values meets such pairs and takes its
64-bit values on the GPU, where the exponential is the same; the small tests' seeds have none.
y_scale is rounded once to fp32."""
import pytest
import torch

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

from conv2d_batchnorm_activation_amd import cvx  # noqa: E402

F32, F16, BF16, E4M3, I8 = cvx.CVX_DT_F32, cvx.CVX_DT_F16, cvx.CVX_DT_BF16, cvx.CVX_DT_E4M3, cvx.CVX_DT_I8
DT = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16, E4M3: torch.float8_e4m3fn, I8: torch.int8}
MOST = {E4M3: 448.0, I8: 127.0}
NONE, RELU, SILU = cvx.CVX_ACT_NONE, cvx.CVX_ACT_RELU, cvx.CVX_ACT_SILU
U = 2.0 ** -24


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def value(g, p, act):
    """u of rows in 64 bits."""
    g = g.double()
    u = g / (1 + torch.exp(-g)) if act == SILU else torch.clamp_min(g, 0) if act == RELU else g
    return u if p is None else u * p.double()


def nearest_e4m3(v):
    """v on the e4m3 grid: 3 fraction bits, exponents down to -6, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def strided(m, pad, fill):
    buf = torch.full((m.shape[0], m.shape[1] + pad), fill, dtype=m.dtype, device=DEV)
    buf[:, :m.shape[1]] = m.to(DEV)
    return buf[:, :m.shape[1]]


def run(g, p, dt, out, act, pads=(0, 0, 0), stream=None):
    rows, c = g.shape
    ybuf = torch.full((rows + 2, c + pads[2]), 99, dtype=torch.float32, device=DEV).to(DT[out])
    y = ybuf[1:-1, :c]
    q = torch.full((rows + 2,), float("nan"), device=DEV)
    gd, pd = strided(g, pads[0], float("nan")), None if p is None else strided(p, pads[1], float("nan"))
    d = cvx.make_gate_desc(rows, c, dt, out, act, c + pads[0], c + pads[1], c + pads[2])
    say(f"gate {rows}x{c} dt={dt} out={out} act={act} up={p is not None} pads={pads}")
    cvx.cvx_gate(d, gd, pd, y, q[1:-1] if out in MOST else None, stream)
    torch.cuda.synchronize()
    edge = torch.tensor(99.0).to(DT[out]).float()
    assert (ybuf[[0, -1]].float().cpu() == edge).all() and (ybuf[:, c:].float().cpu() == edge).all()
    assert torch.isnan(q[0]) and torch.isnan(q[-1])
    return y.float().cpu().double() if out != I8 else y.cpu().double(), q[1:-1].cpu().double()


def check(g, p, dt, out, act, pads=(0, 0, 0)):
    got, q = run(g, p, dt, out, act, pads)
    u = value(g, p, act)
    if out in MOST:
        t = u.abs().amax(1)
        v = u * torch.where(t > 0, MOST[out] * (1.0 / t), 0.0)[:, None]
        want = torch.round(v) if out == I8 else nearest_e4m3(v)
        assert torch.equal(got, want), (got != want).nonzero()[:3].tolist()
        fi = torch.finfo(torch.float32)
        assert ((q - t / MOST[out]).abs() <= 2 * U * t / MOST[out] + fi.smallest_normal * fi.eps).all()
        return
    fi = torch.finfo(DT[dt])
    part = (10 + (2 * g.double().abs() if act == SILU else 0)) * U * u.abs()
    tol = part + (fi.eps / 2) * (u.abs() + part) + fi.smallest_normal * fi.eps
    assert ((got - u).abs() <= tol).all()


def rows_of(seed, rows, c, dt, size=1.0):
    r = torch.Generator().manual_seed(seed)
    m = [(size * torch.randn(rows, c, generator=r) * torch.exp(torch.randn(c, generator=r) * 0.5)).to(DT[dt])
         for _ in range(2)]
    m[0][rows // 2] = 0  # a row of zeros
    return m


SIZES = [(1, 1), (1, 4096), (3, 7), (2, 64), (5, 513), (300, 1337), (33, 2048), (129, 4104), (7, 8200), (2, 14336), (3, 20481),
         (2, 40000), (37, 130), (1001, 300), (70, 512), (17, 128), (2, 33000)]


@pytest.mark.parametrize("rows,c", SIZES)
@pytest.mark.parametrize("dt,out", [(BF16, I8), (F16, E4M3), (F32, I8), (BF16, BF16), (F16, F16), (F32, F32)])
def test_gate(rows, c, dt, out):
    g, p = rows_of(rows + c, rows, c, dt)
    k = rows + c
    check(g, p, dt, out, (SILU, RELU, NONE)[k % 3] if k % 2 else SILU, ((5, 3, 1), (0, 0, 0), (8, 8, 16))[k % 3])


# a row's vectors to where its threads, or the vectors each holds, change: of 8 values, and of 4
WIDTHS = [n * v for v in (8, 4) for n in (8, 16, 32, 64, 128, 256, 512, 768, 1280, 2048, 2560 if v == 8 else 3000, 4096)] + [24576]


@pytest.mark.parametrize("c", WIDTHS)
def test_row_widths(c):
    dt, out = (BF16, I8) if c in WIDTHS[:12] else (F32, E4M3)
    for n in (c - 1, c, c + 1):
        g, p = rows_of(n, 19, n, dt)
        check(g, p, dt, out, SILU, (0, 0, 0) if n % 2 else (4, 8, 4))


@pytest.mark.parametrize("act", [NONE, RELU, SILU])
@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("dt,out", [(BF16, E4M3), (F16, I8), (F32, E4M3), (BF16, BF16), (F32, F32)])
def test_activations(act, up, dt, out):
    g, p = rows_of(act + 5, 70, 700, dt, 4.0)
    check(g, p if up else None, dt, out, act, (0, 2, 4))


@pytest.mark.parametrize("out", [BF16, E4M3, I8])
def test_one_tensor_twice_and_halves_of_one(out):
    g, _ = rows_of(3, 40, 512, BF16)
    d = g.to(DEV)
    y, q = torch.empty(40, 256, dtype=DT[out], device=DEV), torch.empty(40, device=DEV)
    for second in (d[:, 256:], d[:, :256]):
        say(f"gate of halves, out={out}")
        cvx.cvx_gate(cvx.make_gate_desc(40, 256, BF16, out, SILU, 512, 512), d[:, :256], second, y, q if out != BF16 else None)
        got = y.cpu()
        a, _ = run(g[:, :256].contiguous(), second.cpu().contiguous(), BF16, out, SILU)
        assert torch.equal(got.float().double() if out != I8 else got.double(), a)


def test_ties_go_to_even():
    g = torch.tensor([[2.0, 1.0, -1.0, 2 * 3 / 127.0, -2.0, 0.0, 2.0, 2.0]])
    got, q = run(g, None, F32, I8, NONE)
    assert got.tolist()[0] == [127, 64, -64, 3, -127, 0, 127, 127] and q[0] == torch.tensor(2 / 127.0).double()
    v = torch.tensor([[448.0, 17.0, 19.0, -17.0, 2.0 ** -10, 3 * 2.0 ** -10, 447.0, 432.0]])
    got, q = run(v, None, F32, E4M3, NONE)
    assert got.tolist()[0] == [448, 16, 20, -16, 0, 2.0 ** -8, 448, 448] and q[0] == 1.0


@pytest.mark.parametrize("c", [40, 3000, 40000])
def test_bad_rows(c):
    nan, inf = float("nan"), float("inf")
    g, p = torch.ones(7, c), torch.ones(7, c)
    g[1, 3], g[2, c - 1], p[3, c // 2], p[4, 0] = nan, inf, nan, -inf
    g[5, 1], p[5, 1] = 0.0, inf  # their product is a NaN
    for out in (I8, E4M3):
        got, q = run(g, p, F32, out, SILU)
        assert torch.isnan(q).tolist() == [False, True, True, True, True, True, False]
        assert (got[[0, 6]] == MOST[out]).all()
    got, _ = run(g, p, F32, F32, RELU)
    assert torch.isnan(got[1, 3]) and got[2, c - 1] == inf and torch.isnan(got[3, c // 2]) and got[4, 0] == -inf
    assert torch.isnan(got[5, 1]) and int(torch.isfinite(got).sum()) == 7 * c - 5


def test_the_widest_ranges():
    # products that leave fp32, its smallest values, and arguments whose exponential overflows
    big = torch.finfo(torch.float32).max
    g = torch.tensor([[big, big / 2, 1.0, -1.0], [1e-45, 2e-45, 0.0, 3e-45], [-800.0, 800.0, -90.0, -1e30], [5e-20, 1e-20, 0, 0]])
    p = torch.tensor([[big, big, 1.0, big], [1.0, 1.0, 1.0, 1.0], [1.0, 1.0, 1.0, 1.0], [5e-20, 1e-20, 1.0, 1.0]])
    for out in (I8, E4M3):
        got, q = run(g, p, F32, out, NONE)
        assert got[0, 0] == MOST[out] and got[0, 2] == 0 and q[0] == float("inf")
        assert got[1, 3] == MOST[out] and got[3, 0] == MOST[out]
        got, q = run(g, p, F32, out, SILU)
        assert got[2].tolist() == [0, MOST[out], 0, 0]
    got, _ = run(g, p, F32, F32, SILU)
    assert got[2, 0] == 0 and got[2, 1] == 800 and got[2, 3] == 0 and got[0, 0] == float("inf")


@pytest.mark.parametrize("c", [64, 2000, 14336, 40000])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_rows_of_mixed_sizes(c, dt):
    # gates far below zero beside factors that make up for it, rows of tiny and of huge values,
    # rows whose largest value is one of those
    r = torch.Generator().manual_seed(c)
    g, p = 6 * torch.randn(12, c, generator=r), torch.randn(12, c, generator=r)
    g[1, ::7], p[1, ::7] = -30.0, 1e12
    g[2, c // 2], p[2, c // 2] = -70.0, 1e30
    g[3], p[3] = g[3] * 1e-10, p[3] * 1e-15
    g[4], p[4] = g[4] * 1e18, p[4] * 1e15
    g[5, 1:] = -60 - g[5, 1:].abs()
    g[6], p[6] = -100.0, 1e20
    g[7, 3], p[7, 3] = 1e15, 1e15
    g, p = g.to(DT[dt]), p.to(DT[dt])
    for out in (I8, E4M3):
        check(g, p, dt, out, SILU)


@pytest.mark.parametrize("dt", [BF16, F32])
def test_deep_gates(dt):
    # down to where SiLU itself leaves fp32, with factors that bring it back: SiLU is off by a few
    # roundings of its own or, below the normal numbers, by half the smallest of them and |g| times
    # half of it in exp(g) (two halves, the library's exponential being within one), all times |p|
    r = torch.Generator().manual_seed(dt)
    g = -70 - 40 * torch.rand(40, 333, generator=r)
    p = 1e30 * torch.randn(40, 333, generator=r)
    g, p = g.to(DT[dt]), p.to(DT[dt])
    got, _ = run(g, p, dt, dt, SILU)
    u = value(g, p, SILU)
    fi = torch.finfo(DT[dt])
    part = (10 + 2 * g.double().abs()) * U * u.abs() + (0.5 + g.double().abs()) * 2.0 ** -149 * p.double().abs()
    assert ((got - u).abs() <= part + (fi.eps / 2) * (u.abs() + part) + fi.smallest_normal * fi.eps).all()
    assert ((u == 0) == (got == 0))[g > -85].all()


def test_rows_of_more_than_one_launch():
    r = torch.Generator().manual_seed(11)
    rows = (1 << 20) + 77
    g, p = (torch.randn(rows, 8, generator=r).to(torch.bfloat16) for _ in range(2))
    for out in (I8, E4M3):
        check(g, p, BF16, out, NONE, (0, 4, 3))


@pytest.mark.parametrize("dt", [BF16, F32])
def test_borders(dt):
    # products of few values: many u*M/t lie at a border, or a rounding off it
    r = torch.Generator().manual_seed(4)
    g, p = (torch.randint(-256, 257, (1500, 700), generator=r).to(DT[dt]) for _ in range(2))
    for out in (I8, E4M3):
        check(g, p, dt, out, NONE)
        check(g, None, dt, out, RELU)


@pytest.mark.parametrize("out", [I8, E4M3])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("spread", ["normal", "wide", "deep"])
def test_many_values(dt, out, spread):
    # hundreds of millions of values: the few whose codes fp32 does not tell are among them
    r = torch.Generator(device=DEV).manual_seed(dt + out)
    rows, c = 4096, 14336
    for _ in range(3):
        size = torch.exp(0.5 * torch.randn(c, generator=r, device=DEV))
        g = torch.randn(rows, c, generator=r, device=DEV) * size
        if spread != "normal":  # gates down to where the exponential ends, factors that make up for it
            g = 90 * torch.rand(rows, c, generator=r, device=DEV) - 85
        p = torch.randn(rows, c, generator=r, device=DEV)
        if spread != "normal":
            p = p * torch.exp(torch.relu(-g)) * (30 if spread == "wide" else 3)  # 30: some are infinite
        g, p = g.to(DT[dt]), p.to(DT[dt])
        y, q = torch.empty(rows, c, dtype=DT[out], device=DEV), torch.empty(rows, device=DEV)
        say(f"gate of many values, dt={dt} out={out} {spread}")
        cvx.cvx_gate(cvx.make_gate_desc(rows, c, dt, out), g, p, y, q)
        for a in range(0, rows, 512):
            u = value(g[a:a + 512], p[a:a + 512], SILU)
            t = u.abs().amax(1)
            told = torch.isfinite(t)  # a row with an infinity has a NaN scale
            assert torch.equal(torch.isfinite(q[a:a + 512]), told) and (told.all() or spread == "wide")
            u, t, got, scale = u[told], t[told], y[a:a + 512][told], q[a:a + 512][told].double()
            v = u * (MOST[out] * (1.0 / t))[:, None]
            want = torch.round(v) if out == I8 else nearest_e4m3(v)
            assert torch.equal(got.double() if out == I8 else got.float().double(), want)
            assert ((scale - t / MOST[out]).abs() <= 2 * U * t / MOST[out]).all()


def test_far_rows_streams_and_graphs():
    # two rows 3 GB apart
    far, c = 3 << 29, 1000
    buf = torch.zeros(far + c, dtype=torch.float16, device=DEV)
    x = torch.as_strided(buf, (2, c), (far, 1))
    x.copy_(torch.randn(2, c, device=DEV))
    for out in (F16, I8):
        y, q = torch.empty(2, c, dtype=DT[out], device=DEV), torch.empty(2, device=DEV)
        say(f"gate of far rows, out={out}")
        cvx.cvx_gate(cvx.make_gate_desc(2, c, F16, out, SILU, far, far), x, x, y, q if out == I8 else None)
        want, _ = run(x.cpu(), x.cpu(), F16, out, SILU)
        assert torch.equal(y.cpu().double(), want)
    del buf, x
    g, p = (m.to(DEV) for m in rows_of(8, 200, 3000, BF16))
    y, q = torch.empty(200, 3000, dtype=torch.int8, device=DEV), torch.empty(200, device=DEV)
    d = cvx.make_gate_desc(200, 3000, BF16, I8)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        cvx.cvx_gate(d, g, p, y, q)
    for i in range(3):
        g.normal_()
        y.fill_(55)
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone(), q.clone()
        torch.cuda.current_stream().synchronize()
        stream.wait_stream(torch.cuda.current_stream())
        cvx.cvx_gate(d, g, p, y, q, stream)
        torch.cuda.synchronize()
        assert torch.equal(got[0], y) and torch.equal(got[1], q)
