"""8-bit integers: the codes cvx_rmsnorm writes and the projection cvx_linear makes of such
codes, against their definitions in 64 bits, element by element.

Tolerances.  A code is the integer nearest to u*(127*(1/t)), taken in 64 bits on both sides by
the same operations, so codes are equal.  y_scale is a 64-bit value rounded to fp32, 2^-24,
and the definition's own 64-bit roundings are far below that; 2^-23 is allowed.  Sums of
products of integers are exact; rounded to fp32 (2^-24), they take two scales, the bias,
a residual and an activation, whose slope is at most 1.1 and which is good to 8 units of
fp32: at most sixteen roundings of the magnitudes that meet there.  v is such a product
of integers held in 16 bits (exact) and 16-bit values, with `c_in` fp32 roundings at most,
and two 16-bit parts of 2^-16 of the token's largest between its two products (more than
64 tokens).  The output is rounded once, eps/2 or half the smallest subnormal."""
import pytest
import torch

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

from conv2d_batchnorm_activation_amd import cvx  # noqa: E402

F32, F16, BF16, I8 = cvx.CVX_DT_F32, cvx.CVX_DT_F16, cvx.CVX_DT_BF16, cvx.CVX_DT_I8
DT = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16}
U = 2.0 ** -24
NONE, RELU, SILU = cvx.CVX_ACT_NONE, cvx.CVX_ACT_RELU, cvx.CVX_ACT_SILU
EPS = 1e-5


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# ------------------------------------------------------------------ the norm
def codes_of(u, most=127.0):
    """(codes, the rows' largest magnitudes) of rows in 64 bits."""
    t = u.abs().amax(1)
    return torch.round(u * torch.where(t > 0, most * (1.0 / t), 0.0)[:, None]), t


def norm_of(x, r, g):
    """codes, scales and sums of rows on the CPU."""
    if r is None:
        h = x.double()
    else:
        h = x.double() + r.double() if x.dtype == torch.float32 else (x.float() + r.float()).double()
    q = 1.0 / torch.sqrt((h * h).mean(1) + EPS)
    codes, t = codes_of(h * g.double())
    return codes, t * q / 127.0, h


@pytest.mark.parametrize("rows,c,dt,res,pad", [
    (1, 1, BF16, False, 0), (1, 4096, BF16, True, 0), (3, 7, F16, True, 1), (5, 513, F32, True, 3), (2, 64, F32, False, 0),
    (300, 1337, BF16, True, 5), (33, 2048, F16, False, 8), (600, 4104, BF16, True, 0), (7, 20480, F32, True, 0),
    (2, 33000, BF16, True, 6), (2, 50003, F16, False, 0), (1100, 96, F32, True, 0)])
def test_norm(rows, c, dt, res, pad):
    g = torch.Generator().manual_seed(rows * 7 + c)
    big = lambda s: (s * torch.randn(rows, c + pad, generator=g)).to(DT[dt])  # noqa: E731
    x, r = big(1.0), big(3.0) if res else None
    gamma = 1 + 0.2 * torch.randn(c, generator=g)
    x[-1] = 0  # a row of zeros, or of the residual alone
    xd, rd = x.to(DEV)[:, :c], r.to(DEV)[:, :c] if res else None
    y = torch.full((rows, c + pad), 99, dtype=torch.int8, device=DEV)
    s = torch.empty(rows, c, dtype=DT[dt], device=DEV)
    q = torch.full((rows + 2,), float("nan"), device=DEV)
    d = cvx.make_rmsnorm_desc(rows, c, dt, I8, EPS, xd.stride(0), rd.stride(0) if res else 0, 0, c + pad)
    say(f"norm to integers: {rows}x{c} dt={dt} res={res} pad={pad}")
    cvx.cvx_rmsnorm(d, xd, rd, gamma.to(DEV), s, y[:, :c], q[1:rows + 1])
    torch.cuda.synchronize()
    codes, scale, h = norm_of(x[:, :c], r[:, :c] if res else None, gamma)
    assert torch.equal(y[:, :c].cpu().double(), codes)
    assert (y[:, c:] == 99).all() and torch.isnan(q[0]) and torch.isnan(q[-1])
    assert ((q[1:-1].cpu().double() - scale).abs() <= 2 * U * scale).all()
    assert torch.equal(s.cpu(), h.to(DT[dt]))


@pytest.mark.parametrize("c,dt", [(8193, BF16), (10240, F16), (10241, BF16), (16384, BF16), (16391, F16), (20480, BF16),
                                  (20481, BF16), (4097, F32), (5120, F32), (5123, F32), (8192, F32), (8193, F32)])
def test_norm_many_long_rows(c, dt):
    # widths to where a row's threads, or the vectors each holds, change
    test_norm(517, c, dt, c % 2 == 0, 3 * (c % 4))


def test_norm_ties_and_limits():
    # half of the largest is 63.5 exactly: the even one of its neighbours
    x = torch.tensor([[2.0, 1.0, -1.0, -2.0, 0.0, 3 * 2.0 / 127, 2.0 / 127, 2.5]])
    x[0, 7] = 2.0
    y = torch.empty(1, 8, dtype=torch.int8, device=DEV)
    q = torch.empty(1, device=DEV)
    say("norm to integers: ties")
    cvx.cvx_rmsnorm(cvx.make_rmsnorm_desc(1, 8, F32, I8, EPS), x.to(DEV), None, torch.ones(8, device=DEV), None, y, q)
    assert y.cpu().tolist()[0] == [127, 64, -64, -127, 0, 3, 1, 127]


@pytest.mark.parametrize("dt", [BF16, F32])
def test_norm_borders(dt):
    # multiples of few values: many u*127/t lie at a border, or a rounding off it
    g = torch.Generator().manual_seed(3)
    x = torch.randint(-256, 257, (2000, 700), generator=g).to(DT[dt])
    y = torch.empty(2000, 700, dtype=torch.int8, device=DEV)
    q = torch.empty(2000, device=DEV)
    say("norm to integers: borders")
    cvx.cvx_rmsnorm(cvx.make_rmsnorm_desc(2000, 700, dt, I8, EPS), x.to(DEV), None, torch.ones(700, device=DEV), None, y, q)
    assert torch.equal(y.cpu().double(), norm_of(x, None, torch.ones(700))[0])


def test_norm_bad_rows():
    nan, inf = float("nan"), float("inf")
    x = torch.ones(5, 40)
    x[1, 3], x[2, 39], x[3, 0] = nan, inf, -inf
    x[4] = torch.finfo(torch.float32).max
    x = x.to(DEV)
    y = torch.empty(5, 40, dtype=torch.int8, device=DEV)
    q = torch.empty(5, device=DEV)
    say("norm to integers: NaN and infinities")
    cvx.cvx_rmsnorm(cvx.make_rmsnorm_desc(5, 40, F32, I8, EPS), x, None, torch.ones(40, device=DEV), None, y, q)
    assert torch.isnan(q).tolist() == [False, True, True, True, False]
    assert (y[[0, 4]] == 127).all()


# ------------------------------------------------------------ the projection
class Case:
    """Operands on the CPU, seeded; `run` puts them on the GPU, strided, and calls the library."""

    def __init__(self, seed, t, ci, co, dt=BF16, rank=0, n=0, act=NONE, res=0, pads=(0, 0, 0), scale=True, bias=True,
                 least=-127):
        g = torch.Generator().manual_seed(seed)
        self.t, self.ci, self.co, self.dt, self.rank, self.n, self.act, self.res_mode = t, ci, co, dt, rank, n, act, res
        self.pads = pads
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.x = (rnd(t, ci) * 40).round().clamp(least, 127).to(torch.int8)
        self.w = (rnd(co, ci) * 40).round().clamp(least, 127).to(torch.int8)
        self.sx = (0.5 + torch.rand(t, generator=g)) / 40
        self.scale = (1 + 0.3 * rnd(co)) / 40 / ci ** 0.5 if scale else None
        self.bias = rnd(co) if bias else None
        self.res = rnd(t, co).to(DT[dt]) if res else None
        self.a = self.b = self.alpha = self.ids = None
        if rank:
            self.a, self.b = (rnd(n, rank, ci) / ci ** 0.5).to(DT[dt]), (rnd(n, co, rank) / rank ** 0.5).to(DT[dt])
            self.alpha = 0.5 + torch.rand(n, generator=g)
            self.ids = torch.randint(-1, n + 1, (t,), generator=g).to(torch.int32)

    def desc(self):
        px, pr, py = self.pads
        return cvx.make_linear_desc(self.t, self.ci, self.co, self.dt, I8, self.act, self.res_mode, self.rank, self.n,
                                    self.ci + px, self.co + pr if self.res is not None else 0, self.co + py)

    def run(self):
        px, pr, py = self.pads

        def rows(m, pad, fill):
            buf = torch.full((m.shape[0], m.shape[1] + pad), fill, dtype=m.dtype, device=DEV)
            buf[:, :m.shape[1]] = m.to(DEV)
            return buf[:, :m.shape[1]]

        dev = lambda m: None if m is None else m.to(DEV)  # noqa: E731
        d = self.desc()
        ybuf = torch.full((self.t + 2, self.co + py), float("nan"), dtype=DT[self.dt], device=DEV)
        ws = torch.full((cvx.cvx_linear_workspace_bytes(d) + 64,), 255, dtype=torch.uint8, device=DEV)
        say(f"{cvx.cvx_linear_plan(d)} t={self.t} ci={self.ci} co={self.co} act={self.act} res={self.res_mode} {self.pads}")
        cvx.cvx_linear(d, rows(self.x, px, 77), dev(self.w), ybuf[1:-1, :self.co], dev(self.sx), dev(self.scale),
                       dev(self.bias), None if self.res is None else rows(self.res, pr, float("nan")), dev(self.a),
                       dev(self.b), dev(self.alpha), dev(self.ids), ws, ws.numel() - 64)
        torch.cuda.synchronize()
        assert torch.isnan(ybuf[[0, -1]].float()).all() and torch.isnan(ybuf[:, self.co:].float()).all()
        assert (ws[-64:] == 255).all()
        return ybuf[1:-1, :self.co].cpu().double()

    def definition(self):
        """(value, tolerance)"""
        f = torch.float64
        x, w = self.x.to(f), self.w.to(f)
        s = (x @ w.t()) * self.sx.to(f)[:, None]
        if self.scale is not None:
            s = s * self.scale.to(f)
        z, mag, err = s.clone(), s.abs(), torch.zeros_like(s)
        if self.bias is not None:
            z, mag = z + self.bias.to(f), mag + self.bias.to(f).abs()
        for d in range(self.n):
            at = (self.ids == d).nonzero()[:, 0]
            if not at.numel():
                continue
            al, a, b = self.alpha[d].to(f), self.a[d].to(f), self.b[d].to(f)
            xs = x[at] * self.sx.to(f)[at][:, None]
            v, vm = al * (xs @ a.t()), al * (xs.abs() @ a.abs().t())
            z[at] += v @ b.t()
            mag[at] += v.abs() @ b.abs().t()
            big = v.abs().amax(1, keepdim=True).expand_as(v)
            err[at] += ((self.ci + 8) * U * vm + 2.0 ** -16 * big) @ b.abs().t() + 2 * self.rank * U * mag[at]
        if self.res is not None:
            mag = mag + self.res.to(f).abs()
        if self.res_mode == 1:
            z = z + self.res.to(f)
        z = z * torch.sigmoid(z) if self.act == SILU else torch.relu(z) if self.act == RELU else z
        if self.res_mode == 2:
            z = z + self.res.to(f)
        fi = torch.finfo(DT[self.dt])
        tol = 1.1 * (err + 16 * U * mag)
        return z, tol + (fi.eps / 2) * (z.abs() + tol) + fi.smallest_normal * fi.eps / 2


def check(c):
    got = c.run()
    want, tol = c.definition()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} out of bound, first at {bad.nonzero()[0].tolist()}: " \
                          f"{got[bad][0].item()!r} for {want[bad][0].item()!r}"


@pytest.mark.parametrize("t,ci,co,kw", [
    (1, 16, 4, {}), (1, 4096, 256, dict(act=SILU)), (2, 144, 36, dict(dt=F16, res=1)), (8, 1008, 68, dict(res=2)),
    (9, 272, 100, dict(act=RELU, pads=(16, 4, 8))), (17, 128, 132, dict(dt=F16)), (33, 2064, 64, dict(res=2, act=SILU)),
    (64, 112, 4100, {}), (64, 256, 48, dict(scale=False, bias=False, dt=F16)), (65, 64, 64, {}),
    (129, 4096, 260, dict(res=1, act=RELU)), (200, 1040, 516, dict(pads=(32, 12, 4))), (333, 1008, 1284, dict(dt=F16, act=SILU)),
    (700, 80, 2052, dict(res=2)), (1500, 144, 3000, dict(dt=F16, res=2, act=SILU, pads=(16, 0, 4)))])
def test_projection(t, ci, co, kw):
    check(Case(t * 31 + ci, t, ci, co, **kw))


@pytest.mark.parametrize("t,ci,co,rank,n,kw", [
    (1, 512, 64, 8, 3, {}), (5, 1040, 36, 16, 4, dict(dt=F16)), (40, 272, 132, 24, 6, dict(res=2)), (64, 64, 4100, 128, 2, {}),
    (100, 528, 260, 8, 5, dict(act=SILU)), (333, 1008, 1284, 8, 5, dict(dt=F16, act=SILU)), (300, 1040, 68, 64, 4, dict(res=1)),
    (2100, 96, 516, 40, 3, dict(dt=F16)), (2100, 144, 2052, 16, 3, {})])
def test_projection_with_adapters(t, ci, co, rank, n, kw):
    check(Case(t * 17 + rank, t, ci, co, rank=rank, n=n, **kw))


@pytest.mark.parametrize("t", [1, 8, 9, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("ci,co", [(2064, 4100), (1040, 8192), (528, 8196), (2064, 8200)])
def test_few_tokens_of_wide_layers(t, ci, co):
    # where the rules of few tokens change
    check(Case(t + co, t, ci, co, res=2 if t % 2 else 0))
    check(Case(t + co, t, ci, co, F16, rank=16, n=4, act=SILU))


@pytest.mark.parametrize("t,ci,co,few", [(65, 256, 2048, True), (128, 272, 2048, True), (129, 272, 2052, False),
                                         (1000, 64, 256, True), (1025, 64, 256, False), (256, 2064, 1024, True)])
def test_many_tokens_of_narrow_layers(t, ci, co, few):
    c = Case(t + co, t, ci, co, res=1, pads=(16, 4, 8))
    assert (cvx.cvx_linear_plan(c.desc()).split()[1] == "few") == few
    check(c)
    check(Case(t + co, t, ci, co, F16, rank=8, n=4, act=RELU))


@pytest.mark.parametrize("t,co,bn", [(2000, 8192, 256), (1500, 2560, 128), (300, 1028, 64)])
def test_every_tile(t, co, bn):
    ci = 1040
    for kw in (dict(), dict(rank=16, n=3, dt=F16)):
        c = Case(t, t, ci, co, **kw)
        plan = cvx.cvx_linear_plan(c.desc())
        assert plan.split()[1] == "tile" and plan.split()[2].endswith(f"x{bn}"), plan
        check(c)


@pytest.mark.parametrize("t", [1, 12, 100, 900])
def test_sums_are_exact(t):
    # the largest magnitudes there are, over a long row: 2^14 * 65536 = 2^30, and one off it
    ci, co = 65536, 68
    c = Case(3, t, ci, co, least=-128, scale=False, bias=False, dt=BF16)
    c.x.fill_(-128)
    c.w.fill_(-128)
    c.w[1::2] = 127
    c.x[::2, :16] = 127
    c.sx.fill_(2.0 ** -30)
    check(c)
    c.w.random_(-128, 128, generator=torch.Generator().manual_seed(5))
    check(c)


@pytest.mark.parametrize("t", [3, 100])
def test_bad_scales_and_adapters_stay_with_their_tokens(t):
    nan, inf = float("nan"), float("inf")
    c = Case(9, t, 256, 128, rank=8, n=3)
    c.ids.fill_(0)
    c.ids[1] = 1
    c.a[1, 0, 0] = nan
    c.sx[2] = inf
    got = c.run()
    assert torch.isnan(got[1]).all()
    assert not torch.isfinite(got[2]).any()
    rest = [i for i in range(t) if i not in (1, 2)]
    assert torch.isfinite(got[rest]).all()


@pytest.mark.parametrize("t", [1, 50, 400])
def test_norm_and_projection_as_a_layer_uses_them(t):
    c = Case(60 + t, t, 1040, 516, act=SILU)
    g = torch.Generator().manual_seed(t)
    x = torch.randn(t, c.ci, generator=g).to(torch.bfloat16)
    gamma = 1 + 0.1 * torch.randn(c.ci, generator=g)
    y, q = torch.empty(t, c.ci, dtype=torch.int8, device=DEV), torch.empty(t, device=DEV)
    out = torch.empty(t, c.co, dtype=torch.bfloat16, device=DEV)
    say(f"norm and projection in integers, {t} tokens")
    d = [cvx.make_rmsnorm_desc(t, c.ci, BF16, I8, EPS), cvx.make_linear_desc(t, c.ci, c.co, BF16, I8, SILU)]
    w, scale, bias, xd, gd = (m.to(DEV) for m in (c.w, c.scale, c.bias, x, gamma))

    def layer():
        cvx.cvx_rmsnorm(d[0], xd, None, gd, None, y, q)
        cvx.cvx_linear(d[1], y, w, out, q, scale, bias)

    layer()
    torch.cuda.synchronize()
    c.x, c.sx = y.cpu(), q.cpu()
    want, tol = c.definition()
    assert ((out.cpu().double() - want).abs() <= tol).all()
    # captured, replayed over other inputs, with eager work between the replays
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        layer()
    for i in range(3):
        xd.copy_(torch.randn(t, c.ci, generator=g).to(torch.bfloat16))
        for m in (y, q, out):
            m.view(torch.uint8).fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        got = [m.clone() for m in (y, q, out)]
        layer()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (y, q, out)))
