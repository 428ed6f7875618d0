"""cvx_linear against its definition in 64 bits, element by element.

Tolerance.  Products of two 16-bit or two e4m3 values are exact in fp32, so a sum
of K of them, in whatever order, is off by at most K*2^-24 of the sum of their
magnitudes.  v carries that error through |lora_b|, and is taken as two 16-bit
values whose sum is within 2^-16 of the token's largest |v|; the second
product's `rank` terms are added to the first sum, at most 2^-24 of the running
magnitude each.  Scales, bias, residual and the activation (whose slope is at
most 1.1, and which is good to 8 units of fp32) take a dozen roundings of the magnitudes that meet there.
The output is rounded once, eps/2, or half the smallest subnormal."""
import pytest
import torch

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

from conv2d_batchnorm_activation_amd import cvx  # noqa: E402

F16, BF16, E4M3 = cvx.CVX_DT_F16, cvx.CVX_DT_BF16, cvx.CVX_DT_E4M3
DT = {F16: torch.float16, BF16: torch.bfloat16, E4M3: torch.float8_e4m3fn}
U = 2.0 ** -24
NONE, RELU, SILU = cvx.CVX_ACT_NONE, cvx.CVX_ACT_RELU, cvx.CVX_ACT_SILU


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Case:
    """Operands on the CPU, seeded; `run` puts them on the GPU, strided, and calls the library."""

    def __init__(self, seed, tokens, ci, co, dt=BF16, x8=False, rank=0, n=0, act=NONE, res=0, ids="each", scale=True,
                 bias=True, alpha=True, pads=(0, 0, 0)):
        g = torch.Generator().manual_seed(seed)
        self.t, self.ci, self.co, self.dt, self.x8, self.rank, self.n = tokens, ci, co, dt, x8, rank, n
        self.act, self.res_mode, self.pads = act, res, pads
        tdt = DT[dt]

        def rnd(*shape):
            return torch.randn(*shape, generator=g)

        self.x, self.w = rnd(tokens, ci), rnd(co, ci) / ci ** 0.5
        self.sx = None
        self.scale = 1 + 0.3 * rnd(co) if scale else None
        self.bias = rnd(co) if bias else None
        if x8:
            self.sx = 0.01 + 0.02 * torch.rand(tokens, generator=g)
            self.x = (self.x * 100).clamp(-448, 448).to(DT[E4M3])
            self.w = (self.w * 40).clamp(-448, 448).to(DT[E4M3])
            self.scale = (self.scale if scale else torch.ones(co)) / 40
        else:
            self.x, self.w = self.x.to(tdt), self.w.to(tdt)
        self.res = rnd(tokens, co).to(tdt) if res else None
        self.a = self.b = self.alpha = self.ids = None
        if rank:
            self.a, self.b = (rnd(n, rank, ci) / ci ** 0.5).to(tdt), (rnd(n, co, rank) / rank ** 0.5).to(tdt)
            self.alpha = 0.5 + torch.rand(n, generator=g) if alpha else None
            if ids == "each":
                self.ids = torch.randint(-1, n, (tokens,), generator=g)
            elif ids == "runs":  # requests of several tokens
                k = torch.randint(-1, n, (tokens,), generator=g)
                self.ids = k[torch.sort(torch.randint(0, tokens, (tokens,), generator=g) // 9 * 9)[0]]
            elif ids == "one":
                self.ids = torch.full((tokens,), n - 1)
            else:  # none of the tokens has one; numbers outside mean that too
                self.ids = torch.tensor([-1, n, n + 1, 2 ** 31 - 1, -2 ** 31])[torch.randint(0, 5, (tokens,), generator=g)]
            self.ids = self.ids.to(torch.int32)

    def describe(self):
        return cvx.cvx_linear_plan(cvx.make_linear_desc(self.t, self.ci, self.co, self.dt, E4M3 if self.x8 else self.dt,
                                                        rank=self.rank, n_adapters=self.n))

    def run(self, stream=None):
        px, pr, py = self.pads

        def rows(m, pad, fill=float("nan")):
            buf = torch.full((m.shape[0], m.shape[1] + pad), fill).to(m.dtype).to(DEV)
            buf[:, :m.shape[1]] = m.to(DEV)
            return buf[:, :m.shape[1]]

        def dev(m):
            return None if m is None else m.to(DEV)

        ys = self.co + py
        head = 64
        ybuf = torch.full((head + self.t * ys + head,), float("nan"), dtype=DT[self.dt], device=DEV)
        y = ybuf[head:head + self.t * ys].view(self.t, ys)[:, :self.co]
        d = cvx.make_linear_desc(self.t, self.ci, self.co, self.dt, E4M3 if self.x8 else self.dt, self.act,
                                 self.res_mode, self.rank, self.n, x_stride=self.ci + px,
                                 res_stride=self.co + pr if self.res is not None else 0, y_stride=ys)
        need = cvx.cvx_linear_workspace_bytes(d)
        ws = torch.full((need + 64,), 255, dtype=torch.uint8, device=DEV)  # NaN in every word
        self.plan = cvx.cvx_linear_plan(d)
        say(f"{self.plan} t={self.t} ci={self.ci} co={self.co} n={self.n} act={self.act} res={self.res_mode} {self.pads}")
        cvx.cvx_linear(d, rows(self.x, px), dev(self.w), y, dev(self.sx), dev(self.scale), dev(self.bias),
                       None if self.res is None else rows(self.res, pr), dev(self.a), dev(self.b), dev(self.alpha),
                       dev(self.ids), ws, need, stream)
        torch.cuda.synchronize()
        b = ybuf.float().cpu()
        assert torch.isnan(b[:head]).all() and torch.isnan(b[-head:]).all()
        assert torch.isnan(b[head:-head].view(self.t, ys)[:, self.co:]).all(), "wrote between rows"
        assert (ws[need:] == 255).all(), "wrote past the workspace"
        return y.cpu().double()

    def definition(self):
        """(value, tolerance)"""
        f = torch.float64
        x, w = self.x.to(f), self.w.to(f)
        if self.x8:
            x = x * self.sx.to(f)[:, None]
        if self.scale is not None:
            w = w * self.scale.to(f)[:, None]
        z, mag = x @ w.t(), x.abs() @ w.abs().t()
        err = self.ci * U * mag
        if self.x8 and "tile" in self.describe():
            gx, gw = x.abs().view(self.t, -1, 8).amax(2), w.abs().view(self.co, -1, 8).amax(2)
            err = err + 7 * 2.0 ** -13 * (gx @ gw.t())
        if self.bias is not None:
            z = z + self.bias.to(f)
            mag = mag + self.bias.to(f).abs()
        if self.rank:
            for d in set(self.ids.tolist()):
                if not 0 <= d < self.n:
                    continue
                at = (self.ids == d).nonzero()[:, 0]
                al = self.alpha[d].to(f) if self.alpha is not None else 1.0
                a, b = self.a[d].to(f), self.b[d].to(f)
                v, vm = al * (x[at] @ a.t()), al * (x[at].abs() @ a.abs().t())
                z[at] += v @ b.t()
                dm = v.abs() @ b.abs().t()
                mag[at] += dm
                err[at] += (self.ci + 8) * U * (vm @ b.abs().t())
                err[at] += 2.0 ** -16 * v.abs().amax(1, keepdim=True) * b.abs().sum(1)[None, :]
            err = err + self.rank * U * mag
        if self.res is not None:
            mag = mag + self.res.to(f).abs()
        r = self.res.to(f) if self.res is not None else 0.0
        if self.res_mode == cvx.CVX_RES_BEFORE_ACT:
            z = z + r
        if self.act == RELU:
            z = z.clamp_min(0)
        elif self.act == SILU:
            z = z * torch.sigmoid(z)
        if self.res_mode == cvx.CVX_RES_AFTER_ACT:
            z = z + r
        err = 1.1 * (err + 20 * U * mag)
        info = torch.finfo(DT[self.dt])
        return z, err + info.eps / 2 * (z.abs() + err) + info.smallest_normal * info.eps

    def check(self):
        got = self.run()
        want, tol = self.definition()
        bad = ~((got - want).abs() <= tol)
        assert not bad.any(), f"{self.plan}: {int(bad.sum())} of {bad.numel()} out of bound, first at " \
                              f"{bad.nonzero()[0].tolist()}: {got[bad][0].item()!r} for {want[bad][0].item()!r}"
        return got


SHAPES = [
    # tokens, c_in, c_out
    (1, 16, 4), (1, 512, 64), (2, 48, 20), (15, 1040, 36), (16, 2064, 16), (17, 80, 300), (31, 4112, 24), (33, 160, 132),
    (64, 1024, 260), (65, 16, 4), (65, 64, 128), (97, 208, 36), (128, 144, 132), (129, 1040, 260), (200, 64, 516),
    (257, 336, 100), (300, 2064, 384), (129, 2064, 1364),
]


@pytest.mark.parametrize("x8", [False, True], ids=["x16", "x8"])
@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=["x".join(map(str, s)) for s in SHAPES])
def test_linear_plain(shape, dt, x8):
    t, ci, co = shape
    Case(t * 7 + ci, t, ci, co, dt, x8).check()


@pytest.mark.parametrize("x8", [False, True], ids=["x16", "x8"])
@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=["x".join(map(str, s)) for s in SHAPES])
def test_linear_adapters(shape, dt, x8):
    t, ci, co = shape
    rank = (8, 16, 24, 64, 128)[(t + ci + co) % 5]
    Case(t * 11 + co, t, ci, co, dt, x8, rank, 1 + t % 13, ids="each").check()


@pytest.mark.parametrize("x8", [False, True], ids=["x16", "x8"])
@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("t,ci,co", [(1, 4096, 12292), (16, 64, 8200), (31, 176, 5000), (33, 80, 4100), (64, 528, 5012)])
def test_linear_many_channels(t, ci, co, dt, x8):
    # more than a workgroup a compute unit
    Case(t + co, t, ci, co, dt, x8, 16, 9, SILU, 2).check()
    Case(t + ci, t, ci, co, dt, x8).check()


@pytest.mark.parametrize("ids", ["runs", "one", "none"])
@pytest.mark.parametrize("t", [1, 16, 50, 150, 333])
def test_linear_adapter_ids(t, ids):
    Case(t, t, 272, 140, (F16, BF16)[t % 2], False, 16, 6, ids=ids, alpha=ids != "one").check()


@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("rank", [8, 16, 24])
@pytest.mark.parametrize("ci,co", [(8, 4), (1000, 60), (4096, 132)])
def test_linear_one_token(ci, co, rank, dt):
    for ids in ("one", "none"):
        Case(ci + rank, 1, ci, co, dt, False, rank, 3, SILU, 2, ids=ids).check()
    Case(ci, 1, ci, co, dt, False, rank, 1, ids="one", alpha=False, scale=False, bias=False).check()


@pytest.mark.parametrize("x8", [False, True], ids=["x16", "x8"])
@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("rank", [8, 24, 64, 72, 128])
def test_linear_adapters_of_prompts(rank, dt, x8):
    # runs of requests in blocks of 64 tokens, slices of c_in, ranks that fill part of a block
    Case(rank, 2070, 1168, 68, dt, x8, rank, 7, ids="runs").check()


@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("co", [68, 2052])
@pytest.mark.parametrize("ci,rank", [(1040, 8), (8192, 16), (8208, 16), (2064, 24)])
def test_linear_adapters_in_slices(ci, rank, co, dt):
    # the first product in few slices, joined by the tiles, and in many or of more ranks, joined before
    Case(ci, 100, ci, co, dt, False, rank, 40).check()


@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("t,ci,co,rank", [(65, 2048, 2048, 0), (129, 2056, 1348, 16), (190, 4104, 132, 64),
                                          (500, 2064, 508, 32), (2100, 2200, 20, 8), (70, 8200, 36, 128)])
def test_linear_blocks_of_few_tokens(t, ci, co, rank, dt):
    # few tiles of a long row: the kernel for few tokens takes them 64 at a time
    c = Case(t, t, ci, co, dt, False, rank, 9 if rank else 0, SILU, 2, pads=(24, 8, 12))
    assert "linear few 16x64" in c.describe()
    c.check()
    Case(t + 1, t, ci, co, dt, False, rank, 3 if rank else 0, ids="runs").check()


@pytest.mark.parametrize("t", [3, 40, 140])
@pytest.mark.parametrize("act", [NONE, RELU, SILU])
@pytest.mark.parametrize("res", [0, 1, 2])
def test_linear_epilogue(t, act, res):
    Case(t + act, t, 128, 68, BF16 if res else F16, t == 40, 8, 3, act, res, scale=act != RELU, bias=res != 2).check()


@pytest.mark.parametrize("t", [5, 100])
def test_linear_without_scale_and_bias(t):
    Case(t, t, 96, 64, scale=False, bias=False).check()
    Case(t, t, 96, 64, x8=True, scale=False, bias=False, rank=8, n=2, alpha=False).check()


@pytest.mark.parametrize("x8", [False, True], ids=["x16", "x8"])
@pytest.mark.parametrize("t", [7, 64, 135])
def test_linear_slices_of_wider_tensors(t, x8):
    Case(t, t, 176, 88, F16, x8, 24, 4, SILU, 2, pads=(48, 12, 20)).check()


@pytest.mark.parametrize("x8", [False, True], ids=["x16", "x8"])
@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("shape", [(4100, 48, 4092), (4097, 272, 3588)], ids=["4100x48", "4097x272"])
def test_linear_large_tiles(shape, dt, x8):
    t, ci, co = shape
    c = Case(t, t, ci, co, dt, x8, 16, 5, SILU, 1, ids="runs")
    c.check()
    Case(t + 1, t, ci, co, dt, x8, 0, 0).check()


@pytest.mark.parametrize("x8", [False, True], ids=["x16", "x8"])
@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("t,ci,co", [(1000, 80, 4092), (1021, 400, 3972)])
def test_linear_middle_tiles(t, ci, co, dt, x8):
    c = Case(t, t, ci, co, dt, x8, 24, 5, SILU, 1)
    assert "tile 128x128" in c.describe()
    c.check()
    Case(t + 2, t, ci, co, dt, x8, 8, 7, ids="runs").check()
    Case(t + 1, t, ci, co, dt, x8, 0, 0).check()


@pytest.mark.parametrize("t", [20, 60, 200])
def test_linear_values_of_other_adapters_stay_out(t):
    c = Case(t, t, 144, 100, BF16, False, 16, 5)
    want, tol = c.definition()
    c.a[2, 3, 5] = float("nan")
    c.b[2, 7, 1] = float("inf")
    c.a[4, 0, 0] = float("-inf")
    c.b[4] = float("nan")
    x2 = c.ids == 1
    c.x[x2.nonzero()[0, 0], 9] = float("nan")
    hit = (c.ids == 2) | (c.ids == 4)
    hit[x2.nonzero()[0, 0]] = True
    got = c.run()
    fine = ~hit
    assert ((got - want).abs() <= tol)[fine].all()
    assert not torch.isfinite(got[hit]).all(1).any()


@pytest.mark.parametrize("t", [20, 100])
def test_linear_low_rank_values_beyond_16_bits(t):
    # v leaves fp16's range, the output does not
    c = Case(t, t, 128, 64, F16, False, 8, 3, ids="one")
    c.a *= 3000
    c.b /= 3000
    c.x *= 100
    c.w /= 100
    assert c.definition()[0].abs().max() < 60000 and (c.x.double() @ c.a[2].double().t()).abs().max() > 70000
    c.check()


@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("t", [20, 100])
def test_linear_sums_beside_huge_low_rank_values(t, dt):
    # channels whose rows of B are zero keep their sums, however large v is
    c = Case(t, t, 128, 64, dt, False, 8, 3, ids="one")
    c.alpha[:] = 1e37
    c.b[:, :40] = 0
    got = c.run()[:, :40]
    want, tol = c.definition()
    assert ((got - want[:, :40]).abs() <= tol[:, :40]).all()


def test_linear_is_the_same_every_time():
    for t in (30, 150):
        c = Case(t, t, 1040, 132, BF16, False, 16, 7)
        first = c.run()
        for _ in range(3):
            assert torch.equal(c.run(), first)
