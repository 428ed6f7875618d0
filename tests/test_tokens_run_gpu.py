"""The operators on tokens together, as a layer uses them: norm to e4m3 -> projection
of the codes with adapters -> norm with the residual's addition -> projection with
the residual.  Every step is held to its 64-bit definition on the values the step
before it left; captured into a graph, on other streams and on tensors whose
offsets pass 32 bits, the results are the same."""
import pytest
import torch

from gpu_util import DEV, say
from test_linear_gpu import BF16, E4M3, SILU, Case
from test_rmsnorm_gpu import EPS, compare

pytestmark = pytest.mark.gpu

from conv2d_batchnorm_activation_amd import cvx  # noqa: E402


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Layer:
    """Weights, adapters and buffers of a small layer for `t` tokens of `c` channels."""

    def __init__(self, t, c=272, inner=320, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.t, self.c, self.inner = t, c, inner
        self.one = Case(seed + 1, t, c, inner, BF16, True, 16, 5, SILU)
        self.two = Case(seed + 2, t, inner, c, BF16, False, 8, 5, res=2)
        self.two.ids = self.one.ids
        self.gamma = [1 + 0.2 * torch.randn(n, generator=g) for n in (c, inner)]
        self.x0 = torch.randn(t, c, generator=g).to(torch.bfloat16)
        self.r0 = torch.randn(t, inner, generator=g).to(torch.bfloat16)

        def dev(m):
            return None if m is None else m.to(DEV)

        self.x, self.r, self.g = dev(self.x0), dev(self.r0), [dev(m) for m in self.gamma]
        self.p = [{k: dev(getattr(k_, k)) for k in ("w", "scale", "bias", "a", "b", "alpha", "ids")}
                  for k_ in (self.one, self.two)]
        self.codes = torch.empty(t, c, dtype=torch.float8_e4m3fn, device=DEV)
        self.scales = torch.empty(t, device=DEV)
        self.y1 = torch.empty(t, inner, dtype=torch.bfloat16, device=DEV)
        self.sum, self.n2 = torch.empty_like(self.y1), torch.empty_like(self.y1)
        self.out = torch.empty_like(self.x)
        self.d = [cvx.make_rmsnorm_desc(t, c, BF16, E4M3, EPS),
                  cvx.make_linear_desc(t, c, inner, BF16, E4M3, SILU, 0, 16, 5),
                  cvx.make_rmsnorm_desc(t, inner, BF16, eps=EPS),
                  cvx.make_linear_desc(t, inner, c, BF16, res_mode=2, rank=8, n_adapters=5)]
        self.ws = torch.empty(max(cvx.cvx_linear_workspace_bytes(self.d[i]) for i in (1, 3)) + 16, dtype=torch.uint8,
                              device=DEV)

    def run(self, stream=None):
        a, b = self.p
        cvx.cvx_rmsnorm(self.d[0], self.x, None, self.g[0], None, self.codes, self.scales, stream)
        cvx.cvx_linear(self.d[1], self.codes, a["w"], self.y1, self.scales, a["scale"], a["bias"], None, a["a"], a["b"],
                       a["alpha"], a["ids"], self.ws, stream=stream)
        cvx.cvx_rmsnorm(self.d[2], self.y1, self.r, self.g[1], self.sum, self.n2, None, stream)
        cvx.cvx_linear(self.d[3], self.n2, b["w"], self.out, None, b["scale"], b["bias"], self.x, b["a"], b["b"],
                       b["alpha"], b["ids"], self.ws, stream=stream)

    def results(self):
        return [m.clone() for m in (self.codes, self.scales, self.y1, self.sum, self.n2, self.out)]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("t", [1, 13, 64, 131, 700])
def test_layer(t):
    L = Layer(t)
    say(f"layer of {t} tokens")
    L.run()
    torch.cuda.synchronize()
    codes, scales, y1, s, n2, out = (m.cpu() for m in L.results())
    compare(L.x0, None, L.gamma[0], BF16, True, (None, codes.float().double(), scales.double()), "first norm")
    L.one.x, L.one.sx = codes, scales
    want, tol = L.one.definition()
    assert ((y1.double() - want).abs() <= tol).all()
    compare(y1, L.r0, L.gamma[1], BF16, False, (s.double(), n2.double(), None), "second norm")
    L.two.x, L.two.res = n2, L.x0
    want, tol = L.two.definition()
    assert ((out.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("t", [1, 20, 200])
def test_layer_in_a_graph(t):
    L = Layer(t, seed=40)
    L.run()
    first = L.results()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    say(f"graph of a layer of {t} tokens")
    with torch.cuda.graph(graph, stream=stream):
        L.run()
    other = torch.randn(t, L.c, device=DEV).to(torch.bfloat16)
    keep = L.x.clone()
    for i in range(4):
        L.x.copy_(other if i % 2 else keep)
        for m in (L.codes, L.y1, L.n2, L.out, L.ws):
            m.view(torch.uint8).fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        got = L.results()
        L.run()  # eager work between the replays
        torch.cuda.synchronize()
        assert same(got, L.results())
        assert same(got, first) == (i % 2 == 0)


def test_layers_on_two_streams():
    layers = [Layer(t, seed=60 + t) for t in (30, 150, 700)]
    want = []
    for L in layers:
        L.run()
        torch.cuda.synchronize()
        want.append(L.results())
    streams = [torch.cuda.Stream() for _ in layers]
    say("layers on streams of their own")
    for _ in range(5):
        for L, s in zip(layers, streams):
            L.run(stream=s)
    torch.cuda.synchronize()
    for L, w in zip(layers, want):
        assert same(L.results(), w)


def test_rows_beyond_32_bit_offsets():
    # two rows 3 GB apart
    far, c = 3 << 29, 1000
    buf = torch.zeros(far + c, dtype=torch.float16, device=DEV)
    x = torch.as_strided(buf, (2, c), (far, 1))
    x.copy_(torch.randn(2, c, device=DEV))
    y = torch.empty(2, c, dtype=torch.float16, device=DEV)
    s = torch.empty_like(y)
    gamma = torch.ones(c, device=DEV)
    say("norm of far rows")
    cvx.cvx_rmsnorm(cvx.make_rmsnorm_desc(2, c, cvx.CVX_DT_F16, eps=EPS, x_stride=far), x, None, gamma, s, y)
    compare(x.cpu(), None, gamma.cpu(), cvx.CVX_DT_F16, False, (s.cpu().double(), y.cpu().double(), None), "far rows")
    del buf, x
    # projections whose rows of x and y are spread over 4.6 GB
    t, wide = 1100, 1 << 21
    c = Case(5, t, 80, 68, BF16, False, 8, 3, ids="runs")
    big = [torch.zeros(t * wide, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    x, y = (torch.as_strided(b, (t, n), (wide, 1)) for b, n in zip(big, (c.ci, c.co)))
    x.copy_(c.x.to(DEV))
    d = cvx.make_linear_desc(t, c.ci, c.co, BF16, rank=8, n_adapters=3, x_stride=wide, y_stride=wide)
    ws = torch.empty(cvx.cvx_linear_workspace_bytes(d), dtype=torch.uint8, device=DEV)
    say("projection of far rows")
    cvx.cvx_linear(d, x, c.w.to(DEV), y, None, c.scale.to(DEV), c.bias.to(DEV), None, c.a.to(DEV), c.b.to(DEV),
                   c.alpha.to(DEV), c.ids.to(DEV), ws)
    want, tol = c.definition()
    assert ((y.cpu().double() - want).abs() <= tol).all()


@pytest.mark.parametrize("t", [2, 70])
def test_weights_beyond_32_bit_offsets(t):
    ci, co = 8192, 290000
    g = torch.Generator(device=DEV).manual_seed(1)
    w = torch.empty(co, ci, dtype=torch.bfloat16, device=DEV)
    w[-300:] = torch.randn(300, ci, generator=g, device=DEV).to(torch.bfloat16) / 90
    w[:300] = 1.0
    x = torch.randn(t, ci, generator=g, device=DEV).to(torch.bfloat16)
    y = torch.empty(t, co, dtype=torch.bfloat16, device=DEV)
    say(f"projection with 4.7 GB of weights, {t} tokens")
    cvx.cvx_linear(cvx.make_linear_desc(t, ci, co, BF16), x, w, y)
    torch.cuda.synchronize()
    xd, wd = x.cpu().double(), w[-300:].cpu().double()
    want = xd @ wd.t()
    tol = ci * 2.0 ** -24 * (xd.abs() @ wd.abs().t()) + 2.0 ** -8 * want.abs() + 1e-30
    assert ((y[:, -300:].cpu().double() - want).abs() <= tol).all()
