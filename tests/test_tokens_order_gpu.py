"""The operators on tokens leave nothing out and keep nothing: on streams of their own and
in replayed graphs, with every output and the workspace filled with NaN before each
pass and other inputs from pass to pass, a layer gives what it gives alone.  And the
largest tile with every fill of its rank loop."""
import pytest
import torch

from gpu_util import DEV, say
from test_linear_gpu import BF16, F16, SILU, Case
from test_tokens_run_gpu import Layer, same

pytestmark = pytest.mark.gpu

from conv2d_batchnorm_activation_amd import cvx  # noqa: E402


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def poison(L):
    for m in (L.codes, L.scales, L.y1, L.sum, L.n2, L.out, L.ws):
        m.view(torch.uint8).fill_(255)


def inputs_of(L, passes):
    g = torch.Generator(device=DEV).manual_seed(L.t)
    return [torch.randn(L.t, L.c, generator=g, device=DEV).to(torch.bfloat16) for _ in range(passes)]


def alone(L, x):
    L.x.copy_(x)
    poison(L)
    torch.cuda.synchronize()
    L.run()
    torch.cuda.synchronize()
    got = L.results()
    assert all(torch.isfinite(m.float()).all() for m in got)
    return got


@pytest.mark.parametrize("named", [False, True], ids=["current", "argument"])
def test_layers_on_streams_with_other_inputs_each_pass(named):
    passes = 5
    layers = [Layer(t, seed=70 + t) for t in (1, 30, 150, 700)]
    xs = [inputs_of(L, passes) for L in layers]
    want = [[alone(L, x) for x in mine] for L, mine in zip(layers, xs)]
    for L in layers:
        poison(L)
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    say("layers on streams of their own")
    got = [[] for _ in layers]
    for k in range(passes):
        for L, x, s, out in zip(layers, xs, streams, got):
            with torch.cuda.stream(s):
                L.x.copy_(x[k])
                poison(L)
                if not named:
                    L.run()
            if named:
                L.run(stream=s)
            with torch.cuda.stream(s):
                out.append(L.results())
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert not same(w[0], w[1])
        for a, b in zip(w, g):
            assert same(a, b)


@pytest.mark.parametrize("t", [1, 8, 40, 130, 700])
def test_replays_with_other_inputs(t):
    L = Layer(t, seed=90 + t)
    xs = inputs_of(L, 3)
    want = [alone(L, x) for x in xs]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    say(f"graph of a layer of {t} tokens")
    with torch.cuda.graph(graph, stream=stream):
        L.run()
    for k in (0, 1, 2, 1, 0):
        L.x.copy_(xs[k])
        poison(L)
        graph.replay()
        torch.cuda.synchronize()
        assert same(L.results(), want[k])
        assert same(alone(L, xs[(k + 1) % 3]), want[(k + 1) % 3])  # eager work between the replays


def test_two_graphs_with_a_workspace_each():
    a, b = Layer(200, seed=11), Layer(200, seed=12)
    xa, xb = inputs_of(a, 2), inputs_of(b, 2)[::-1]
    wa, wb = [alone(a, x) for x in xa], [alone(b, x) for x in xb]
    graphs = []
    for L in (a, b):
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=stream):
            L.run()
    streams = [torch.cuda.Stream() for _ in graphs]
    say("two graphs at once")
    for k in (0, 1, 0):
        a.x.copy_(xa[k])
        b.x.copy_(xb[k])
        poison(a)
        poison(b)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert same(a.results(), wa[k]) and same(b.results(), wb[k])


@pytest.mark.parametrize("x8", [False, True], ids=["x16", "x8"])
@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("rank", [8, 16, 24, 64, 128])
def test_linear_largest_tile_with_every_rank(rank, dt, x8):
    for ids in ("runs", "each"):
        c = Case(rank, 4099, 80, 3588, dt, x8, rank, 4, SILU, 2, ids=ids, pads=(16, 4, 12))
        assert "tile 256x256" in c.describe()
        c.check()


@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("n,c_in,c_out,side", [(1, 64, 48, 7), (2, 32, 68, 13), (1, 128, 256, 40)])
def test_a_channels_last_layer_is_a_projection_of_its_pixels(n, c_in, c_out, side, dt):
    # the output of a 1x1 layer, its pixels taken as rows, is what cvx_linear gives of them:
    # both round their fp32 sums (K products, scale, bias, residual) once
    f = torch.float64
    tdt = torch.float16 if dt == F16 else torch.bfloat16
    g = torch.Generator().manual_seed(c_out)
    rows = n * side * side
    x = torch.randn(rows, c_in, generator=g).to(tdt)
    w = (torch.randn(c_out, c_in, generator=g) / c_in ** 0.5).to(tdt)
    scale, bias = 1 + 0.1 * torch.randn(c_out, generator=g), torch.randn(c_out, generator=g)
    res = torch.randn(rows, c_out, generator=g).to(tdt)
    X, S, B, R = (m.to(DEV) for m in (x, scale, bias, res))
    d = cvx.make_desc(n, c_in, side, side, c_out, 1, 1, 0, act=cvx.CVX_ACT_SILU, res_mode=cvx.CVX_RES_BEFORE_ACT)
    packed = torch.empty(cvx.cvx_nhwc_packed_weights_bytes(d, dt), dtype=torch.uint8, device=DEV)
    w32 = w.float().reshape(c_out, c_in, 1, 1).to(DEV)
    layer, linear = (torch.full((rows, c_out), float("nan"), dtype=tdt, device=DEV) for _ in range(2))
    say(f"channels-last layer and projection, {rows} pixels {c_in} -> {c_out}")
    cvx.cvx_nhwc_pack_weights(d, dt, w32, packed)
    cvx.cvx_conv_bn_act_nhwc(d, dt, X, packed, S, B, R, layer)
    cvx.cvx_linear(cvx.make_linear_desc(rows, c_in, c_out, dt, act=cvx.CVX_ACT_SILU, res_mode=cvx.CVX_RES_BEFORE_ACT),
                   X, w.to(DEV), linear, None, S, B, R)
    z = (x.to(f) @ w.to(f).t()) * scale.to(f) + bias.to(f) + res.to(f)
    mag = (x.to(f).abs() @ w.to(f).abs().t()) * scale.to(f).abs() + bias.to(f).abs() + res.to(f).abs()
    want = z * torch.sigmoid(z)
    err = 1.1 * (c_in + 20) * 2.0 ** -24 * mag
    tol = err + torch.finfo(tdt).eps / 2 * (want.abs() + err) + torch.finfo(tdt).smallest_normal * torch.finfo(tdt).eps
    for name, got in (("layer", layer), ("projection", linear)):
        assert ((got.cpu().double() - want).abs() <= tol).all(), name
