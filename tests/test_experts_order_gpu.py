"""The experts of a layer (two products grouped by expert, the gate between them) on streams of their own and in
replayed graphs, over other inputs each pass and buffers that are filled with a pattern before it: what a
launch leaves out, or reads before it is there, shows."""
import pytest
import torch

from gpu_util import DEV, say
from test_grouped_gpu import Experts

pytestmark = pytest.mark.gpu

from conv2d_batchnorm_activation_amd import cvx  # noqa: E402

BF16, E4M3, I8 = cvx.CVX_DT_BF16, cvx.CVX_DT_E4M3, cvx.CVX_DT_I8


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def written(L):
    """What a pass writes: the first product, codes or values between the products, their scales, the second product."""
    return [m for m in (L.one.ybuf, L.a, L.q, L.two.ybuf) if m is not None]


def poison(L):
    for m in written(L):
        m.view(torch.uint8).fill_(255)


def results(L):
    return [m.view(torch.uint8).clone() for m in written(L)]


class Inputs:
    """Two inputs of a layer and what it makes of each, run alone over poisoned buffers."""

    def __init__(self, L):
        self.x = L.args[0][1].view(torch.uint8)
        self.values = [self.x.clone(), self.x.flip(0).contiguous()]
        self.want = []
        for v in self.values:
            poison(L)
            self.x.copy_(v)
            L.run()
            torch.cuda.synchronize()
            self.want.append(results(L))
        assert not any(torch.equal(a, b) for a, b in zip(*self.want))

    def set(self, i):
        self.x.copy_(self.values[i % 2])

    def same(self, i, got):
        return all(torch.equal(a, b) for a, b in zip(got, self.want[i % 2]))


def test_on_streams_of_their_own():
    layers = [Experts(t, 2, 6, 272, 144, h, 40 + t) for t, h in ((5, BF16), (90, I8), (400, E4M3), (40, E4M3))]
    inputs = [Inputs(L) for L in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    say("experts on streams of their own, poisoned before each pass")
    for i in range(6):
        torch.cuda.synchronize()
        for L, p, s in zip(layers, inputs, streams):
            with torch.cuda.stream(s):
                poison(L)
                p.set(i)
            L.run(s)
        torch.cuda.synchronize()
        for L, p in zip(layers, inputs):
            assert p.same(i, results(L)), (i, L.t)


@pytest.mark.parametrize("held", [BF16, E4M3, I8])
@pytest.mark.parametrize("t", [1, 9, 150, 900])
def test_in_replayed_graphs(t, held):
    L = Experts(t, 3, 7, 272, 144, held, t)
    p = Inputs(L) if t > 1 else None
    say(f"experts in replayed graphs, {t} tokens, held={held}")
    if p is None:
        poison(L)
        L.run()
        torch.cuda.synchronize()
        want = results(L)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        L.run()
    for i in range(5):
        poison(L)
        if p is not None:
            p.set(i)
        graph.replay()
        torch.cuda.synchronize()
        got = results(L)
        assert p.same(i, got) if p is not None else all(torch.equal(a, b) for a, b in zip(got, want))
        torch.empty(1 << 20, device=DEV).normal_()  # eager work between the replays
        torch.cuda.synchronize()
