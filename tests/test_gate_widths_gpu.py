"""cvx_gate to 8 bits at the widths where a long row's threads, or the vectors each holds, change: by the
definition and the bounds of test_gate_gpu.py."""
import pytest
import torch

from gpu_util import DEV, say
from test_gate_gpu import BF16, DT, E4M3, F16, F32, I8, NONE, SILU, check, rows_of

pytestmark = pytest.mark.gpu

from conv2d_batchnorm_activation_amd import cvx  # noqa: E402


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# vectors of 16 bytes
@pytest.mark.parametrize("dt,vectors", [(BF16, 1280), (F16, 1792), (BF16, 2048), (F16, 2560), (BF16, 3 * 1024), (F16, 4096),
                                        (F32, 1280), (F32, 1791), (F32, 1792), (F32, 2048), (F32, 2560), (F32, 3 * 1024), (F32, 4096),
                                        (F32, 6144)])
@pytest.mark.parametrize("out", [I8, E4M3])
def test_long_rows(dt, vectors, out):
    c = vectors * (4 if dt == F32 else 8)
    for n in (c - 3, c, c + 1):
        g, p = rows_of(n, 11, n, dt)
        check(g, p, dt, out, NONE, (0, 0, 0) if n % 2 else (4, 8, 4))


@pytest.mark.parametrize("dt,c", [(BF16, 40000), (F32, 30000)])
def test_rows_too_long_to_be_held(dt, c):
    # read again for every step, in a replayed graph over other values
    g, p = (m.to(DEV) for m in rows_of(5, 130, c, dt))
    y, q = torch.empty(130, c, dtype=DT[I8], device=DEV), torch.empty(130, device=DEV)
    d = cvx.make_gate_desc(130, c, dt, I8, SILU)
    say(f"gate of rows too long to be held, c={c} dt={dt}")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        cvx.cvx_gate(d, g, p, y, q)
    for _ in range(3):
        g.normal_()
        y.fill_(55)
        q.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone(), q.clone()
        y.fill_(55)
        q.fill_(-1)
        cvx.cvx_gate(d, g, p, y, q)
        torch.cuda.synchronize()
        assert torch.equal(got[0], y) and torch.equal(got[1], q) and (q > 0).all() and (y.abs() == 127).any(1).all()
