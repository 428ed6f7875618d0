"""cvx_gate to 8 bits, rows whose largest value all but vanishes: SiLU of a gate far below zero, times
a small factor, is a value of 64 bits whose M*(1/t) is none.  Such rows are zeros, with a scale of zero;
one whose M*(1/t) is finite has the codes of the formula, whose scale is zero all the same.

The values of a row are one gate's times factors, so u/t is a ratio of factors and the exponential, which the
two sides may take differently, cancels but for a few roundings of 2^-53: codes are compared where u*f
lies further than 2^-40 of itself from a border."""
import pytest
import torch

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

from conv2d_batchnorm_activation_amd import cvx  # noqa: E402

F32, BF16, E4M3, I8 = cvx.CVX_DT_F32, cvx.CVX_DT_BF16, cvx.CVX_DT_E4M3, cvx.CVX_DT_I8
DT = {F32: torch.float32, BF16: torch.bfloat16, E4M3: torch.float8_e4m3fn, I8: torch.int8}
MOST = {E4M3: 448.0, I8: 127.0}


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# gate and factor of the row's largest value: M*(1/t) is a finite 64-bit value in some
ROWS = [(-700.0, 1e-5), (-700.0, 1e-3), (-709.0, 1e-1), (-650.0, 1e-30), (-650.0, 1e-20), (-700.0, 1e-30), (-708.0, 1e-38),
        (-600.0, 1e-38)]


@pytest.mark.parametrize("c", [1, 24, 100, 700, 4100, 40000])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("out", [E4M3, I8])
def test_rows_that_all_but_vanish(out, dt, c):
    g, p = torch.full((len(ROWS) + 1, c), -720.0), torch.zeros(len(ROWS) + 1, c)
    for i, (a, b) in enumerate(ROWS):
        n = min(c, 9)
        g[i, :n], p[i, :n] = a, b * torch.tensor([1.0, 0.8, -0.3, 0.05, 0.6, -1.0, 0.0, 0.11, -0.02])[:n]
    g[-1], p[-1] = 1.0, 1.0  # and one as rows are
    g, p = g.to(DT[dt]), p.to(DT[dt])
    rows = len(g)
    y, q = torch.full((rows, c), 99, device=DEV).to(DT[out]), torch.full((rows,), 7.0, device=DEV)
    say(f"gate of rows that all but vanish: c={c} dt={dt} out={out}")
    cvx.cvx_gate(cvx.make_gate_desc(rows, c, dt, out), g.to(DEV), p.to(DEV), y, q)
    torch.cuda.synchronize()
    got, q = (y.float() if out == E4M3 else y).cpu().double(), q.cpu()
    assert q[:-1].tolist() == [0.0] * len(ROWS) and (got[-1] == MOST[out]).all()
    gd = g.double()
    u = gd / (1 + torch.exp(-gd)) * p.double()
    told = 0
    for i in range(len(ROWS)):
        t = u[i].abs().max()
        f = MOST[out] * (1.0 / t)
        if not torch.isfinite(f):
            assert (got[i] == 0).all(), got[i, :9].tolist()
            continue
        told += 1
        v = u[i] * f
        step = torch.ones_like(v) if out == I8 else torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
        off = (v / step - torch.floor(v / step) - 0.5).abs() * step
        assert torch.equal(got[i], torch.where(off < 2.0 ** -40 * v.abs(), got[i], torch.round(v / step) * step))
    assert 2 < told < len(ROWS) - 2


def test_such_rows_are_zeros_to_a_projection():
    # a token that all but vanishes is its projection's bias, whatever stands beside it
    t, c, co = 70, 64, 132
    for n in (3, t):
        g, p = torch.ones(n, c, device=DEV), torch.ones(n, c, device=DEV)
        g[1], p[1], p[1, 0] = -700.0, 0.0, 1e-5
        y, q = torch.empty(n, c, device=DEV).to(DT[E4M3]), torch.empty(n, device=DEV)
        say(f"such a row projected, {n} tokens")
        cvx.cvx_gate(cvx.make_gate_desc(n, c, F32, E4M3), g, p, y, q)
        w = torch.ones(co, c, device=DEV).to(DT[E4M3])
        bias = torch.arange(co, device=DEV).float()
        out = torch.empty(n, co, dtype=torch.bfloat16, device=DEV)
        cvx.cvx_linear(cvx.make_linear_desc(n, c, co, BF16, E4M3), y, w, out, q, None, bias)
        assert torch.equal(out[1], bias.bfloat16()) and torch.isfinite(out.float()).all()
