"""Refusals of the gated activation: nothing here needs a GPU, and the addresses are never
dereferenced."""
import ctypes

import pytest
import torch

from conv2d_batchnorm_activation_amd import cvx
from test_tokens_abi import ALIAS, ALIGN, ARG, BF16, E4M3, F16, F32, NULL, Q, SHAPE, X, Y
from test_tokens_binding import HELD, On, taken  # noqa: F401

P = 0x100000000 * 20
I8 = cvx.CVX_DT_I8


def gate(g=X, p=P, y=Y, q=None, **kw):
    d = cvx.make_gate_desc(**{**dict(rows=7, c=40, dtype=BF16), **kw})
    return cvx.lib.cvx_gate(ctypes.byref(d), g, p, y, q, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), SHAPE), (dict(c=0), SHAPE), (dict(rows=-1), SHAPE), (dict(rows=1, c=(1 << 30) + 1), SHAPE),
    (dict(gate_stride=39), SHAPE), (dict(up_stride=1), SHAPE), (dict(y_stride=-1), SHAPE), (dict(gate_stride=1 << 41), SHAPE),
    (dict(rows=1 << 30, up_stride=1 << 11), SHAPE),
    (dict(dtype=E4M3), ARG), (dict(dtype=I8), ARG), (dict(dtype=-1), ARG), (dict(out_dtype=F16), ARG),
    (dict(out_dtype=F32), ARG), (dict(out_dtype=5), ARG), (dict(act=3), ARG), (dict(act=-1), ARG),
    (dict(g=None), NULL), (dict(y=None), NULL), (dict(out_dtype=I8), NULL), (dict(out_dtype=E4M3), NULL),
    (dict(g=X + 1), ALIGN), (dict(p=P + 1), ALIGN), (dict(y=Y + 1), ALIGN), (dict(dtype=F32, p=P + 2), ALIGN),
    (dict(out_dtype=I8, q=Q + 2), ALIGN),
    (dict(y=X), ALIAS), (dict(y=P), ALIAS), (dict(y=X + 2 * (7 * 40 - 1)), ALIAS), (dict(p=Y + 2), ALIAS),
    (dict(out_dtype=I8, q=Y + 276), ALIAS), (dict(out_dtype=I8, q=X), ALIAS), (dict(out_dtype=I8, q=P + 4), ALIAS),
    (dict(gate_stride=100, y=X + 2 * 40), ALIAS),
])
def test_refusals(kw, code):
    assert gate(**kw) == code


def test_null_descriptor():
    assert cvx.lib.cvx_gate(None, X, P, Y, None, None) == NULL


NAMES = ("gate", "up", "y", "y_scale")


def operands(dt, out, device=0):
    t = {n: On(HELD[dt], device, (i + 1) << 32) for i, n in enumerate(NAMES)}
    t["y"].dtype = cvx._HELD[out]
    t["y_scale"].dtype = torch.float32
    return t


def call(t, dt, out):
    cvx.cvx_gate(cvx.make_gate_desc(2, 32, dt, out), *(t[n] for n in NAMES))


@pytest.mark.parametrize("dt,out", [(BF16, I8), (F16, E4M3), (F32, F32)])
def test_binding(taken, dt, out):  # noqa: F811
    call(operands(dt, out), dt, out)
    assert len(taken) == 1 and taken[0][0] == "cvx_gate"
    for n in NAMES:
        t = operands(dt, out)
        t[n].device = -1 if n == "gate" else 1
        with pytest.raises(ValueError, match=n):
            call(t, dt, out)
        t = operands(dt, out)
        t[n].dtype = torch.int64
        with pytest.raises(ValueError, match=n):
            call(t, dt, out)
    assert len(taken) == 1
