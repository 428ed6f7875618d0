"""Refusals and host-only queries of the products grouped by expert: nothing here needs a GPU, and
the addresses are never dereferenced."""
import ctypes

import pytest
import torch

from conv2d_batchnorm_activation_amd import cvx
from test_tokens_abi import ALIAS, ALIGN, ARG, BF16, E4M3, F16, F32, NULL, SHAPE, UNSUPPORTED
from test_tokens_binding import On, taken  # noqa: F401

I8 = cvx.CVX_DT_I8
X, Q, W, SC, BI, OF, ID, RW, Y = (0x1000000000000 * i for i in range(1, 10))


def desc(**kw):
    return cvx.make_grouped_desc(**{**dict(rows=33, tokens=33, n_groups=5, c_in=64, c_out=48, dtype=BF16), **kw})


def call(x=X, xs=None, w=W, sc=SC, bi=BI, of=OF, ids=None, rw=None, y=Y, **kw):
    d = desc(**kw)
    return cvx.lib.cvx_linear_grouped(ctypes.byref(d), x, xs, w, sc, bi, of, ids, rw, y, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), SHAPE), (dict(tokens=0, ids=ID), SHAPE), (dict(c_in=0), SHAPE), (dict(c_out=0), SHAPE),
    (dict(n_groups=0), SHAPE), (dict(n_groups=1025), SHAPE), (dict(n_groups=-1), SHAPE), (dict(rows=-4), SHAPE),
    (dict(rows=(1 << 24) + 1, ids=ID), SHAPE), (dict(tokens=(1 << 24) + 1), SHAPE), (dict(c_in=(1 << 20) + 8), SHAPE),
    (dict(c_out=(1 << 20) + 4), SHAPE), (dict(rows=1 << 24, tokens=1 << 24, c_out=(1 << 13) + 4), SHAPE),
    (dict(n_groups=1024, c_in=1 << 20, c_out=1028), SHAPE),             # 2^40 weights and some
    (dict(tokens=32), SHAPE),                                           # fewer rows of x than of y
    (dict(x_stride=56), SHAPE), (dict(y_stride=44), SHAPE), (dict(x_stride=(1 << 21) + 8), SHAPE), (dict(y_stride=-4), SHAPE),
    (dict(ids=ID, tokens=(1 << 24) + 8, c_in=64), SHAPE),
    (dict(ids=ID, tokens=1 << 24, c_in=72), SHAPE),                     # 2^31 bytes and some, by number
    (dict(ids=ID, tokens=1025, c_in=64, x_stride=1 << 20), SHAPE),
    (dict(x_dtype=I8, c_in=1 << 17, xs=Q), SHAPE),
    (dict(dtype=F32), ARG), (dict(dtype=E4M3), ARG), (dict(dtype=I8, x_dtype=I8), ARG), (dict(x_dtype=F16), ARG),
    (dict(x_dtype=5), ARG), (dict(act=3), ARG), (dict(act=-1), ARG),
    (dict(c_in=60), UNSUPPORTED), (dict(c_out=46), UNSUPPORTED), (dict(x_stride=68), UNSUPPORTED), (dict(y_stride=50), UNSUPPORTED),
    (dict(x_dtype=E4M3, c_in=72, xs=Q), UNSUPPORTED), (dict(x_dtype=I8, x_stride=72, xs=Q), UNSUPPORTED),
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(y=None), NULL), (dict(of=None), NULL), (dict(x_dtype=E4M3), NULL),
    (dict(x_dtype=I8), NULL),
    (dict(x=X + 8), ALIGN), (dict(w=W + 8), ALIGN), (dict(y=Y + 4), ALIGN), (dict(sc=SC + 2), ALIGN), (dict(bi=BI + 1), ALIGN),
    (dict(of=OF + 2), ALIGN), (dict(ids=ID + 1), ALIGN), (dict(rw=RW + 2), ALIGN), (dict(x_dtype=I8, xs=Q + 2), ALIGN),
    (dict(y=X), ALIAS), (dict(y=X + 2 * 33 * 64 - 8), ALIAS), (dict(y=W), ALIAS), (dict(y=W + 2 * 5 * 48 * 64 - 8), ALIAS),
    (dict(y=SC), ALIAS), (dict(y=BI + 4 * 5 * 48 - 8), ALIAS), (dict(y=OF + 16), ALIAS), (dict(y=ID, ids=ID), ALIAS),
    (dict(y=RW + 128, rw=RW), ALIAS), (dict(x_dtype=E4M3, xs=Y), ALIAS), (dict(of=Y + 33 * 48 * 2 - 4), ALIAS),
])
def test_refusals(kw, code):
    assert call(**kw) == code


def test_null_descriptor():
    assert cvx.lib.cvx_linear_grouped(None, X, None, W, None, None, OF, None, None, Y, None) == NULL
    buf = ctypes.create_string_buffer(64)
    assert cvx.lib.cvx_linear_grouped_plan(None, buf, 64) == NULL


def test_plans():
    buf = ctypes.create_string_buffer(8)
    d = desc()
    assert cvx.lib.cvx_linear_grouped_plan(ctypes.byref(d), buf, 8) == 0 and buf.value == b"grouped"
    assert cvx.lib.cvx_linear_grouped_plan(ctypes.byref(d), None, 8) == NULL
    assert cvx.lib.cvx_linear_grouped_plan(ctypes.byref(d), buf, 0) == NULL
    for rows in (1, 8, 100, 5000, 1 << 20, 1 << 24):
        for n in (1, 8, 128, 1024):
            for c_in, c_out in ((8, 4), (64, 260), (4096, 8192), (1 << 16, 64)):
                if rows * c_out > 1 << 37 or rows * c_in > 1 << 40:
                    continue
                for x in (BF16, E4M3, I8):
                    if x != BF16 and c_in == 8:
                        continue
                    plan = cvx.cvx_linear_grouped_plan(desc(rows=rows, tokens=rows, n_groups=n, c_in=c_in, c_out=c_out, x_dtype=x))
                    assert plan.startswith("grouped ") and "kernel=cvx::k_" in plan
                    groups = int(plan.split("workgroups=")[1].split()[0])
                    kind = plan.split()[1]
                    assert groups % 8 == 0 and groups <= 512 if kind == "tile" else kind == "few" and groups <= 512


NAMES = ("x", "w", "offset", "y", "x_scale", "scale", "bias", "row_id", "row_weight")


def operands(dt, held, device=0):
    t = {n: On(torch.float32, device, (i + 1) << 40) for i, n in enumerate(NAMES)}
    t["x"].dtype = t["w"].dtype = cvx._HELD[held]
    t["y"].dtype = cvx._HELD[dt]
    t["offset"].dtype = t["row_id"].dtype = torch.int32
    return t


def bound(t, dt, held):
    cvx.cvx_linear_grouped(desc(dtype=dt, x_dtype=held), *(t[n] for n in NAMES))


@pytest.mark.parametrize("dt,held", [(BF16, BF16), (F16, E4M3), (BF16, I8)])
def test_binding(taken, dt, held):  # noqa: F811
    bound(operands(dt, held), dt, held)
    assert len(taken) == 1 and taken[0][0] == "cvx_linear_grouped"
    assert [a for a in taken[0][1][1:10]] == [(NAMES.index(n) + 1) << 40 for n in
                                             ("x", "x_scale", "w", "scale", "bias", "offset", "row_id", "row_weight", "y")]
    for n in NAMES:
        t = operands(dt, held)
        t[n].device = -1 if n == "x" else 1
        with pytest.raises(ValueError, match=n):
            bound(t, dt, held)
        for wrong in (torch.int64, torch.float64, torch.uint8 if held != E4M3 else torch.int16):
            t = operands(dt, held)
            t[n].dtype = wrong
            with pytest.raises(ValueError, match=n):
                bound(t, dt, held)
    assert len(taken) == 1
