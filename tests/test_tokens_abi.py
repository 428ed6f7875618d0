"""Refusals and host-only queries of the operators on tokens (cvx_rmsnorm,
cvx_linear): every check returns before anything is enqueued, so none of this
needs a GPU.  The addresses are never dereferenced."""
import ctypes

import pytest

from conv2d_batchnorm_activation_amd import cvx

X, R, G, S, Y, Q, W, SC, BI, LA, LB, AL, ID, WS = (0x100000000 * i for i in range(1, 15))
F32, F16, BF16, E4M3 = cvx.CVX_DT_F32, cvx.CVX_DT_F16, cvx.CVX_DT_BF16, cvx.CVX_DT_E4M3
NULL, SHAPE, UNSUPPORTED, ALIGN, ALIAS, WORKSPACE, ARG = -1, -2, -3, -4, -5, -6, -8


def norm(x=X, r=None, g=G, s=None, y=Y, q=None, **kw):
    base = dict(rows=7, c=40, dtype=BF16)
    base.update(kw)
    d = cvx.make_rmsnorm_desc(**base)
    return cvx.lib.cvx_rmsnorm(ctypes.byref(d), x, r, g, s, y, q, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=1, c=(1 << 30) + 1), SHAPE), (dict(rows=1, c=(1 << 31) - 1), SHAPE),
    (dict(rows=0), SHAPE), (dict(c=0), SHAPE), (dict(rows=-1), SHAPE), (dict(c=-8), SHAPE),
    (dict(x_stride=39), SHAPE), (dict(y_stride=-1), SHAPE), (dict(x_stride=1 << 41), SHAPE),
    (dict(rows=1 << 30, x_stride=1 << 11), SHAPE),           # 2^41 elements from first to last
    (dict(r=R, res_stride=1), SHAPE), (dict(s=S, sum_stride=1), SHAPE),
    (dict(dtype=E4M3), ARG), (dict(dtype=4), ARG), (dict(dtype=-1), ARG),
    (dict(out_dtype=F16), ARG), (dict(out_dtype=F32), ARG), (dict(out_dtype=7), ARG),
    (dict(eps=0.0), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG),
    (dict(eps=float("inf")), ARG),
    (dict(x=None), NULL), (dict(g=None), NULL), (dict(y=None), NULL),
    (dict(out_dtype=E4M3), NULL),                            # 8 bits without scales
    (dict(x=X + 1), ALIGN), (dict(y=Y + 1), ALIGN), (dict(g=G + 2), ALIGN), (dict(r=R + 1), ALIGN),
    (dict(s=S + 1), ALIGN), (dict(dtype=F32, x=X + 2), ALIGN), (dict(out_dtype=E4M3, q=Q + 2), ALIGN),
    (dict(y=X), ALIAS), (dict(y=X + 2 * (7 * 40 - 1)), ALIAS), (dict(y=G + 4 * 39), ALIAS),
    (dict(r=R, y=R), ALIAS), (dict(s=Y), ALIAS), (dict(s=X + 2), ALIAS),
    (dict(s=X, x_stride=48), ALIAS),                         # the same address, another stride
    (dict(r=R, s=R, res_stride=48), ALIAS),
    (dict(out_dtype=E4M3, q=Y + 4), ALIAS), (dict(out_dtype=E4M3, q=X), ALIAS),
    (dict(x_stride=100, y=X + 2 * 40), ALIAS),               # between x's rows: inside its range
])
def test_rmsnorm_refusals(kw, code):
    assert norm(**kw) == code


def test_rmsnorm_null_descriptor():
    assert cvx.lib.cvx_rmsnorm(None, X, None, G, None, Y, None, None) == NULL


def lin_desc(**kw):
    base = dict(tokens=33, c_in=64, c_out=48, dtype=BF16)
    base.update(kw)
    return cvx.make_linear_desc(**base)


def lin(x=X, xs=None, w=W, sc=SC, bi=BI, r=None, la=None, lb=None, al=None, ids=None, y=Y, ws=None, wb=0, **kw):
    d = lin_desc(**kw)
    return cvx.lib.cvx_linear(ctypes.byref(d), x, xs, w, sc, bi, r, la, lb, al, ids, y, ws, wb, None)


LORA = dict(la=LA, lb=LB, al=AL, ids=ID, ws=WS, wb=1 << 30, rank=16, n_adapters=3)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=0), SHAPE), (dict(c_in=0), SHAPE), (dict(c_out=0), SHAPE), (dict(tokens=-3), SHAPE),
    (dict(tokens=(1 << 24) + 1), SHAPE), (dict(c_in=(1 << 20) + 8), SHAPE), (dict(c_out=(1 << 20) + 4), SHAPE),
    (dict(x_stride=56), SHAPE), (dict(y_stride=44), SHAPE), (dict(x_stride=(1 << 21) + 8), SHAPE),
    (dict(res_mode=1, r=R, res_stride=44), SHAPE), (dict(y_stride=-4), SHAPE),
    (dict(dtype=F32), ARG), (dict(dtype=E4M3), ARG), (dict(dtype=9), ARG), (dict(x_dtype=F16), ARG),
    (dict(x_dtype=F32), ARG), (dict(act=3), ARG), (dict(act=-1), ARG), (dict(res_mode=3), ARG),
    (dict(rank=16), ARG), (dict(n_adapters=2), ARG), (dict(rank=-8, n_adapters=1), ARG),
    (dict(rank=8, n_adapters=-1), ARG),
    (dict(c_in=60), UNSUPPORTED), (dict(c_out=46), UNSUPPORTED), (dict(x_stride=68), UNSUPPORTED),
    (dict(y_stride=50), UNSUPPORTED), (dict(res_mode=2, r=R, res_stride=50), UNSUPPORTED),
    (dict(x_dtype=E4M3, c_in=72, xs=Q), UNSUPPORTED), (dict(x_dtype=E4M3, x_stride=72, xs=Q), UNSUPPORTED),
    (dict(rank=12, n_adapters=1), UNSUPPORTED), (dict(rank=136, n_adapters=1), UNSUPPORTED),
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(y=None), NULL), (dict(x_dtype=E4M3), NULL),
    (dict(res_mode=1), NULL), (dict(LORA, la=None), NULL), (dict(LORA, lb=None), NULL), (dict(LORA, ids=None), NULL),
    (dict(x=X + 8), ALIGN), (dict(w=W + 8), ALIGN), (dict(sc=SC + 4), ALIGN), (dict(bi=BI + 8), ALIGN),
    (dict(y=Y + 4), ALIGN), (dict(res_mode=1, r=R + 4), ALIGN), (dict(LORA, la=LA + 8), ALIGN),
    (dict(LORA, lb=LB + 2), ALIGN), (dict(LORA, al=AL + 2), ALIGN), (dict(LORA, ids=ID + 1), ALIGN),
    (dict(x_dtype=E4M3, xs=Q + 2), ALIGN), (dict(LORA, ws=WS + 8), ALIGN),
    (dict(y=X), ALIAS), (dict(y=X + 2 * 33 * 64 - 8), ALIAS), (dict(y=W), ALIAS), (dict(y=SC), ALIAS),
    (dict(y=BI), ALIAS), (dict(res_mode=2, r=Y), ALIAS), (dict(LORA, y=LA + 16), ALIAS), (dict(LORA, y=LB), ALIAS),
    (dict(LORA, y=AL), ALIAS), (dict(LORA, y=ID), ALIAS), (dict(x_dtype=E4M3, xs=Y), ALIAS),
    (dict(LORA, ws=Y), ALIAS), (dict(LORA, ws=X), ALIAS), (dict(LORA, ws=LB), ALIAS), (dict(LORA, ws=ID), ALIAS),
    (dict(LORA, ws=None), WORKSPACE), (dict(LORA, wb=16), WORKSPACE),
])
def test_linear_refusals(kw, code):
    assert lin(**kw) == code


def test_linear_null_descriptor():
    assert cvx.lib.cvx_linear(None, X, None, W, None, None, None, None, None, None, None, Y, None, 0, None) == NULL
    assert cvx.lib.cvx_linear_workspace_bytes(None) == 0


def test_linear_queries():
    assert cvx.cvx_linear_workspace_bytes(lin_desc()) == 0
    assert cvx.cvx_linear_workspace_bytes(lin_desc(c_in=60)) == 0
    # one token takes up to 16 ranks in the projection's own kernel
    assert cvx.cvx_linear_workspace_bytes(lin_desc(tokens=1, rank=16, n_adapters=3)) == 0
    assert cvx.cvx_linear_workspace_bytes(lin_desc(tokens=1, rank=24, n_adapters=3)) > 0
    # ... of weights up to 3 * 2^24 values
    assert cvx.cvx_linear_workspace_bytes(lin_desc(tokens=1, c_in=4096, c_out=12288, rank=16, n_adapters=3)) == 0
    assert cvx.cvx_linear_workspace_bytes(lin_desc(tokens=1, c_in=4096, c_out=12292, rank=16, n_adapters=3)) > 0
    for t in (2, 17, 64, 65, 300, 5000):
        d = lin_desc(tokens=t, c_in=4096, rank=16, n_adapters=3)
        need = cvx.cvx_linear_workspace_bytes(d)
        assert need >= 4 * t * 16
        assert lin(**dict(LORA, tokens=t, c_in=4096, wb=need - 1)) == WORKSPACE
        assert "kernel=cvx::k_linear" in cvx.cvx_linear_plan(d)
    buf = ctypes.create_string_buffer(4)
    d = lin_desc()
    assert cvx.lib.cvx_linear_plan(ctypes.byref(d), buf, 4) == 0 and buf.value == b"lin"
    assert cvx.lib.cvx_linear_plan(ctypes.byref(d), None, 4) == NULL
    assert cvx.lib.cvx_linear_plan(ctypes.byref(d), buf, 0) == NULL


def test_older_calls_do_not_take_8_bits():
    d = cvx.make_desc(1, 64, 8, 8, 64, 1, 1, 0)
    assert cvx.cvx_nhwc_packed_weights_bytes(d, E4M3) == 0
    assert cvx.lib.cvx_conv_bn_act_nhwc(ctypes.byref(d), E4M3, X, W, SC, BI, None, Y, None) == ARG


def test_host_tensors_are_refused():
    import torch
    t = torch.zeros(8, 64)
    with pytest.raises(ValueError):
        cvx.cvx_rmsnorm(cvx.make_rmsnorm_desc(8, 64, F32), t, None, t[0], None, t.clone())
    with pytest.raises(ValueError):
        cvx.cvx_linear(lin_desc(tokens=8, c_out=64), t, t, t.clone())
    # ... whichever they are: the rest are addresses here, which no call is made with
    for i in range(1, 6):
        args = [X, R, SC, W, Y, Q]
        args[i] = t
        with pytest.raises(ValueError):
            cvx.cvx_rmsnorm(cvx.make_rmsnorm_desc(8, 64, F32, E4M3), *args)
    for i in range(1, 12):
        args = [X, W, Y, Q, SC, BI, R, LA, LB, AL, ID, WS]
        args[i] = t
        with pytest.raises(ValueError):
            cvx.cvx_linear(lin_desc(tokens=8, c_out=64), *args)
