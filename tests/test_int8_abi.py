"""Refusals and host-only queries of the 8-bit integers: nothing here needs a GPU, and the
addresses are never dereferenced."""
import ctypes

import pytest
import torch

from conv2d_batchnorm_activation_amd import cvx
from test_tokens_abi import ALIAS, ALIGN, ARG, BF16, E4M3, F16, F32, NULL, Q, SHAPE, UNSUPPORTED, X, Y, lin, lin_desc, norm
from test_tokens_binding import On, linear_call, linear_operands, norm_call, norm_operands, taken  # noqa: F401

I8 = cvx.CVX_DT_I8


@pytest.mark.parametrize("kw,code", [
    (dict(out_dtype=I8), NULL), (dict(out_dtype=I8, q=Q + 2), ALIGN), (dict(out_dtype=I8, q=X), ALIAS),
    (dict(out_dtype=I8, q=Y + 4), ALIAS), (dict(dtype=I8, out_dtype=I8, q=Q), ARG), (dict(dtype=I8), ARG),
    (dict(out_dtype=5, q=Q), ARG), (dict(out_dtype=I8, q=Q, y_stride=39), SHAPE),
    # codes of seven rows end 280 bytes on
    (dict(out_dtype=I8, q=Y + 276), ALIAS),
])
def test_norm_refusals(kw, code):
    assert norm(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x_dtype=I8), NULL), (dict(x_dtype=I8, xs=Q + 2), ALIGN), (dict(x_dtype=I8, xs=Y), ALIAS),
    (dict(x_dtype=I8, c_in=72, xs=Q), UNSUPPORTED), (dict(x_dtype=I8, x_stride=72, xs=Q), UNSUPPORTED),
    (dict(x_dtype=I8, c_in=1 << 17, xs=Q), SHAPE), (dict(x_dtype=5, xs=Q), ARG), (dict(dtype=I8), ARG),
    (dict(dtype=I8, x_dtype=I8, xs=Q), ARG), (dict(x_dtype=I8, xs=Q, y=X + 33 * 64 - 8), ALIAS),
])
def test_linear_refusals(kw, code):
    assert lin(**kw) == code


def test_longest_rows_of_integers():
    # 2^17 - 16 products of 2^14 at most: below 2^31
    assert ((1 << 17) - 16) << 14 < 1 << 31
    assert "kernel=cvx::k_linear" in cvx.cvx_linear_plan(lin_desc(x_dtype=I8, c_in=(1 << 17) - 16))
    with pytest.raises(cvx.CvxError):
        cvx.cvx_linear_plan(lin_desc(x_dtype=I8, c_in=1 << 17))
    assert cvx.cvx_linear_workspace_bytes(lin_desc(x_dtype=I8, c_in=1 << 17, rank=8, n_adapters=1)) == 0
    assert "k_linear" in cvx.cvx_linear_plan(lin_desc(x_dtype=E4M3, c_in=1 << 17))


def test_convolutions_do_not_take_integers():
    d = cvx.make_desc(1, 64, 8, 8, 64, 1, 1, 0)
    assert cvx.cvx_nhwc_packed_weights_bytes(d, I8) == 0


@pytest.mark.parametrize("make,call,dt,at", [(norm_operands, norm_call, BF16, ("y",)), (norm_operands, norm_call, F32, ("y",)),
                                             (linear_operands, linear_call, F16, ("x", "w"))])
def test_integers_are_held_as_int8(taken, make, call, dt, at):  # noqa: F811
    def operands():
        t = make(dt, dt)
        for n in at:
            t[n].dtype = torch.int8
        return t

    call(operands(), dt, I8)
    assert len(taken) == 1
    for n in at:
        for wrong in (torch.uint8, torch.float8_e4m3fn, torch.int32, torch.bfloat16):
            t = operands()
            t[n].dtype = wrong
            with pytest.raises(ValueError, match=n):
                call(t, dt, I8)
    assert len(taken) == 1
