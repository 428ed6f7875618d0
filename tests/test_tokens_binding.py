"""What the binding takes and refuses for the operators on tokens before any call is
made with it.  Host only: tensors are stand-ins that answer what the binding asks."""
import enum

import pytest

from conv2d_batchnorm_activation_amd import cvx

BF16 = cvx.CVX_DT_BF16


class At(enum.IntEnum):
    """Addresses by name: a subclass of int."""
    X = 0x100000000
    W = 0x200000000
    S = 0x300000000
    B = 0x400000000
    Y = 0x500000000


def test_addresses_of_a_subclass_of_int():
    # the calls get as far as the library, which refuses the output over the input
    with pytest.raises(cvx.CvxError) as e:
        cvx.cvx_conv_bn_act(cvx.make_desc(1, 8, 8, 8, 8, 1, 1, 0), At.X, At.W, At.S, At.B, None, At.X)
    assert e.value.status == -5
    with pytest.raises(cvx.CvxError) as e:
        cvx.cvx_rmsnorm(cvx.make_rmsnorm_desc(2, 8, BF16), At.X, None, At.W, None, At.X)
    assert e.value.status == -5
    with pytest.raises(cvx.CvxError) as e:
        cvx.cvx_linear(cvx.make_linear_desc(2, 8, 8, BF16), At.X, At.W, At.X)
    assert e.value.status == -5
