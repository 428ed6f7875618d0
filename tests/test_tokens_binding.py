"""What the binding takes and refuses for the operators on tokens before any call is
made with it.  Host only: tensors are stand-ins that answer what the binding asks."""
import enum

import pytest
import torch

from conv2d_batchnorm_activation_amd import cvx

F32, F16, BF16, E4M3 = cvx.CVX_DT_F32, cvx.CVX_DT_F16, cvx.CVX_DT_BF16, cvx.CVX_DT_E4M3


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


class On:
    """A tensor as the binding sees it: its GPU, its element type, its address."""
    is_cuda = True

    def __init__(self, dtype, device=0, at=0x100000000):
        self.dtype, self.device, self.at = dtype, device, at

    def get_device(self):
        return self.device

    def data_ptr(self):
        return self.at


HELD = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16, E4M3: torch.float8_e4m3fn}
NORM = ("x", "residual", "gamma", "sum_out", "y", "y_scale")
LINEAR = ("x", "w", "y", "x_scale", "scale", "bias", "residual", "lora_a", "lora_b", "lora_alpha", "lora_id",
          "workspace")


def norm_operands(dt, out, device=0):
    t = {n: On(HELD[dt], device, (i + 1) << 32) for i, n in enumerate(NORM)}
    t["gamma"].dtype = t["y_scale"].dtype = torch.float32
    t["y"].dtype = HELD[out]
    return t


def linear_operands(dt, xdt, device=0):
    t = {n: On(HELD[dt], device, (i + 1) << 32) for i, n in enumerate(LINEAR)}
    t["x"].dtype = t["w"].dtype = HELD[xdt]
    for n in ("x_scale", "scale", "bias", "lora_alpha"):
        t[n].dtype = torch.float32
    t["lora_id"].dtype = torch.int32
    t["workspace"].dtype = torch.uint8
    return t


@pytest.fixture
def taken(monkeypatch):
    """The calls the library is given, in place of it; the current GPU is 0."""
    calls = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: calls.append((name, a)) or 0

    monkeypatch.setattr(cvx, "lib", Lib())
    monkeypatch.setattr(cvx, "_stream", lambda s: s)
    monkeypatch.setattr(cvx, "_raw_stream", lambda d: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return calls


def norm_call(t, dt, out):
    cvx.cvx_rmsnorm(cvx.make_rmsnorm_desc(2, 32, dt, out), *(t[n] for n in NORM))


def linear_call(t, dt, xdt):
    cvx.cvx_linear(cvx.make_linear_desc(2, 32, 32, dt, xdt, res_mode=1, rank=8, n_adapters=2),
                   *(t[n] for n in LINEAR), 1 << 20)


CALLS = [(norm_operands, norm_call, F32, F32), (norm_operands, norm_call, F16, F16), (norm_operands, norm_call, BF16, E4M3),
         (linear_operands, linear_call, F16, F16), (linear_operands, linear_call, BF16, BF16),
         (linear_operands, linear_call, BF16, E4M3)]


@pytest.mark.parametrize("make,call,dt,other", CALLS)
def test_operands_on_one_gpu_and_of_the_descriptor_s_types(taken, make, call, dt, other):
    t = make(dt, other)
    call(t, dt, other)
    assert len(taken) == 1 and {t[n].at for n in t} <= set(taken[0][1])
    for n in t:
        if t[n].dtype == torch.float8_e4m3fn:  # codes held as bytes
            t[n].dtype = torch.uint8
    call(t, dt, other)
    t["x"] = t["x"].at  # with an address the current GPU is the input's
    call(t, dt, other)
    assert len(taken) == 3


@pytest.mark.parametrize("make,call,dt,other", CALLS)
def test_operands_on_another_gpu_are_refused(taken, make, call, dt, other):
    for n in make(dt, other):
        for address in (False, True):
            t = make(dt, other)
            if address and n != "x":
                t["x"] = t["x"].at
            if n == "x":
                t["x"].device = -1
            else:
                t[n].device = 1
            with pytest.raises(ValueError, match=n):
                call(t, dt, other)
    assert not taken


@pytest.mark.parametrize("make,call,dt,other", CALLS)
def test_operands_of_other_types_are_refused(taken, make, call, dt, other):
    for n in make(dt, other):
        if n == "workspace":
            continue
        for wrong in (torch.int64, torch.float64, torch.float8_e4m3fnuz, torch.float16, torch.bfloat16, torch.float32):
            t = make(dt, other)
            if t[n].dtype == wrong:
                continue
            t[n].dtype = wrong
            with pytest.raises(ValueError, match=n):
                call(t, dt, other)
    assert not taken


def test_an_input_on_another_gpu_is_made_current(taken, monkeypatch):
    now = [0]

    class Device:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            self.was, now[0] = now[0], self.d

        def __exit__(self, *_):
            now[0] = self.was

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    norm_call(norm_operands(F16, F16, 1), F16, F16)
    linear_call(linear_operands(F16, F16, 1), F16, F16)
    assert len(taken) == 2 and now == [0]


def tiles(d):
    """(workgroups, threads of one) of the projection's launch for a descriptor."""
    plan = cvx.cvx_linear_plan(d)
    kind, size = plan.split()[1:3]
    bm, bn = map(int, size.split("x"))
    n = -(-d.c_out // bm) * -(-d.tokens // bn)
    return n, 512 if kind == "few" or bm == 256 else 256


@pytest.mark.parametrize("tokens,c_out", [(1 << 24, 1 << 20), (1 << 24, (1 << 13) + 4), ((1 << 17) + 1, 1 << 20)])
def test_more_outputs_than_a_launch_takes(tokens, c_out):
    # refused as a size, before the adapters' first product is enqueued
    at = [(i + 1) << 50 for i in range(12)]
    for rank in (0, 16):
        d = cvx.make_linear_desc(tokens, 64, c_out, BF16, rank=rank, n_adapters=3 if rank else 0)
        with pytest.raises(cvx.CvxError) as e:
            cvx.cvx_linear(d, at[0], at[1], at[2], lora_a=at[3], lora_b=at[4], lora_id=at[5], workspace=at[6],
                           ws_bytes=1 << 49)
        assert e.value.status == -2
        assert cvx.cvx_linear_workspace_bytes(d) == 0
        with pytest.raises(cvx.CvxError):
            cvx.cvx_linear_plan(d)


def test_the_most_outputs_are_one_launch():
    for c_in in (8, 64, 4096, 1 << 20):
        for t in range(25):
            for tokens in {1 << t, (1 << t) - 1, (1 << t) + 1, (1 << t) * 5 // 4 + 1}:
                if not 1 <= tokens <= 1 << 24:
                    continue
                for c_out in {min(1 << 20, (1 << 37) // tokens) // 4 * 4, 4, 260, 516, 4100}:
                    if tokens * c_out > 1 << 37 or tokens * c_in > 1 << 40:  # (no operand spans more)
                        continue
                    n, threads = tiles(cvx.make_linear_desc(tokens, c_in, c_out, BF16))
                    assert n * threads < 1 << 32, (tokens, c_in, c_out)
