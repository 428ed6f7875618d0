"""Cases of the token operators: the root-mean-square norm with the residual's addition
(``cvx_rmsnorm``) and the projection with low-rank adapters (``cvx_linear``).

``run`` computes them in their plain form, or, where ``own`` is true, with the library's
kernels.  ``exact`` gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0


def _norm(name, rows, c, dtype, residual, out8, pad=0):
    """pad: elements between the rows of x and the residual (slices of wider tensors)."""
    return dict(name=name, op="norm", rows=rows, c=c, dtype=dtype, residual=residual, out8=out8, pad=pad)


def _linear(name, tokens, c_in, c_out, dtype, x8, rank, adapters, requests, act="none", residual=False, pad=0):
    """requests: tokens come in that many runs of one adapter each (0: an adapter drawn for every
    token, as when every sequence of a batch generates its next token)."""
    return dict(name=name, op="linear", tokens=tokens, c_in=c_in, c_out=c_out, dtype=dtype, x8=x8, rank=rank,
                adapters=adapters, requests=requests, act=act, residual=residual, pad=pad)


def listed():
    return [
        # one new token between two layers, its norm going into an 8-bit projection: latency counts
        _norm("norm_token_8bit", 1, 4096, "bf16", True, True),
        # the tokens that a batch generates at once, 16-bit output
        _norm("norm_batch", 96, 8192, "f16", True, False),
        # prompts of several thousand tokens, for an 8-bit projection
        _norm("norm_prompt_8bit", 16384, 4096, "bf16", True, True),
        # odd width, rows that are slices of a wider tensor, no residual: rows start misaligned
        _norm("norm_odd", 2057, 1337, "bf16", False, False, pad=6),
        # fp32 storage and a long row
        _norm("norm_f32_long", 517, 20480, "f32", True, False),
        # one token of one request: the weights' stream
        _linear("proj_token", 1, 4096, 4096, "bf16", False, 16, 8, 0),
        # a batch of generated tokens, each with its own request's adapter, wide output
        _linear("proj_batch", 48, 4096, 8192, "bf16", False, 32, 32, 0, residual=True),
        # the same in 8 bits
        _linear("proj_batch_8bit", 16, 8192, 8192, "bf16", True, 16, 16, 0),
        # a short prompt beside generated tokens, odd sizes, an activation, slices of wider tensors
        _linear("proj_odd", 333, 1000, 1284, "f16", False, 8, 5, 9, act="silu", pad=24),
        # a few hundred tokens: neither the weights' stream nor the matrix cores alone
        _linear("proj_mid", 512, 4096, 4096, "bf16", False, 16, 8, 6, residual=True),
        # prompts of many requests together
        _linear("proj_prompt", 4096, 4096, 4096, "bf16", False, 16, 9, 23),
        # the largest: prompts in 8 bits, wide output, higher rank
        _linear("proj_prompt_8bit", 8192, 4096, 14336, "bf16", True, 64, 12, 31),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` in lo..hi, even in its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return int(min(hi, max(lo, int(v) // step * step)))


def draw(rng):
    if rng.random() < 0.4:
        c = _spread(rng, 64, 20480)
        rows = min(_spread(rng, 1, 16384), max(1, 64_000_000 // c))
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        case = _norm("", rows, c, dtype, rng.random() < 0.7, rng.random() < 0.5, rng.choice([0, 0, 8, 5]))
    else:
        x8 = rng.random() < 0.4
        c_in = _spread(rng, 64, 8192, 16 if x8 else 8)
        c_out = _spread(rng, 64, 16384, 4)
        tokens = min(_spread(rng, 1, 8192), max(1, 400_000_000_000 // (c_in * c_out)))
        requests = 0 if tokens <= 64 else rng.randint(1, min(tokens, 40))
        rank = rng.choice([0, 8, 16, 16, 24, 32, 64])
        case = _linear("", tokens, c_in, c_out, rng.choice(["bf16", "bf16", "f16"]), x8, rank, rng.randint(1, 32),
                       requests, rng.choice(["none", "none", "silu", "relu"]), rng.random() < 0.4,
                       rng.choice([0, 0, 16]))
    del case["name"]
    return case


def _rows(g, rows, c, pad, scale=1.0):
    """Normal values whose channels differ in size, as a network's activations do, in rows c + pad apart."""
    size = torch.exp(torch.randn(c + pad, generator=g, device=DEV) * 0.5) * scale
    return torch.randn(rows, c + pad, generator=g, device=DEV) * size


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = DT[case["dtype"]]
    s = dict(case)
    if case["op"] == "norm":
        rows, c = case["rows"], case["c"]
        s["x"] = _rows(g, rows, c, case["pad"]).to(dt)[:, :c]
        s["res"] = _rows(g, rows, c, case["pad"], 4.0).to(dt)[:, :c] if case["residual"] else None
        s["gamma"] = 1.0 + 0.2 * torch.randn(c, generator=g, device=DEV)
        s["eps"] = 1e-5
        # buffers that a program keeps for its outputs
        s["sum"] = torch.empty(rows, c, dtype=dt, device=DEV) if case["residual"] else None
        s["y"] = torch.empty(rows, c, dtype=E4M3 if case["out8"] else dt, device=DEV)
        s["y_scale"] = torch.empty(rows, dtype=torch.float32, device=DEV) if case["out8"] else None
    else:
        t, ci, co, pad = case["tokens"], case["c_in"], case["c_out"], case["pad"]
        x = _rows(g, t, ci, pad)
        w = torch.randn(co, ci, generator=g, device=DEV) / math.sqrt(ci)
        scale = 1.0 + 0.1 * torch.randn(co, generator=g, device=DEV)
        if case["x8"]:
            s["x_scale"] = x.abs().amax(1) / E4M3_MAX
            s["x"] = (x / s["x_scale"][:, None]).to(E4M3)[:, :ci]
            w_scale = w.abs().amax(1) / E4M3_MAX
            s["w"] = (w / w_scale[:, None]).to(E4M3)
            scale = scale * w_scale
        else:
            s["x_scale"] = None
            s["x"] = x.to(dt)[:, :ci]
            s["w"] = w.to(dt)
        s["scale"] = scale
        s["bias"] = 0.1 * torch.randn(co, generator=g, device=DEV)
        s["res"] = _rows(g, t, co, pad).to(dt)[:, :co] if case["residual"] else None
        n, r = case["adapters"], case["rank"]
        s["a"] = s["b"] = s["alpha"] = s["ids"] = None
        if r:
            s["a"] = (torch.randn(n, r, ci, generator=g, device=DEV) / math.sqrt(ci)).to(dt)
            s["b"] = (0.3 * torch.randn(n, co, r, generator=g, device=DEV) / math.sqrt(r)).to(dt)
            s["alpha"] = 0.5 + torch.rand(n, generator=g, device=DEV)
            if case["requests"]:
                ids = torch.randint(-1, n, (case["requests"],), generator=g, device=DEV)
                cuts = torch.randint(0, t, (case["requests"] - 1,), generator=g, device=DEV)
                s["ids"] = ids[(torch.arange(t, device=DEV)[:, None] >= cuts[None, :]).sum(1)].to(torch.int32)
            else:
                s["ids"] = torch.randint(-1 if t > 1 else 0, n, (t,), generator=g, device=DEV).to(torch.int32)
        s["y"] = torch.empty(t, co, dtype=dt, device=DEV)
    if own:
        # descriptor and workspace, which a program makes once for a layer and a number of tokens
        from conv2d_batchnorm_activation_amd import cvx
        code = {"f32": cvx.CVX_DT_F32, "f16": cvx.CVX_DT_F16, "bf16": cvx.CVX_DT_BF16}[case["dtype"]]
        res_stride = s["res"].stride(0) if s["res"] is not None else 0
        if case["op"] == "norm":
            s["desc"] = cvx.make_rmsnorm_desc(case["rows"], case["c"], code, cvx.CVX_DT_E4M3 if case["out8"] else code,
                                              s["eps"], x_stride=s["x"].stride(0), res_stride=res_stride)
        else:
            act = {"none": cvx.CVX_ACT_NONE, "relu": cvx.CVX_ACT_RELU, "silu": cvx.CVX_ACT_SILU}[case["act"]]
            s["desc"] = cvx.make_linear_desc(case["tokens"], case["c_in"], case["c_out"], code,
                                             cvx.CVX_DT_E4M3 if case["x8"] else code, act,
                                             cvx.CVX_RES_AFTER_ACT if case["residual"] else cvx.CVX_RES_NONE,
                                             case["rank"], case["adapters"] if case["rank"] else 0,
                                             x_stride=s["x"].stride(0), res_stride=res_stride)
            s["ws"] = torch.empty(max(16, cvx.cvx_linear_workspace_bytes(s["desc"])), dtype=torch.uint8, device=DEV)
        s["cvx"] = cvx
    return s


def _plain_norm(s):
    h = s["x"].float()
    if s["res"] is not None:
        h = h + s["res"].float()
    q = 1.0 / torch.sqrt((h * h).mean(1) + s["eps"])
    u = h * s["gamma"]
    out = {}
    if s["out8"]:
        top = u.abs().amax(1)
        out["y"] = (u * torch.where(top > 0, E4M3_MAX / top, 0.0)[:, None]).to(E4M3)
        out["y_scale"] = top * q / E4M3_MAX
    else:
        out["y"] = (u * q[:, None]).to(s["x"].dtype)
    if s["res"] is not None:
        out["sum"] = h.to(s["x"].dtype)
    return out


def _plain_linear(s):
    x = s["x"].float()
    z = (x @ s["w"].float().t()) * s["scale"]
    if s["x8"]:
        z = z * s["x_scale"][:, None]
    z = z + s["bias"]
    if s["rank"]:
        n, r = s["adapters"], s["rank"]
        v = x @ s["a"].float().reshape(n * r, -1).t()
        if s["x8"]:
            v = v * s["x_scale"][:, None]
        # every adapter's low-rank values, those of other requests' adapters taken as zero
        mine = s["ids"][:, None] == torch.arange(n, device=DEV)[None, :]
        v = v.reshape(-1, n, r) * torch.where(mine, s["alpha"][None, :], 0.0)[:, :, None]
        z = z + v.reshape(-1, n * r) @ s["b"].float().permute(0, 2, 1).reshape(n * r, -1)
    if s["act"] == "silu":
        z = z / (1.0 + torch.exp(-z))
    elif s["act"] == "relu":
        z = torch.clamp_min(z, 0.0)
    if s["res"] is not None:
        z = z + s["res"].float()
    return {"y": z.to(DT[s["dtype"]])}


def run(s):
    if own:
        cvx = s["cvx"]
        if s["op"] == "norm":
            cvx.cvx_rmsnorm(s["desc"], s["x"], s["res"], s["gamma"], s["sum"], s["y"], s["y_scale"])
            return {k: s[k] for k in ("y", "y_scale", "sum") if s[k] is not None}
        cvx.cvx_linear(s["desc"], s["x"], s["w"], s["y"], s["x_scale"], s["scale"], s["bias"], s["res"], s["a"],
                       s["b"], s["alpha"], s["ids"], s["ws"])
        return {"y": s["y"]}
    return _plain_norm(s) if s["op"] == "norm" else _plain_linear(s)


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        n = case["rows"] * case["c"]
        per = e * (3 if case["residual"] else 1) + (1 if case["out8"] else e)
        return {"bytes": n * per + 4 * case["c"] + (4 * case["rows"] if case["out8"] else 0), "flops": 6 * n}
    t, ci, co, r = case["tokens"], case["c_in"], case["c_out"], case["rank"]
    ex = 1 if case["x8"] else 2
    runs = case["requests"] or t
    used = min(case["adapters"], runs) if r else 0
    nbytes = ex * (t * ci + co * ci) + 2 * t * co * (2 if case["residual"] else 1) + 8 * co
    nbytes += 4 * t * ((1 if case["x8"] else 0) + (1 if r else 0)) + 2 * used * r * (ci + co)
    return {"bytes": nbytes, "flops": 2 * t * ci * co + 2 * t * r * (ci + co)}


def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] == "norm":
        h = s["x"].to(f)
        if case["residual"]:
            h = h + s["res"].to(f)
        inv = torch.rsqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / case["c"] + s["eps"])
        y = h * inv * s["gamma"].to(f)
        out = {"y": y, "sum": h} if case["residual"] else {"y": y}
        if case["out8"]:
            # the e4m3 grid: 3 fraction bits, exponents down to -6, ties to even
            out["y_scale"] = y.abs().amax(1) / E4M3_MAX
            v = y / out["y_scale"][:, None]
            step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
            out["y"] = torch.round(v / step) * step
        return out
    out = torch.empty(case["tokens"], case["c_out"], dtype=f, device=DEV)
    w = s["w"].to(f) * s["scale"].to(f)[:, None]
    for t0 in range(0, case["tokens"], 1024):
        t1 = min(t0 + 1024, case["tokens"])
        x = s["x"][t0:t1].to(f)
        if case["x8"]:
            x = x * s["x_scale"][t0:t1].to(f)[:, None]
        z = torch.addmm(s["bias"].to(f), x, w.t())
        if case["rank"]:
            ids = s["ids"][t0:t1]
            for d in range(case["adapters"]):
                at = (ids == d).nonzero()[:, 0]
                if at.numel():
                    v = x[at] @ s["a"][d].to(f).t()
                    z[at] += s["alpha"][d].to(f) * (v @ s["b"][d].to(f).t())
        if case["act"] == "silu":
            z = z * torch.sigmoid(z)
        elif case["act"] == "relu":
            z = torch.relu(z)
        out[t0:t1] = z + s["res"][t0:t1].to(f) if case["residual"] else z
    return {"y": out}
