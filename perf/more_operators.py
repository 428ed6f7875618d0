"""Cases of the token operators in 8-bit integers and by expert: the norm's output (``cvx_rmsnorm``), the
gated activation (``cvx_gate``), the projection (``cvx_linear``) and the products grouped by expert
(``cvx_linear_grouped``, in 16 and 8 bits).

``run`` computes them in their plain form, or, where ``own`` is true, with the library's
kernels.  ``exact`` gives the same outputs from the definitions in 64 bits.  Codes in 8-bit integers
are whole numbers, so the plain form takes them in 64 bits, as the definitions say.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
MOST = {"e4m3": 448.0, "i8": 127.0}  # the largest value of an 8-bit type


def _norm(name, rows, c, dtype, residual, pad=0):
    """pad: elements between the rows of x and the residual (slices of wider tensors)."""
    return dict(name=name, op="norm", rows=rows, c=c, dtype=dtype, residual=residual, pad=pad)


def _gate(name, rows, c, dtype, out, act="silu", up=True, pad=0):
    """out: "same" as dtype, or 8 bits.  Without `up` the activation alone (none: rows are only brought to 8 bits)."""
    return dict(name=name, op="gate", rows=rows, c=c, dtype=dtype, out=out, act=act, up=up, pad=pad)


def _linear(name, tokens, c_in, c_out, dtype, rank=0, adapters=0, act="none", residual=False, pad=0):
    """adapters: each token draws one of them, or none."""
    return dict(name=name, op="linear", tokens=tokens, c_in=c_in, c_out=c_out, dtype=dtype, rank=rank,
                adapters=adapters, act=act, residual=residual, pad=pad)


def _experts(name, tokens, top, groups, active, c_in, c_out, dtype, held="16", gather=True, weighted=False, act="none",
             skew=0.0, tail=0, pad=0):
    """Each token is in `top` of the `active` experts (of `groups`), every one of which has a row at least;
    skew: how far the experts differ in how many they get.  gather: x holds the tokens, and rows name theirs,
    else x holds the rows.  held: x and w in 16 bits, or in 8.  weighted: a factor of each row.  tail: rows behind the last expert's."""
    return dict(name=name, op="experts", tokens=tokens, top=top, groups=groups, active=active, c_in=c_in, c_out=c_out,
                dtype=dtype, held=held, gather=gather, weighted=weighted, act=act, skew=skew, tail=tail, pad=pad)


def listed():
    return [
        # one new token between two layers, for a projection in 8-bit integers: latency counts
        _norm("norm_token_i8", 1, 4096, "bf16", True),
        # prompts of several thousand tokens
        _norm("norm_prompt_i8", 16384, 4096, "bf16", True),
        # prompts between the two products of a wide layer
        _gate("gate_prompt_i8", 8192, 14336, "bf16", "i8"),
        # odd width, rows that are slices of a wider tensor, 16-bit output
        _gate("gate_odd", 333, 1337, "f16", "same", pad=6),
        # one token: the weights' stream
        _linear("proj_token_i8", 1, 4096, 4096, "bf16"),
        # the tokens that a batch generates at once, wide output
        _linear("proj_batch_i8", 48, 4096, 8192, "bf16", residual=True),
        # a short prompt beside generated tokens, odd sizes, adapters, an activation, slices of wider tensors
        _linear("proj_odd_i8", 333, 1008, 1284, "f16", 8, 5, act="silu", pad=16),
        # the largest: prompts, wide output
        _linear("proj_prompt_i8", 8192, 4096, 14336, "bf16"),
        # one token in 8 of 64 experts: the stream of their weights, and latency
        _experts("experts_token_i8", 1, 8, 64, 8, 2048, 2816, "bf16", "i8"),
        # the tokens that a batch generates at once: a few rows of every expert
        _experts("experts_batch_8bit", 64, 8, 64, 64, 2048, 2816, "bf16", "e4m3", skew=0.3),
        # second products (a factor a row, x by rows), experts without rows, one with most, odd sizes
        _experts("experts_odd", 333, 2, 7, 5, 1000, 1284, "f16", gather=False, weighted=True, act="silu", skew=2.0,
                 tail=13, pad=24),
        # prompts of many requests together
        _experts("experts_prompt", 4096, 8, 64, 64, 2048, 2816, "bf16", skew=0.3),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` in lo..hi, even in its logarithm."""
    if hi <= lo:
        return lo
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return int(min(hi, max(lo, int(v) // step * step)))


def draw(rng):
    kind = rng.random()
    dtype = rng.choice(["bf16", "bf16", "f16"])
    act = rng.choice(["none", "none", "silu", "relu"])
    if kind < 0.15:
        c = _spread(rng, 64, 20480)
        rows = min(_spread(rng, 1, 16384), max(1, 64_000_000 // c))
        case = _norm("", rows, c, rng.choice([dtype, "f32"]), rng.random() < 0.7, rng.choice([0, 0, 8, 5]))
    elif kind < 0.35:
        c = _spread(rng, 64, 20480)
        rows = min(_spread(rng, 1, 32768), max(1, 100_000_000 // c))
        case = _gate("", rows, c, rng.choice([dtype, dtype, "f32"]), rng.choice(["same", "e4m3", "i8", "i8"]),
                     rng.choice(["silu", "silu", "relu", "none"]), rng.random() < 0.8, rng.choice([0, 0, 8, 5]))
    elif kind < 0.65:
        c_in = _spread(rng, 64, 8192, 16)
        c_out = _spread(rng, 64, 16384, 4)
        tokens = min(_spread(rng, 1, 8192), max(1, 400_000_000_000 // (c_in * c_out)))
        rank = rng.choice([0, 0, 0, 8, 16, 32, 64])
        case = _linear("", tokens, c_in, c_out, dtype, rank, rng.randint(1, 8) if rank else 0, act, rng.random() < 0.4,
                       rng.choice([0, 0, 16]))
    else:
        held = rng.choice(["16", "e4m3", "i8"])
        c_in = _spread(rng, 64, 8192, 8 if held == "16" else 16)
        c_out = _spread(rng, 64, 16384, 4)
        groups = min(_spread(rng, 1, 128), max(1, 250_000_000 // (c_in * c_out)))
        active = rng.randint(max(1, groups // 2), groups)
        top = min(rng.choice([1, 2, 4, 8]), active)
        tokens = min(_spread(rng, 1, 8192), max(1, 200_000_000_000 // (c_in * c_out * top)))
        case = _experts("", tokens, top, groups, min(active, tokens * top), c_in, c_out, dtype, held, rng.random() < 0.6,
                        rng.random() < 0.5, act, rng.choice([0.0, 0.3, 1.0]), rng.choice([0, 0, 5, 64]),
                        rng.choice([0, 0, 16]))
    del case["name"]
    return case


def _rows(g, rows, c, pad, scale=1.0):
    """Normal values whose channels differ in size, as a network's activations do, in rows c + pad apart."""
    size = torch.exp(torch.randn(c + pad, generator=g, device=DEV) * 0.5) * scale
    return torch.randn(rows, c + pad, generator=g, device=DEV) * size


def _held(v, kind, dt):
    """Rows of values in 16 bits, or in 8 bits with a scale each (the last axis is the row's)."""
    if kind == "16":
        return v.to(dt), None
    scale = v.abs().amax(-1) / MOST[kind]
    q = v / scale[..., None]
    return (q.to(E4M3) if kind == "e4m3" else q.round().to(torch.int8)), scale


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = DT[case["dtype"]]
    s = dict(case)
    pad = case["pad"]
    if case["op"] == "norm":
        rows, c = case["rows"], case["c"]
        s["x"] = _rows(g, rows, c, pad).to(dt)[:, :c]
        s["res"] = _rows(g, rows, c, pad, 4.0).to(dt)[:, :c] if case["residual"] else None
        s["gamma"] = 1.0 + 0.2 * torch.randn(c, generator=g, device=DEV)
        s["eps"] = 1e-5
        # buffers that a program keeps for its outputs
        s["sum"] = torch.empty(rows, c, dtype=dt, device=DEV) if case["residual"] else None
        s["y"] = torch.empty(rows, c, dtype=torch.int8, device=DEV)
        s["y_scale"] = torch.empty(rows, dtype=torch.float32, device=DEV)
    elif case["op"] == "gate":
        # gate and up are the halves of one product's output
        rows, c = case["rows"], case["c"]
        both = _rows(g, rows, 2 * c, pad).to(dt)
        s["x"] = both[:, :c]
        s["u"] = both[:, c:2 * c] if case["up"] else None
        out8 = case["out"] != "same"
        s["y"] = torch.empty(rows, c, dtype={"same": dt, "e4m3": E4M3, "i8": torch.int8}[case["out"]], device=DEV)
        s["y_scale"] = torch.empty(rows, dtype=torch.float32, device=DEV) if out8 else None
    elif case["op"] == "linear":
        t, ci, co = case["tokens"], case["c_in"], case["c_out"]
        x, s["x_scale"] = _held(_rows(g, t, ci, pad), "i8", dt)
        s["x"] = x[:, :ci]
        s["w"], w_scale = _held(torch.randn(co, ci, generator=g, device=DEV) / math.sqrt(ci), "i8", dt)
        s["scale"] = w_scale
        s["bias"] = 0.1 * torch.randn(co, generator=g, device=DEV)
        s["res"] = _rows(g, t, co, pad).to(dt)[:, :co] if case["residual"] else None
        n, r = case["adapters"], case["rank"]
        s["a"] = s["b"] = s["alpha"] = s["ids"] = None
        if r:
            s["a"] = (torch.randn(n, r, ci, generator=g, device=DEV) / math.sqrt(ci)).to(dt)
            s["b"] = (0.3 * torch.randn(n, co, r, generator=g, device=DEV) / math.sqrt(r)).to(dt)
            s["alpha"] = 0.5 + torch.rand(n, generator=g, device=DEV)
            s["ids"] = torch.randint(-1, n, (t,), generator=g, device=DEV).to(torch.int32)
        s["y"] = torch.empty(t, co, dtype=dt, device=DEV)
    else:
        t, top, n, ci, co = case["tokens"], case["top"], case["groups"], case["c_in"], case["c_out"]
        rows = t * top
        # the experts that tokens go to, and each token's: by a score, the first tokens' in turn so that each has a row
        at = torch.randperm(n, generator=g, device=DEV)[:case["active"]].sort()[0]
        likes = case["skew"] * torch.randn(case["active"], generator=g, device=DEV)
        score = torch.randn(t, case["active"], generator=g, device=DEV) + likes
        pick = score.topk(top, dim=1)[1].reshape(-1)
        first = min(rows, -(-case["active"] // top) * top)
        pick[:first] = torch.arange(first, device=DEV) % case["active"]
        expert, order = at[pick].sort(stable=True)
        size = torch.bincount(expert, minlength=n)
        s["offset"] = torch.cat([size.new_zeros(1), size.cumsum(0)]).to(torch.int32)
        s["row_id"] = (order // top).to(torch.int32) if case["gather"] else None
        s["most"], s["live"] = int(size.max()), at  # a host that sorts the rows knows both
        s["rows"] = rows + case["tail"]
        x, s["x_scale"] = _held(_rows(g, t if case["gather"] else s["rows"], ci, pad), case["held"], dt)
        s["x"] = x[:, :ci]
        if case["gather"] and case["tail"]:
            s["row_id"] = torch.cat([s["row_id"], s["row_id"].new_zeros(case["tail"])])
        s["w"], s["scale"] = _held(torch.randn(n, co, ci, generator=g, device=DEV) / math.sqrt(ci), case["held"], dt)
        s["bias"] = 0.1 * torch.randn(n, co, generator=g, device=DEV)
        s["weight"] = torch.rand(s["rows"], generator=g, device=DEV) if case["weighted"] else None
        s["y"] = torch.ones(s["rows"], co, dtype=dt, device=DEV)  # a program's buffer; the tail stays as it is
    return s


def _act(z, act):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return torch.clamp_min(z, 0.0) if act == "relu" else z


def _codes(u, kind):
    """Rows u in 8 bits, and the largest magnitude of each."""
    top = u.abs().amax(1)
    v = u * torch.where(top > 0, MOST[kind] / top, 0.0)[:, None]
    return (v.to(E4M3) if kind == "e4m3" else torch.round(v).to(torch.int8)), top


def _plain_norm(s):
    h = s["x"].float()
    if s["res"] is not None:
        h = h.double() + s["res"].double() if s["dtype"] == "f32" else h + s["res"].float()
    h = h.double()
    q = 1.0 / torch.sqrt((h * h).mean(1) + s["eps"])
    y, top = _codes(h * s["gamma"].double(), "i8")
    out = {"y": y, "y_scale": (top * q / 127.0).float()}
    if s["res"] is not None:
        out["sum"] = h.to(s["x"].dtype)
    return out


def _plain_gate(s):
    f = torch.float64 if s["out"] == "i8" else torch.float32
    u = _act(s["x"].to(f), s["act"])
    if s["u"] is not None:
        u = u * s["u"].to(f)
    if s["out"] == "same":
        return {"y": u.to(s["x"].dtype)}
    y, top = _codes(u, s["out"])
    return {"y": y, "y_scale": (top / MOST[s["out"]]).float()}


def _plain_linear(s):
    x = s["x"].float()
    z = (x @ s["w"].float().t()) * s["scale"] * s["x_scale"][:, None] + s["bias"]
    if s["rank"]:
        n, r = s["adapters"], s["rank"]
        v = (x @ s["a"].float().reshape(n * r, -1).t()) * s["x_scale"][:, None]
        # every adapter's low-rank values, those of other tokens' adapters taken as zero
        mine = s["ids"][:, None] == torch.arange(n, device=DEV)[None, :]
        v = v.reshape(-1, n, r) * torch.where(mine, s["alpha"][None, :], 0.0)[:, :, None]
        z = z + v.reshape(-1, n * r) @ s["b"].float().permute(0, 2, 1).reshape(n * r, -1)
    z = _act(z, s["act"])
    if s["res"] is not None:
        z = z + s["res"].float()
    return {"y": z.to(DT[s["dtype"]])}


def _plain_experts(s):
    # the rows of the experts that have any side by side, filled up to the most that one has, and one product of all
    offset = s["offset"].long()
    rows = s["tokens"] * s["top"]
    i = torch.arange(rows, device=DEV)
    g = torch.searchsorted(offset, i, right=True) - 1
    place = torch.searchsorted(s["live"], g) * s["most"] + i - offset[g]
    j = s["row_id"][:rows].long() if s["gather"] else i
    x = torch.zeros(s["active"] * s["most"], s["c_in"], device=DEV)
    x[place] = s["x"][j].float()
    w = (s["w"][s["live"]] if s["active"] < s["groups"] else s["w"]).float()
    z = torch.bmm(x.view(s["active"], s["most"], -1), w.transpose(1, 2)).view(-1, s["c_out"])[place]
    if s["held"] != "16":
        z = z * s["scale"][g] * s["x_scale"][j][:, None]
    z = _act(z + s["bias"][g], s["act"])
    if s["weight"] is not None:
        z = z * s["weight"][:rows, None]
    s["y"][:rows] = z.to(s["y"].dtype)
    return {"y": s["y"]}


def _call(s):
    """Binds a call to the state's buffers; the descriptor and the workspace are made once, as a program does for a
    layer and a number of tokens."""
    from conv2d_batchnorm_activation_amd import cvx
    dt = {"f32": cvx.CVX_DT_F32, "f16": cvx.CVX_DT_F16, "bf16": cvx.CVX_DT_BF16}[s["dtype"]]
    act = {"none": cvx.CVX_ACT_NONE, "relu": cvx.CVX_ACT_RELU, "silu": cvx.CVX_ACT_SILU}[s.get("act", "none")]
    stride = lambda t: 0 if t is None else t.stride(0)  # noqa: E731
    if s["op"] == "norm":
        d = cvx.make_rmsnorm_desc(s["rows"], s["c"], dt, cvx.CVX_DT_I8, s["eps"], stride(s["x"]), stride(s["res"]))
        return lambda: cvx.cvx_rmsnorm(d, s["x"], s["res"], s["gamma"], s["sum"], s["y"], s["y_scale"])
    if s["op"] == "gate":
        out = {"same": dt, "e4m3": cvx.CVX_DT_E4M3, "i8": cvx.CVX_DT_I8}[s["out"]]
        d = cvx.make_gate_desc(s["rows"], s["c"], dt, out, act, stride(s["x"]), stride(s["u"]))
        return lambda: cvx.cvx_gate(d, s["x"], s["u"], s["y"], s["y_scale"])
    if s["op"] == "linear":
        d = cvx.make_linear_desc(s["tokens"], s["c_in"], s["c_out"], dt, cvx.CVX_DT_I8, act,
                                 cvx.CVX_RES_AFTER_ACT if s["residual"] else cvx.CVX_RES_NONE, s["rank"], s["adapters"],
                                 x_stride=stride(s["x"]), res_stride=stride(s["res"]))
        ws = torch.empty(max(16, cvx.cvx_linear_workspace_bytes(d)), dtype=torch.uint8, device=DEV)
        return lambda: cvx.cvx_linear(d, s["x"], s["w"], s["y"], s["x_scale"], s["scale"], s["bias"], s["res"], s["a"],
                                      s["b"], s["alpha"], s["ids"], ws)
    xdt = {"16": dt, "e4m3": cvx.CVX_DT_E4M3, "i8": cvx.CVX_DT_I8}[s["held"]]
    d = cvx.make_grouped_desc(s["rows"], s["x"].shape[0], s["groups"], s["c_in"], s["c_out"], dt, xdt, act,
                              x_stride=stride(s["x"]))
    return lambda: cvx.cvx_linear_grouped(d, s["x"], s["w"], s["offset"], s["y"], s["x_scale"], s["scale"], s["bias"],
                                          s["row_id"], s["weight"])


def run(s):
    if own:
        if "call" not in s:
            s["call"] = _call(s)
        s["call"]()
        return {k: s[k] for k in ("y", "y_scale", "sum") if s.get(k) is not None}
    return {"norm": _plain_norm, "gate": _plain_gate, "linear": _plain_linear, "experts": _plain_experts}[s["op"]](s)


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        n = case["rows"] * case["c"]
        return {"bytes": n * (e * (3 if case["residual"] else 1) + 1) + 4 * (case["c"] + case["rows"]), "flops": 6 * n}
    if case["op"] == "gate":
        n = case["rows"] * case["c"]
        out8 = case["out"] != "same"
        return {"bytes": n * (e * (2 if case["up"] else 1) + (1 if out8 else e)) + (4 * case["rows"] if out8 else 0),
                "flops": 8 * n}
    ci, co, t = case["c_in"], case["c_out"], case["tokens"]
    if case["op"] == "linear":
        r = case["rank"]
        used = min(case["adapters"], t) if r else 0
        nbytes = t * ci + co * ci + 2 * t * co * (2 if case["residual"] else 1) + 8 * co + 4 * t * (2 if r else 1)
        return {"bytes": nbytes + 2 * used * r * (ci + co), "flops": 2 * t * ci * co + 2 * t * r * (ci + co)}
    rows = t * case["top"]
    ex = 2 if case["held"] == "16" else 1
    nbytes = ex * ci * (t if case["gather"] else rows) + case["active"] * co * (ex * ci + (8 if ex == 1 else 4))
    nbytes += 2 * rows * co + 4 * (case["groups"] + 1) + 4 * rows * (case["gather"] + case["weighted"])
    return {"bytes": nbytes + (4 * t if ex == 1 else 0), "flops": 2 * rows * ci * co}


def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] in ("norm", "gate"):
        v = s["x"].to(f)
        if case["op"] == "norm":
            if case["residual"]:
                v = v + s["res"].to(f)
            out = {"sum": v} if case["residual"] else {}
            size = torch.linalg.vector_norm(v, dim=1, keepdim=True) ** 2 / case["c"]
            v = v * torch.rsqrt(size + s["eps"]) * s["gamma"].to(f)
            kind = "i8"
        else:
            out, kind = {}, case["out"]
            v = v * torch.sigmoid(v) if case["act"] == "silu" else torch.relu(v) if case["act"] == "relu" else v
            if case["up"]:
                v = v * s["u"].to(f)
        if kind == "same":
            return {"y": v}
        out["y_scale"] = v.abs().amax(1) / MOST[kind]
        if kind == "i8":
            out["y"] = None  # whole numbers, which are compared with the plain form's
        else:
            # the e4m3 grid: 3 fraction bits, exponents down to -6, ties to even
            v = v / torch.where(out["y_scale"] > 0, out["y_scale"], 1.0)[:, None]
            step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
            out["y"] = torch.round(v / step) * step
        return out

    def activated(z):
        return z * torch.sigmoid(z) if case["act"] == "silu" else torch.relu(z) if case["act"] == "relu" else z

    if case["op"] == "experts":
        out = torch.ones(s["rows"], case["c_out"], dtype=f, device=DEV)
        ends = s["offset"].tolist()
        for d in range(case["groups"]):
            a, b = ends[d], ends[d + 1]
            if a == b:
                continue
            at = s["row_id"][a:b].long() if case["gather"] else torch.arange(a, b, device=DEV)
            x, w = s["x"][at].to(f), s["w"][d].to(f)
            if case["held"] != "16":
                x, w = x * s["x_scale"][at].to(f)[:, None], w * s["scale"][d].to(f)[:, None]
            z = activated(torch.addmm(s["bias"][d].to(f), x, w.t()))
            out[a:b] = z * s["weight"][a:b].to(f)[:, None] if case["weighted"] else z
        return {"y": out}
    out = torch.empty(case["tokens"], case["c_out"], dtype=f, device=DEV)
    w = s["w"].to(f) * s["scale"].to(f)[:, None]
    for t0 in range(0, case["tokens"], 1024):
        t1 = min(t0 + 1024, case["tokens"])
        x = s["x"][t0:t1].to(f) * s["x_scale"][t0:t1].to(f)[:, None]
        z = torch.addmm(s["bias"].to(f), x, w.t())
        if case["rank"]:
            ids = s["ids"][t0:t1]
            for d in range(case["adapters"]):
                at = (ids == d).nonzero()[:, 0]
                if at.numel():
                    z[at] += s["alpha"][d].to(f) * ((x[at] @ s["a"][d].to(f).t()) @ s["b"][d].to(f).t())
        z = activated(z)
        out[t0:t1] = z + s["res"][t0:t1].to(f) if case["residual"] else z
    return {"y": out}
