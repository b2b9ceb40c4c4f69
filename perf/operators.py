"""The cases that the feed-forward and normalisation operators are measured on.

Three operators of a transformer block, each in both directions:

  linear  y = act(x W^T + b) + r, and its gradients (dx, dW, db; dr is dy itself);
  gated   a = act(x Wg^T + bg) * (x Wu^T + bu), and its gradients;
  norm    s = alpha x + gate * p, p = y or post_gain * rms(y); h = rms(s) * gain * (1 + scale) + shift,
          and its gradients; gate, scale and shift are one vector per group of rows (a sample).

With `own` false `run` computes them by elementary torch operations in 32 bits; with `own` true it
calls this repository's operators on the same state.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}
ACTS = ("none", "relu", "silu", "gelu_tanh", "gelu_erf")
GATES = ("silu", "gelu_tanh", "gelu_erf", "relu", "sigmoid")


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # One token through a feed-forward up-projection (1536 -> 6144): the smallest serving call, weights alone count.
        dict(name="linear one token", op="linear", dtype="bf16", out="bf16", act="gelu_tanh", M=1, N=6144, K=1536, res=False, save=False),
        # The 16 action tokens of the joint model through the down-projection, added to the 32-bit residual stream.
        dict(name="linear 16 tokens down", op="linear", dtype="bf16", out="fp32", act="none", M=16, N=1536, K=6144, res=True, save=False),
        # The 64 + 1024 video tokens of one sample through the down-projection with its residual.
        dict(name="linear video down", op="linear", dtype="bf16", out="fp32", act="none", M=1088, N=1536, K=6144, res=True, save=False),
        # A training step's backward pass at ragged sizes: rows and features that no tile divides.
        dict(name="linear backward ragged", op="linear_bwd", dtype="bf16", out="bf16", act="gelu_tanh", M=2049, N=4111, K=1544),
        # One token through a gated feed-forward.
        dict(name="gated one token", op="gated", dtype="bf16", act="silu", M=1, F=4096, K=1536, bias=False, save=False),
        # The video tokens of one sample, with the pre-activations that a backward pass needs.
        dict(name="gated video train", op="gated", dtype="bf16", act="silu", M=1088, F=6144, K=1536, bias=True, save=True),
        # The batch of 8 samples with 2048 + 64 tokens: the largest forward call.
        dict(name="gated batch", op="gated", dtype="bf16", act="gelu_tanh", M=16896, F=6144, K=1536, bias=False, save=False),
        # A training step's backward pass over four such samples.
        dict(name="gated backward", op="gated_bwd", dtype="bf16", act="silu", M=8448, F=4096, K=1536, bias=True),
        # The debug precision, backward, at odd sizes.
        dict(name="gated backward fp32", op="gated_bwd", dtype="fp32", act="silu", M=264, F=777, K=321, bias=True),
        # One token between two blocks of the action expert.
        dict(name="norm one token", op="norm", dtype="bf16", res="fp32", M=1, G=1, D=768, post=True, gate=True, mod=True, gain=True),
        # The batch of 8 samples with their own modulation vectors.
        dict(name="norm batch", op="norm", dtype="bf16", res="fp32", M=16896, G=8, D=1536, post=True, gate=True, mod=True, gain=False),
        # The backward pass of a batch with a residual stream in bf16 and an odd width.
        dict(name="norm backward", op="norm_bwd", dtype="bf16", res="bf16", M=8448, G=4, D=1537, post=True, gate=True, mod=True, gain=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "linear_bwd", "gated", "gated_bwd", "norm", "norm_bwd"))
    dtype = "fp32" if rng.random() < 0.2 else "bf16"
    if op.startswith("norm"):
        M, D = _log(rng, 1, 16896), _log(rng, 32, 8192)
        if rng.random() < 0.5:
            D = max(32, D // 8 * 8)
        M = max(1, min(M, 16896 * 1536 // D))
        G = min(M, _log(rng, 1, 16))
        return dict(op=op, dtype=dtype, res=rng.choice(("fp32", dtype)), M=M, G=-(-M // -(-M // G)), D=D, post=rng.random() < 0.6,
                    gate=rng.random() < 0.7, mod=rng.random() < 0.6, gain=rng.random() < 0.6)
    M = _log(rng, 1, 16896) if op in ("linear", "gated") else _log(rng, 32, 8448)
    K, N = _log(rng, 64, 6144), _log(rng, 64, 6144)
    if rng.random() < 0.85:  # widths are whole numbers of 16-byte vectors, as models have them; now and then they are not
        K = K // 8 * 8
    if rng.random() < 0.6:
        N = N // 8 * 8
    most = 2.0e10 if dtype == "fp32" else 8.0e10 if op in ("linear", "gated") else 4.0e10  # products of one direction
    if K % 8:
        most = 2.0e10
    M = max(1, min(M, int(most / (N * K))))
    if op == "linear":
        out = rng.choice(("fp32", dtype))
        return dict(op=op, dtype=dtype, out=out, act=rng.choice(ACTS), M=M, N=N, K=K, res=rng.random() < 0.5, save=rng.random() < 0.3)
    if op == "linear_bwd":
        return dict(op=op, dtype=dtype, out=rng.choice(("fp32", dtype)), act=rng.choice(ACTS), M=M, N=N, K=K)
    if op == "gated":
        return dict(op=op, dtype=dtype, act=rng.choice(GATES), M=M, F=N, K=K, bias=rng.random() < 0.5, save=rng.random() < 0.5)
    return dict(op=op, dtype=dtype, act=rng.choice(GATES), M=M, F=N, K=K, bias=rng.random() < 0.5)


def work(case):
    c, e = case, SIZE[case["dtype"]]
    M = c["M"]
    if c["op"] in ("linear", "linear_bwd"):
        N, K, o = c["N"], c["K"], SIZE[c["out"]]
        if c["op"] == "linear":
            return {"bytes": (M * K + N * K) * e + 4 * N + M * N * (o * (2 if c["res"] else 1) + (e if c["save"] else 0)), "flops": 2.0 * M * N * K}
        return {"bytes": 2 * (M * K + N * K) * e + M * N * (o + (e if c["act"] != "none" else 0)) + 4 * N, "flops": 4.0 * M * N * K}
    if c["op"] in ("gated", "gated_bwd"):
        F, K = c["F"], c["K"]
        if c["op"] == "gated":
            return {"bytes": (M * K + 2 * F * K + M * F * (3 if c["save"] else 1)) * e + (8 * F if c["bias"] else 0), "flops": 4.0 * M * F * K}
        return {"bytes": (2 * M * K + 4 * F * K + 3 * M * F) * e + (8 * F if c["bias"] else 0), "flops": 8.0 * M * F * K}
    D, r = c["D"], SIZE[c["res"]]
    vec = 4 * D * (c["G"] * (c["gate"] + 2 * c["mod"]) + c["post"] + c["gain"])
    if c["op"] == "norm":
        return {"bytes": M * D * (2 * r + 2 * e) + vec, "flops": 12.0 * M * D}
    return {"bytes": M * D * (3 * r + 3 * e) + 2 * vec, "flops": 30.0 * M * D}


# ----------------------------------------------------------------- the inputs
def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device=DEV) * std + mean).to(dtype)

    t, M = TYPES[c["dtype"]], c["M"]
    s = {"case": dict(c)}
    if c["op"] in ("linear", "linear_bwd"):
        N, K, o = c["N"], c["K"], TYPES[c["out"]]
        s["x"] = normal(M, K, dtype=t)
        s["w"] = normal(N, K, std=K ** -0.5, dtype=t)
        if c["op"] == "linear":
            s["bias"] = normal(N, std=0.1)
            s["res"] = normal(M, N, dtype=o) if c["res"] else None
        else:
            s["z"] = normal(M, N, dtype=t) if c["act"] != "none" else None
            s["dy"] = normal(M, N, dtype=o)
    elif c["op"] in ("gated", "gated_bwd"):
        F, K = c["F"], c["K"]
        s["x"] = normal(M, K, dtype=t)
        s["wg"] = normal(F, K, std=K ** -0.5, dtype=t)
        s["wu"] = normal(F, K, std=K ** -0.5, dtype=t)
        if c["op"] == "gated":
            s["bg"] = normal(F, std=0.1) if c["bias"] else None
            s["bu"] = normal(F, std=0.1) if c["bias"] else None
        else:
            s["g"] = normal(M, F, dtype=t)
            s["u"] = normal(M, F, dtype=t)
            s["da"] = normal(M, F, dtype=t)
    else:
        D, r = c["D"], TYPES[c["res"]]
        s["x"] = normal(M, D, std=2.0, dtype=r)  # the stream: s itself in the backward cases
        s["y"] = normal(M, D, std=0.7, dtype=t)
        s["post_gain"] = normal(D, std=0.2, mean=1.0) if c["post"] else None
        s["gain"] = normal(D, std=0.2, mean=1.0) if c["gain"] else None
        table = normal(c["G"], 3, D, std=0.5)  # gate, scale and shift lie in one table, as a modulation map writes them
        s["gate"] = table[:, 0] if c["gate"] else None
        s["scale"], s["shift"] = (table[:, 1], table[:, 2]) if c["mod"] else (None, None)
        if c["op"] == "norm_bwd":
            s["dh"] = normal(M, D, dtype=t)
            s["ds"] = normal(M, D, dtype=r)
    return s


# ------------------------------------------------------------- the plain form
def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return z.clamp(min=0)
    if act == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))


def _act_grad(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "sigmoid":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 - p)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)


def _rows(v, M):
    """A vector per group, spread over the rows of its group."""
    per = -(-M // v.shape[0])
    return v.repeat_interleave(per, 0)[:M]


def _over_groups(v, G):
    """The sum over the rows of each group (the last one may be short)."""
    M, D = v.shape
    per = -(-M // G)
    whole = torch.zeros(G * per, D, device=v.device, dtype=v.dtype)
    whole[:M] = v
    return whole.view(G, per, D).sum(1)


def _plain(s):
    c = s["case"]
    t = TYPES[c["dtype"]]
    if c["op"] == "linear":
        z = s["x"].float() @ s["w"].float().t() + s["bias"]
        y = _act(z, c["act"])
        if s["res"] is not None:
            y = y + s["res"].float()
        out = {"y": y.to(TYPES[c["out"]])}
        if c["save"]:
            out["z"] = z.to(t)
        return out
    if c["op"] == "linear_bwd":
        dz = s["dy"].float()
        if s["z"] is not None:
            dz = dz * _act_grad(s["z"].float(), c["act"])
        return {"dx": (dz @ s["w"].float()).to(t), "dw": (dz.t() @ s["x"].float()).to(t), "db": dz.sum(0)}
    if c["op"] == "gated":
        x = s["x"].float()
        g, u = x @ s["wg"].float().t(), x @ s["wu"].float().t()
        if s["bg"] is not None:
            g, u = g + s["bg"], u + s["bu"]
        out = {"a": (_act(g, c["act"]) * u).to(t)}
        if c["save"]:
            out["g"], out["u"] = g.to(t), u.to(t)
        return out
    if c["op"] == "gated_bwd":
        g, u, da, x = s["g"].float(), s["u"].float(), s["da"].float(), s["x"].float()
        dg, du = da * u * _act_grad(g, c["act"]), da * _act(g, c["act"])
        out = {"dx": (dg @ s["wg"].float() + du @ s["wu"].float()).to(t), "dwg": (dg.t() @ x).to(t), "dwu": (du.t() @ x).to(t)}
        if c["bias"]:
            out["dbg"], out["dbu"] = dg.sum(0), du.sum(0)
        return out
    M, D, G = c["M"], c["D"], c["G"]
    x, y, r = s["x"].float(), s["y"].float(), TYPES[c["res"]]
    gain = s["gain"] if s["gain"] is not None else 1.0
    mul = gain * (1 + _rows(s["scale"], M)) if s["scale"] is not None else gain
    gate = _rows(s["gate"], M) if s["gate"] is not None else 1.0
    ry = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
    if c["op"] == "norm":
        p = y * ry * s["post_gain"] if c["post"] else y
        v = x + gate * p
        h = v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * mul
        if s["shift"] is not None:
            h = h + _rows(s["shift"], M)
        return {"s": v.to(r), "h": h.to(t)}
    dh = s["dh"].float()
    rx = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    n = x * rx
    dn = dh * mul
    dv = s["ds"].float() + rx * (dn - n * (dn * n).mean(1, keepdim=True))
    out = {"dx": dv.to(r)}
    dp = dv * gate
    if c["post"]:
        ny = y * ry
        out["dpost_gain"] = (dp * ny).sum(0)
        dny = dp * s["post_gain"]
        out["dy"] = (ry * (dny - ny * (dny * ny).mean(1, keepdim=True))).to(t)
        p = ny * s["post_gain"]
    else:
        out["dy"] = dp.to(t)
        p = y
    if s["gate"] is not None:
        out["dgate"] = _over_groups(dv * p, G)
    if s["gain"] is not None:
        out["dgain"] = (dh * n * (1 + _rows(s["scale"], M)) if s["scale"] is not None else dh * n).sum(0)
    if s["scale"] is not None:
        out["dscale"] = _over_groups(dh * n * gain, G)
        out["dshift"] = _over_groups(dh, G)
    return out


# ------------------------------------------------------ the framework's calls
def _buffer(s, name, shape, dtype):
    """An output or a workspace that a program keeps from step to step."""
    if name not in s:
        s[name] = torch.empty(shape, dtype=dtype, device=DEV)
    return s[name]


def _own(s):
    import mot_dit_b200 as W

    c = s["case"]
    t, M = TYPES[c["dtype"]], c["M"]
    code = {"bf16": W.BF16, "fp32": W.FP32}
    dtype = code[c["dtype"]]
    if c["op"] in ("linear", "linear_bwd"):
        N, K, act = c["N"], c["K"], W.ACTS.index(c["act"])
        if c["op"] == "linear":
            y = _buffer(s, "o_y", (M, N), TYPES[c["out"]])
            z = _buffer(s, "o_z", (M, N), t) if c["save"] else None
            W.op_linear_act(dtype, s["x"], s["w"], s["bias"], y, M, N, K, act=act, residual=s["res"], z=z, out_dtype=code[c["out"]])
            return {"y": y, "z": z} if c["save"] else {"y": y}
        out = {"dx": _buffer(s, "o_dx", (M, K), t), "dw": _buffer(s, "o_dw", (N, K), t), "db": _buffer(s, "o_db", (N,), torch.float32)}
        if "ws" not in s:
            _buffer(s, "ws", (W.op_linear_act_workspace(dtype, M, N, K, act=act, dy_dtype=code[c["out"]]),), torch.uint8)
        W.op_linear_act_backward(dtype, s["x"], s["w"], s["z"], s["dy"], out["dx"], out["dw"], out["db"], M, N, K, act=act,
                                 dy_dtype=code[c["out"]], workspace=s["ws"])
        return out
    if c["op"] in ("gated", "gated_bwd"):
        F, K, act = c["F"], c["K"], W.ACTS.index(c["act"])
        if c["op"] == "gated":
            out = {"a": _buffer(s, "o_a", (M, F), t)}
            if c["save"]:
                out["g"], out["u"] = _buffer(s, "o_g", (M, F), t), _buffer(s, "o_u", (M, F), t)
            W.op_gated(dtype, s["x"], s["wg"], s["wu"], out["a"], M, F, K, act=act, bias_g=s["bg"], bias_u=s["bu"], g=out.get("g"), u=out.get("u"))
            return out
        out = {"dx": _buffer(s, "o_dx", (M, K), t), "dwg": _buffer(s, "o_dwg", (F, K), t), "dwu": _buffer(s, "o_dwu", (F, K), t)}
        if c["bias"]:
            out["dbg"], out["dbu"] = _buffer(s, "o_dbg", (F,), torch.float32), _buffer(s, "o_dbu", (F,), torch.float32)
        if "ws" not in s:
            _buffer(s, "ws", (W.op_gated_workspace(dtype, M, F, K),), torch.uint8)
        W.op_gated_backward(dtype, s["x"], s["wg"], s["wu"], s["g"], s["u"], s["da"], out["dx"], out["dwg"], out["dwu"], M, F, K, act=act,
                            dbias_g=out.get("dbg"), dbias_u=out.get("dbu"), workspace=s["ws"])
        return out
    D, G, r = c["D"], c["G"], TYPES[c["res"]]
    vec = dict(post_gain=s["post_gain"], gate=s["gate"], gain=s["gain"], scale=s["scale"], shift=s["shift"], post_norm=c["post"],
               rows_per_group=-(-M // G), ld_mod=3 * D, res_dtype=code[c["res"]])
    if c["op"] == "norm":
        out = {"s": _buffer(s, "o_s", (M, D), r), "h": _buffer(s, "o_h", (M, D), t)}
        W.op_residual_norm(dtype, s["x"], s["y"], out["s"], out["h"], M, D, **vec)
        return out
    out = {"dx": _buffer(s, "o_dx", (M, D), r), "dy": _buffer(s, "o_dy", (M, D), t)}
    for name, given, shape in (("dpost_gain", s["post_gain"], (D,)), ("dgate", s["gate"], (G, D)), ("dgain", s["gain"], (D,)),
                               ("dscale", s["scale"], (G, D)), ("dshift", s["shift"], (G, D))):
        if given is not None:
            out[name] = _buffer(s, "o_" + name, shape, torch.float32)
    if "ws" not in s:
        _buffer(s, "ws", (W.op_residual_norm_workspace(M, D, rows_per_group=-(-M // G)),), torch.uint8)
    W.op_residual_norm_backward(dtype, s["x"], s["y"], s["ds"], s["dh"], out["dx"], out["dy"], M, D, dpost_gain=out.get("dpost_gain"),
                                dgate=out.get("dgate"), dgain=out.get("dgain"), dscale=out.get("dscale"), dshift=out.get("dshift"),
                                workspace=s["ws"], **{k: v for k, v in vec.items() if k != "shift"})
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------- the definition, in 64 bits
def _act64(z, act):
    f = torch.nn.functional
    return {"none": lambda: z, "relu": lambda: f.relu(z), "sigmoid": lambda: torch.sigmoid(z), "silu": lambda: f.silu(z),
            "gelu_tanh": lambda: f.gelu(z, approximate="tanh"), "gelu_erf": lambda: f.gelu(z)}[act]()


def _norm64(c, x, y, post_gain, gate, gain, scale, shift):
    """(s, h) of the definition, row group by row group."""
    M, G = x.shape[0], c["G"]
    per = -(-M // G)
    rms = lambda v: v / torch.sqrt((v ** 2).mean(-1, keepdim=True) + EPS)  # noqa: E731
    out_s, out_h = [], []
    for k in range(G):
        xs, p = x[k * per:(k + 1) * per], y[k * per:(k + 1) * per]
        if c["post"]:
            p = rms(p) * post_gain
        v = xs + (p * gate[k] if gate is not None else p)
        h = rms(v)
        if gain is not None:
            h = h * gain
        if scale is not None:
            h = h * (1 + scale[k]) + shift[k]
        out_s.append(v)
        out_h.append(h)
    return torch.cat(out_s), torch.cat(out_h)


def exact(case, seed):
    c = case
    s = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in prepare(case, seed).items()}
    if c["op"] == "linear":
        z = torch.addmm(s["bias"], s["x"], s["w"].t())
        y = _act64(z, c["act"])
        if s["res"] is not None:
            y = y + s["res"]
        return {"y": y, "z": z} if c["save"] else {"y": y}
    if c["op"] == "linear_bwd":
        dz = s["dy"]
        if s["z"] is not None:
            z = s["z"].requires_grad_()
            dz, = torch.autograd.grad(_act64(z, c["act"]), z, dz)
        return {"dx": torch.mm(dz, s["w"]), "dw": torch.mm(dz.t(), s["x"]), "db": dz.sum(0)}
    if c["op"] == "gated":
        g, u = torch.mm(s["x"], s["wg"].t()), torch.mm(s["x"], s["wu"].t())
        if s["bg"] is not None:
            g, u = g + s["bg"], u + s["bu"]
        a = _act64(g, c["act"]) * u
        return {"a": a, "g": g, "u": u} if c["save"] else {"a": a}
    if c["op"] == "gated_bwd":
        g, u = s["g"].requires_grad_(), s["u"].requires_grad_()
        dg, du = torch.autograd.grad(_act64(g, c["act"]) * u, (g, u), s["da"])
        out = {"dx": torch.mm(dg, s["wg"]) + torch.mm(du, s["wu"]), "dwg": torch.mm(dg.t(), s["x"]), "dwu": torch.mm(du.t(), s["x"])}
        return {**out, "dbg": dg.sum(0), "dbu": du.sum(0)} if c["bias"] else out
    vec = {k: s[k].clone().requires_grad_() for k in ("post_gain", "gate", "gain", "scale", "shift") if s[k] is not None}
    full = {k: vec.get(k) for k in ("post_gain", "gate", "gain", "scale", "shift")}
    if c["op"] == "norm":
        with torch.no_grad():
            v, h = _norm64(c, s["x"], s["y"], **full)
        return {"s": v, "h": h}
    # The gradient at the point whose stream value is the given one: x is chosen so that s comes out as it.
    y = s["y"].requires_grad_()
    with torch.no_grad():
        v0, _ = _norm64(c, torch.zeros_like(s["x"]), y, **full)
    x = (s["x"] - v0).requires_grad_()
    v, h = _norm64(c, x, y, **full)
    names = [k for k in ("post_gain", "gate", "gain", "scale", "shift") if k in vec]
    got = torch.autograd.grad([v, h], [x, y] + [vec[k] for k in names], [s["ds"], s["dh"]])
    return {"dx": got[0], "dy": got[1], **{"d" + k: d for k, d in zip(names, got[2:])}}
